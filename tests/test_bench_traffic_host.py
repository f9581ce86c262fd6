"""The bench's measured DRAM traffic belongs to the sources that are there."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_committed_traffic_is_of_the_present_sources():
    committed = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))
    for workload, entry in committed.items():
        assert bench.measured_traffic(workload) == entry["dram_bytes_per_step"], (
            f"{workload}: measured on sources {entry['kernel_sha']}, "
            f"present ones are {bench.kernel_source_sha()}")
