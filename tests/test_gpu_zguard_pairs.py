"""Bounded waits of the product's kernels that run out at any point: a call either
finishes, and is right, or gives up, says so in the device status word within a
few seconds, and leaves nothing behind: the next call is right."""
import time

import pytest
import torch

import _token_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    return p


# CTA pairs for both types (more than 152 tiles of 128 x 128), one or several tiles a
# pair, fewer and more k-steps than the rings hold; clusters of 8, 4 and 1 CTA a tile
@pytest.mark.parametrize("m,n,k", [(2048, 2048, 2048), (4000, 3000, 640), (300, 8200, 256),
                                   (64, 256, 8192), (128, 4096, 4096), (100, 14000, 1024)])
@pytest.mark.parametrize("q", [torch.int8, torch.float8_e4m3fn])
def test_waits_that_run_out_midway(pkg, m, n, k, q):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = (torch.randn(m, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    w = (torch.randn(n, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    want = pkg.linear_w8a8(x, w)
    ref.check_linear(want, x, w)
    assert pkg.conv_get_device_status() == 0
    gave_up = 0
    for limit in (0, 300, 700, 1000, 1500, 2500, 5000, 0):
        try:
            pkg.conv_set_wait_limit_ns(limit)
            start = time.monotonic()
            got = pkg.linear_w8a8(x, w)
            status = pkg.conv_get_device_status()
            took = time.monotonic() - start
        finally:
            pkg.conv_set_wait_limit_ns(2_000_000_000)
        assert status in (0, pkg.CONV_ERR_TIMEOUT)
        assert took < 8.0
        if status == 0:
            assert torch.equal(got, want)
        gave_up += status != 0
        assert torch.equal(pkg.linear_w8a8(x, w), want)
        assert pkg.conv_get_device_status() == 0
    assert gave_up > 0


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 2048), (4000, 3000, 640)])
@pytest.mark.parametrize("q", [torch.int8, torch.float8_e4m3fn])
def test_pairs_give_up_at_once(pkg, m, n, k, q):
    """One CTA of a pair may give up earlier than the other: the loads that it never
    issued are not waited for."""
    x = torch.ones(m, k, device="cuda").to(q)
    w = torch.ones(n, k, device="cuda").to(q)
    pkg.linear_w8a8(x, w)
    assert pkg.conv_get_device_status() == 0
    try:
        for limit in (0, 300, 700, 1000, 1500, 2500, 5000) * 3:
            pkg.conv_set_wait_limit_ns(limit)
            start = time.monotonic()
            pkg.linear_w8a8(x, w)
            pkg.conv_get_device_status()
            assert time.monotonic() - start < 0.5, limit
    finally:
        pkg.conv_set_wait_limit_ns(2_000_000_000)
    assert (pkg.linear_w8a8(x, w) == k).all()
    assert pkg.conv_get_device_status() == 0
