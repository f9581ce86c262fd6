"""Bounded waits of the product's kernels: with the wait limit at zero a kernel
gives up on its first unsatisfied wait, records CONV_ERR_TIMEOUT in the device
status word, drains its copies and MMAs in flight, frees its tensor memory and
returns.  The context stays usable: the next call at the normal limit is
correct."""
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


# one CTA a tile, a cluster a tile, CTA pairs
@pytest.mark.parametrize("m,n,k", [(128, 14000, 4096), (64, 256, 8192), (1100, 2048, 2048)])
@pytest.mark.parametrize("q", [torch.int8, torch.float8_e4m3fn])
def test_forced_wait_timeout_reports_status_and_recovers(pkg, m, n, k, q):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = (torch.randn(m, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    w = (torch.randn(n, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    ref.check_linear(pkg.linear_w8a8(x, w), x, w)
    assert pkg.conv_get_device_status() == 0
    try:
        pkg.conv_set_wait_limit_ns(0)
        pkg.linear_w8a8(x, w)
        status = pkg.conv_get_device_status()
    finally:
        pkg.conv_set_wait_limit_ns(2_000_000_000)
    assert status == pkg.CONV_ERR_TIMEOUT
    y = pkg.linear_w8a8(x, w)
    assert pkg.conv_get_device_status() == 0
    ref.check_linear(y, x, w)
