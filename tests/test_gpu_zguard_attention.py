"""Bounded waits of packed_attention and paged_attention: with the wait limit at zero the kernel gives up
on its first unsatisfied wait, records CONV_ERR_TIMEOUT in the device status word,
drains its copies and products in flight, frees its tensor memory and returns.  The
next call at the normal limit is right."""
import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    return p


@pytest.mark.parametrize("lens,heads", [([300, 100], 4), ([1100, 1500], 32)])
@pytest.mark.parametrize("width", [64, 128])
def test_forced_wait_timeout_reports_status_and_recovers(pkg, lens, heads, width):
    g = torch.Generator(device="cuda").manual_seed(width)
    n = sum(lens)
    q, k, v = (torch.randn(n, heads, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    off = torch.tensor([0, lens[0], n], dtype=torch.int32, device="cuda")
    want = pkg.packed_attention(q, k, v, off)
    assert pkg.conv_get_device_status() == 0
    try:
        pkg.conv_set_wait_limit_ns(0)
        pkg.packed_attention(q, k, v, off)
        status = pkg.conv_get_device_status()
    finally:
        pkg.conv_set_wait_limit_ns(2_000_000_000)
    assert status == pkg.CONV_ERR_TIMEOUT
    got = pkg.packed_attention(q, k, v, off)
    assert pkg.conv_get_device_status() == 0
    assert torch.equal(got, want)
    a = lens[0]
    ref_, tol = ref.attention64(q[:a], k[:a], v[:a], causal=False, weights=torch.bfloat16)
    ref.check(got[:a], ref_, tol)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
def test_paged_without_a_wait_is_right_or_says_so(pkg, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    lens, page, per = [3000, 4096, 17], 16, 256
    k, v = (torch.randint(-9, 10, (3 * per, 4, page, 128), generator=g, device="cuda").to(dtype) for _ in range(2))
    s = torch.full((3 * per, 4, page), 0.1, device="cuda") if dtype is torch.int8 else None
    q = torch.randn(3, 8, 128, generator=g, device="cuda").bfloat16()
    table = torch.randperm(3 * per, generator=g, device="cuda").int().view(3, per)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    run = lambda: pkg.paged_attention(q, k, v, table, n, k_scale=s, v_scale=s)   # noqa: E731
    want = run()
    assert pkg.conv_get_device_status() == 0
    try:
        pkg.conv_set_wait_limit_ns(0)
        got = run()
        status = pkg.conv_get_device_status()
    finally:
        pkg.conv_set_wait_limit_ns(2_000_000_000)
    # a load may have landed before the first look at its barrier: then nothing was waited for
    assert status == pkg.CONV_ERR_TIMEOUT or (status == 0 and torch.equal(got, want))
    got = run()
    assert pkg.conv_get_device_status() == 0
    assert torch.equal(got, want)
