"""Rows that packed_attention computes again, next to values that are not finite, may take
longer than the bound on its waits: the warps that wait for them see that they go on."""
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


def test_rows_computed_again_outlast_the_waits(pkg):
    """127 rows of each head over 30000 keys, 32 rows a warp: some 130 ms a job, several jobs a
    CTA and a bound of 5 ms; the call without such rows takes 1 ms."""
    nk, nq, heads, width = 30000, 300, 160, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(nq, heads, width, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(nk, 1, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    off, koff = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (nq, nk))
    want = pkg.packed_attention(q, k, v, off, koff, causal=True)
    v[-1] = float("nan")
    v[-45] = float("inf")
    try:
        pkg.conv_set_wait_limit_ns(5_000_000)
        got = pkg.packed_attention(q, k, v, off, koff, causal=True)
        torch.cuda.synchronize()
        assert pkg.conv_get_device_status() == 0
    finally:
        pkg.conv_set_wait_limit_ns(2_000_000_000)
    assert torch.equal(got[:128], want[:128])        # (their tiles do not reach those keys)
    assert not torch.isfinite(got[-44:]).all(-1).any()
    rows = slice(nq - 127, nq - 45)
    for h in (0, heads - 1):
        ref_, tol = ref.attention64(q[:nq - 45, h:h + 1], k[:-45], v[:-45], causal=True, weights=torch.bfloat16)
        ref.check(got[rows, h:h + 1], ref_[rows], tol[rows])
