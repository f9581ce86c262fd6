"""paged_attention with a workspace of exactly the bytes that were asked for, 0 among them."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages,bytes_", [(4, "asked"), (40, "asked"), (40, "less")])
def test_workspace_of_the_bytes_asked_for(pkg, pages, bytes_):
    """At the C ABI: a buffer of exactly the size that was queried, 0 bytes too, will do."""
    from implicit_gemm_convolution_conv3d_gb300 import token_attention as t
    lib = t._bind()
    heads, kv, width, page = 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(pages)
    k, v = (torch.randn(2 * pages, kv, page, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(2, heads, width, generator=g, device="cuda").bfloat16()
    table = torch.randperm(2 * pages, generator=g, device="cuda").int().view(2, pages)
    lengths = _ints([pages * page, 5])
    want = pkg.paged_attention(q, k, v, table, lengths)
    need = pkg.paged_attention_workspace_size(2, heads, kv, width, page, pages)
    assert (need == 0) == (pages == 4)
    buf = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    size = need if bytes_ == "asked" else need - 1
    st = lib.paged_attention_fwd(
        q.data_ptr(), 0, heads * width, width, ctypes.byref(t._cache(k, v, None, None)), table.data_ptr(), pages, pages,
        lengths.data_ptr(), None, None, width ** -0.5, 0.0, 0, 2, heads, out.data_ptr(), heads * width, width,
        buf.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    if bytes_ == "less":
        assert st == 1 and not out.any()
    else:
        assert st == 0 and torch.equal(out, want)
