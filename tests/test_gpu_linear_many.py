"""linear_w8a8 in its form for many tokens (CTA pairs: more than 256 tokens and
more than 152 tiles of 128 x 128): output rows that TMA can and cannot address,
outputs and operands of any stride and alignment, in both types of codes."""
import math

import pytest
import torch

import _token_ref as ref

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.float8_e4m3fn
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _operands(m, n, k, q):
    assert m > 256 and -(-m // 128) * -(-n // 128) > 152
    g = torch.Generator(device="cuda").manual_seed(m + 3 * n + k)
    make = lambda r: torch.randint(-127, 128, (r, k), generator=g, device="cuda").to(I8) \
        if q == I8 else (torch.randn(r, k, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4)  # noqa: E731
    sx = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.001
    sw = (torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001) / math.sqrt(k)
    return make(m), make(n), sx, sw, torch.randn(n, generator=g, device="cuda")


def _view(t, pad, off):
    """The same bytes as rows `pad` longer that start `off` bytes in."""
    rows, width = t.shape
    flat = torch.full((rows * (width + pad) + off,), 0x55, dtype=torch.uint8, device="cuda")
    v = flat[off:].view(rows, width + pad)[:, :width]
    v.copy_(t.view(torch.uint8))
    return v.view(t.dtype)


# n: rows of 16-byte multiples or not, the last tile full, of one column, of 32 and odd
@pytest.mark.parametrize("m,n,k", [(1000, 2501, 320), (1025, 2304, 128), (2500, 1281, 1283),
                                   (300, 8200, 272), (257, 6943, 64), (700, 3360, 2064)])
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("out_dtype", [BF, HF, FF])
@pytest.mark.parametrize("bias,act", [(False, "none"), (True, "gelu"), (True, "relu"),
                                      (False, "silu")])
def test_outputs(pkg, m, n, k, q, out_dtype, bias, act):
    x, w, sx, sw, b = _operands(m, n, k, q)
    b = b if bias else None
    got = pkg.linear_w8a8(x, w, sx, sw, bias=b, act=act, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    ref.check_linear(got, x, w, sx, sw, b, act)


# the output inside a wider matrix: `left` elements before it, rows `more` longer
@pytest.mark.parametrize("n,left,more", [(2504, 16, 40), (2504, 8, 8), (2503, 16, 41),
                                         (2504, 1, 3), (2501, 3, 4)])
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("out_dtype", [BF, FF])
def test_strided_outputs(pkg, n, left, more, q, out_dtype):
    """The columns beside the rows and the row after them stay."""
    m, k = 1000, 336
    x, w, sx, sw, b = _operands(m, n, k, q)
    buf = torch.full((m + 1, left + n + more), 3.0, dtype=out_dtype, device="cuda")
    got = pkg.linear_w8a8(x, w, sx, sw, bias=b, out=buf[:m, left:left + n])
    ref.check_linear(got, x, w, sx, sw, b)
    assert torch.equal(got, pkg.linear_w8a8(x, w, sx, sw, bias=b, out_dtype=out_dtype))
    assert (buf[:, :left] == 3).all() and (buf[:, left + n:] == 3).all() and (buf[m] == 3).all()


# row padding and offset in bytes of the tokens, of the weights
@pytest.mark.parametrize("px,ox,pw,ow", [(3, 0, 0, 0), (0, 1, 0, 0), (0, 0, 5, 2), (7, 3, 1, 9),
                                         (16, 16, 32, 0), (0, 0, 16, 16), (0, 0, 0, 8)])
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("k", [656, 1283])
@pytest.mark.parametrize("n", [2048, 2501])
def test_unaligned_operands(pkg, px, ox, pw, ow, q, k, n):
    """Staged tokens and weights (int8 weights are widened in the same launch), and
    operands that are read in place: the same bits."""
    m = 1300
    x, w, sx, sw, _ = _operands(m, n, k, q)
    want = pkg.linear_w8a8(_view(x, -k % 16, 0), _view(w, -k % 16, 0), sx, sw)
    got = pkg.linear_w8a8(_view(x, px, ox), _view(w, pw, ow), sx, sw)
    assert torch.equal(got, want)
    ref.check_linear(got, x, w, sx, sw)


# one wave of 128 x 128 tiles (clusters split the reduction): more tokens than 512 over
# few outputs, long and short reductions, as many tiles as there are SMs
@pytest.mark.parametrize("m,n,k", [(600, 640, 8192), (1024, 1024, 8192), (700, 1279, 1283),
                                   (2000, 640, 2560), (9500, 128, 1280), (19456, 100, 64),
                                   (513, 1, 4096), (1024, 2432, 144)])
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("out_dtype,act", [(BF, "gelu"), (FF, "none")])
def test_many_tokens_within_one_wave(pkg, m, n, k, q, out_dtype, act):
    assert -(-m // 128) * -(-n // 128) <= 152
    g = torch.Generator(device="cuda").manual_seed(m + n)
    make = lambda r: (torch.randn(r, k, generator=g, device="cuda") * 40).clamp(-127, 127).to(q)  # noqa: E731
    x, w = make(m), make(n)
    sx = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.001
    sw = (torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001) / math.sqrt(k)
    b = torch.randn(n, generator=g, device="cuda")
    got = pkg.linear_w8a8(x, w, sx, sw, bias=b, act=act, out_dtype=out_dtype)
    ref.check_linear(got, x, w, sx, sw, b, act)
    assert torch.equal(got, pkg.linear_w8a8(x, w, sx, sw, bias=b, act=act, out_dtype=out_dtype))
