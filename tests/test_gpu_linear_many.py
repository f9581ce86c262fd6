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
