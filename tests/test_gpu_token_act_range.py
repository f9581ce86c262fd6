"""act_quant at the ends of the range: -inf under each activation, and rows that
lie in an activation's vanishing tail, on both sides of the width that one
block holds in registers (32760)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.float8_e4m3fn
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
WIDTHS = [1, 24, 33, 4096, 5000, 32760, 32761, 40000]


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("x_type", [BF, HF, FF])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("q", [I8, E4])
def test_minus_infinity(pkg, width, x_type, act, gated, q):
    """-inf spoils its row under none, SiLU and GELU (its product with a sigmoid or
    a Phi of 0 is NaN), at any width; max(-inf, 0) is 0."""
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(3, 2 * width if gated else width, generator=g, device="cuda").to(x_type)
    x[:, 0] = 1
    if gated:
        x[:, width] = 1
    clean = pkg.act_quant(x, act=act, gated=gated, qdtype=q)
    bad = x.clone()
    bad[1, width - 1] = -math.inf
    codes, scale = pkg.act_quant(bad, act=act, gated=gated, qdtype=q)
    if act == "relu":
        same = x.clone()
        same[1, width - 1] = 0
        want = pkg.act_quant(same, act=act, gated=gated, qdtype=q)
        assert torch.equal(scale, want[1])
        assert (codes.double() == want[0].double()).all()
    else:
        assert math.isnan(float(scale[1])) and not codes[1].view(torch.uint8).any()
    for r in (0, 2):
        assert float(scale[r]) == float(clean[1][r])
        assert torch.equal(codes[r].view(torch.uint8), clean[0][r].view(torch.uint8))


@pytest.mark.parametrize("act,values", [
    ("silu", [-70.0, -86.0, -87.5, -88.0, -88.5, -90.0, -100.0, -104.0, -200.0, -1e30, -3.3e38]),
    ("gelu", [-5.0, -12.0, -13.0, -13.25, -13.5, -14.0, -14.5, -60.0, -70.0, -1e30, -3.3e38])])
@pytest.mark.parametrize("x_type", [BF, FF])
@pytest.mark.parametrize("q", [I8, E4])
def test_vanishing_tails_do_not_depend_on_the_width(pkg, act, values, x_type, q):
    """Rows of one value deep in the tail: the same scale and codes at every width,
    and within 2^-119 of the activation."""
    v = torch.tensor(values, device="cuda").to(x_type)
    narrow = pkg.act_quant(v[:, None].expand(-1, 64).contiguous(), act=act, qdtype=q)
    wide = pkg.act_quant(v[:, None].expand(-1, 33000).contiguous(), act=act, qdtype=q)
    assert torch.equal(narrow[1], wide[1])
    assert torch.equal(narrow[0][:, :1].double().expand(-1, 33000), wide[0].double())
    d = v.double()
    want = d * torch.sigmoid(d) if act == "silu" else 0.5 * d * torch.special.erfc(-d / 2 ** 0.5)
    got = narrow[0][:, 0].double() * narrow[1].double()
    # a row of one value has the largest code, and its scale has one rounding
    assert ((got - want).abs() <= 2.0 ** -119 + 2.0 ** -19 * want.abs()).all(), (got, want)
