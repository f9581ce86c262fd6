"""GELU and SiLU of linear_w8a8's outputs: relative accuracy in the negative tail
for every output type, and -inf."""
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


# up to 16 tokens; one wave of tiles; CTA pairs (n: more than 152 tiles), output rows
# that TMA can and cannot address
FORMS = [(3, 200), (40, 200), (300, 8192), (700, 8191)]


@pytest.mark.parametrize("m,n", FORMS)
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("out_dtype", [BF, HF, FF])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_negative_tails(pkg, m, n, q, out_dtype, act):
    """One product per output, so that y is three roundings from exact.  The
    activation's relative condition in the tail is y^2 (GELU) or |y| (SiLU); its
    evaluation adds a few units, times the argument's size in the exponential:
    |y| 2^-22 (SiLU, 16 bits), y^2 2^-24 (GELU)."""
    low = 13.0 if act == "gelu" else 80.0
    x = torch.ones(m, 16, device="cuda")
    x[:, 1:] = 0
    w = torch.zeros(n, 16, device="cuda")
    w[:, 0] = -(torch.arange(n, device="cuda") % 15 + 1).float()
    sw = torch.ones(n, device="cuda")
    sx = torch.linspace(0.001, low / 15, m, device="cuda")
    got = pkg.linear_w8a8(x.to(q), w.to(q), sx, sw, act=act, out_dtype=out_dtype)
    y = sx.double()[:, None] * w[:, 0].double()
    want = ref.act64(y, act)
    tol = want.abs() * (8 + 2 * (y * y if act == "gelu" else y.abs())) * 2.0 ** -22
    ref.check_rounded(got, want, tol)


@pytest.mark.parametrize("m,n", FORMS)
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("out_dtype", [BF, HF, FF])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_infinite_arguments(pkg, m, n, q, out_dtype, act):
    """A bias of -inf is -inf, max(-inf, 0) = 0, or NaN (a product with 0); +inf
    stays +inf; other columns are as they were."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randint(-3, 4, (m, 32), generator=g, device="cuda").float().to(q)
    w = torch.randint(-3, 4, (n, 32), generator=g, device="cuda").float().to(q)
    bias = torch.randn(n, generator=g, device="cuda")
    clean = pkg.linear_w8a8(x, w, bias=bias, act=act, out_dtype=out_dtype)
    bad = bias.clone()
    bad[5], bad[n - 1] = -math.inf, math.inf
    got = pkg.linear_w8a8(x, w, bias=bad, act=act, out_dtype=out_dtype)
    if act == "none":
        assert (got[:, 5] == -math.inf).all()
    elif act == "relu":
        assert (got[:, 5] == 0).all()
    else:
        assert torch.isnan(got[:, 5]).all()
    assert (got[:, n - 1] == math.inf).all()
    keep = [c for c in range(n) if c not in (5, n - 1)]
    assert torch.equal(got[:, keep], clean[:, keep])
