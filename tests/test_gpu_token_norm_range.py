"""rms_norm_quant over the whole fp32 range: mean squares about the largest fp32
number, rows of zeros and rows whose squares underflow, with and without eps.

Tolerances as in _token_ref: v is within (width/32 + 64) 2^-24."""
import math

import pytest
import torch

import _token_ref as ref

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.float8_e4m3fn
BF, FF = torch.bfloat16, torch.float32
WIDTHS = [1, 8, 33, 640, 999, 1280, 2048, 5120, 40000]


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _blank(codes):
    return not codes.view(torch.uint8).any()


# sqrt of the largest fp32 number is 1.8447e19
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("with_residual", [False, True])
def test_mean_square_about_the_largest_number(pkg, width, q, with_residual):
    """Rows of one magnitude: those whose mean square is beyond fp32 are marked,
    those just below it have v = 1 everywhere."""
    mags = [1.8e19, 1.85e19, 1.9e19, 2.0e19, 2.3e19, 2.5e19, 3.6e19, 3e38, 1.0]
    x = torch.tensor(mags, device="cuda")[:, None].expand(-1, width).contiguous()
    res = None
    if with_residual:
        res = 0.25 * x
        x = 0.75 * x
    codes, scale, _ = pkg.rms_norm_quant(x, residual=res, qdtype=q)
    qmax = ref.QMAX[q]
    for r, m in enumerate(mags):
        if 1.8e19 < m:
            assert math.isnan(float(scale[r])) and _blank(codes[r]), (m, float(scale[r]))
        else:
            assert abs(float(scale[r]) * qmax - 1) < (width / 32 + 64) * 2.0 ** -24
            assert (codes[r].double() == qmax).all(), m


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("x_type", [BF, FF])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_zero_rows_at_any_eps(pkg, width, q, x_type, eps):
    """A row of zeros has scale 1 and codes 0 whatever eps is; its neighbours are
    as they would be without it."""
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(4, width, generator=g, device="cuda").to(x_type)
    x[x == 0] = 1
    x[1] = 0
    x[3] = -0.0
    w = torch.randn(width, generator=g, device="cuda").to(x_type)
    w[w == 0] = 1
    for weight in (None, w):
        codes, scale, _ = pkg.rms_norm_quant(x, weight, eps, qdtype=q)
        for r in (1, 3):
            assert float(scale[r]) == 1.0 and _blank(codes[r])
        _, v = ref.norm64(x[::2], weight, eps, None)
        ref.check_quant(v, codes.view(torch.uint8)[::2].view(q), scale[::2],
                        (width / 32 + 64) * 2.0 ** -24)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30])
def test_rows_whose_squares_underflow(pkg, width, q, eps):
    """Rows far below 1 with an eps that does not hide them: the mean square is
    taken as if fp32 had no lower end."""
    g = torch.Generator(device="cuda").manual_seed(width + 1)
    mags = torch.tensor([1.0, 1e-9, 3e-10, 1e-15, 1e-19, 1e-22, 1e-25, 1e-30, 1e-36], device="cuda")
    x = torch.randn(len(mags), width, generator=g, device="cuda")
    x = torch.where(x.abs() < 0.1, torch.ones_like(x), x) * mags[:, None]
    w = 1 + 0.25 * torch.rand(width, generator=g, device="cuda")
    res = (x * torch.rand(x.shape, generator=g, device="cuda")).contiguous()
    for weight, residual in ((None, None), (w, res)):
        codes, scale, _ = pkg.rms_norm_quant(x, weight, eps, residual=residual, qdtype=q)
        # the sum itself is rounded to fp32: h of the reference is that sum
        h = x if residual is None else x + residual
        _, v = ref.norm64(h, weight, eps, None)
        keep = v.abs().amax(1) > 1e-30     # below: the scale's own lower end
        ref.check_quant(v[keep], codes.view(torch.uint8)[keep].view(q), scale[keep],
                        (width / 32 + 64) * 2.0 ** -24)
        assert torch.isfinite(scale).all()


def test_row_of_almost_two_to_the_31(pkg):
    """One row whose width is within a block's stride of 2^31: a few elements that
    are not zero, at both ends and about 2^30."""
    width = 2 ** 31 - 7
    at = torch.tensor([0, 1023, 1024, 2 ** 30 - 1, 2 ** 30, width - 1025, width - 1024, width - 1],
                      device="cuda")
    values = torch.tensor([1.0, -2.0, 3.0, -4.0, 5.0, -6.0, 7.0, -8.0], device="cuda")
    x = torch.zeros(1, width, dtype=BF, device="cuda")
    x[0, at] = values.to(BF)
    codes, scale, _ = pkg.rms_norm_quant(x, eps=1e-12)
    v = values.double() / math.sqrt(float((values.double() ** 2).sum()) / width + 1e-12)
    assert abs(float(scale) * 127 / float(v.abs().max()) - 1) < 64 * 2.0 ** -24
    assert torch.equal(codes[0, at].double(), torch.round(v / v.abs().max() * 127))
    assert int((codes != 0).sum()) == len(at)
