"""rms_norm_quant over the whole fp32 range: mean squares about the largest fp32
number.

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
