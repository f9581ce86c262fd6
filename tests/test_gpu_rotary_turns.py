"""rotary's angles for slow, fast and negative frequencies at far positions, and the
kernels' trips over many heads."""
import math
from fractions import Fraction

import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def test_slow_and_negative_frequencies(pkg):
    """Against position * frequency in rational arithmetic.  The turn of a frequency is held
    to 2^-65 of a turn, so an angle is within 2 pi |position| 2^-65 beside its fp32 rounding
    and the sine's and cosine's (2^-20 with the products, as for near positions)."""
    freq = [1.0, 1e-4, -1e-4, 1e-7, -1e-7, -3e-10, 2e-13, -2e-13, -1.0, -0.7, 6.25, -6.25, 1e5, -1e9, -1e-20, 1e-25]
    far = [0, 1, -1, 12345, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 1, -2 ** 40 - 7, 2 ** 45 + 3]
    n = len(freq)
    x = torch.ones(len(far), 1, 2 * n, device="cuda")
    p = torch.tensor(far, dtype=torch.int64, device="cuda")
    got = pkg.rotary(x, p, (n,), pairs="interleaved", frequencies=freq).double().cpu()
    for t, pos in enumerate(far):
        for i, f in enumerate(freq):
            turn = Fraction(f) * pos / (2 * PI)
            a = float((turn - math.floor(turn)) * 2 * PI)
            tol = 2 * (2.0 ** -20 + 2 * math.pi * abs(pos) * 2.0 ** -65) + 2.0 ** -22
            assert abs(float(got[t, 0, 2 * i]) - (math.cos(a) - math.sin(a))) <= tol, (pos, f)
            assert abs(float(got[t, 0, 2 * i + 1]) - (math.cos(a) + math.sin(a))) <= tol, (pos, f)


def test_a_negative_frequency_turns_back(pkg):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(50, 3, 64, generator=g, device="cuda")
    p = torch.randint(-2 ** 40, 2 ** 40, (50, 1), generator=g, device="cuda")
    freq = [10.0 ** (-i / 4) for i in range(32)]
    back = pkg.rotary(x, p, (32,), frequencies=[-f for f in freq])
    assert torch.equal(back, pkg.rotary(x, p, (32,), frequencies=freq, inverse=True))


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("tokens,heads,width,sections", [
    (700, 48, 128, (16, 24, 24)), (900, 33, 64, (16, 16)), (700, 48, 72, (18, 18)), (1500, 40, 80, (33,))])
def test_many_heads(pkg, pairs, dtype, tokens, heads, width, sections):
    """Several trips over the heads by every thread: rows, in place and beside."""
    g = torch.Generator(device="cuda").manual_seed(tokens + width)
    x = torch.randn(tokens, heads, width, generator=g, device="cuda").to(dtype)
    p = torch.randint(-900, 900, (tokens, len(sections)), generator=g, device="cuda").int()
    axis, freq = ref.ladder64(sections)
    want, tol = ref.rotary64(x, p, axis, freq, pairs == "interleaved")
    got = pkg.rotary(x, p, sections, pairs=pairs)
    ref.check(got, want, tol)
    pkg.rotary(x, p, sections, pairs=pairs, out=x)
    assert torch.equal(x, got)
