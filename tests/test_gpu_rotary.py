"""rotary against its definition in 64 bits: types, pairings, ladders, axes, odd
sizes, strides, far and negative positions, in place, its gradient, streams and graphs."""
import math
from fractions import Fraction

import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _inputs(tokens, heads, width, axes, dtype, seed=0, far=5000, pos=torch.int32):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + width)
    x = torch.randn(tokens, heads, width, generator=g, device="cuda").to(dtype)
    p = torch.randint(-far, far, (tokens, axes), generator=g, device="cuda").to(pos)
    return x, p


def _check(got, x, p, sections, pairs="half", inverse=False, **kw):
    axis, freq = ref.ladder64(sections, **kw)
    want, tol = ref.rotary64(x, p, axis, freq, pairs == "interleaved", inverse)
    assert got.dtype == x.dtype
    ref.check(got, want, tol)


@pytest.mark.parametrize("width,sections", [
    (128, (16, 24, 24)), (64, (16, 16)), (80, (10, 15, 15)), (96, (48,)), (72, (12, 12, 12)),
    (128, (8, 8)), (80, (7, 3, 11)), (256, (64, 64)), (2, (1,)), (33, (5, 0, 7)), (700, (100,))])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_widths(pkg, width, sections, pairs, dtype):
    x, p = _inputs(13, 5, width, len(sections), dtype)
    _check(pkg.rotary(x, p, sections, pairs=pairs), x, p, sections, pairs)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 24), (2, 300), (31, 7), (4097, 3), (700, 48)])
@pytest.mark.parametrize("inverse", [False, True])
def test_sizes(pkg, tokens, heads, inverse):
    x, p = _inputs(tokens, heads, 128, 3, BF)
    got = pkg.rotary(x, p, (16, 24, 24), ladder="shared", inverse=inverse)
    _check(got, x, p, (16, 24, 24), inverse=inverse, ladder="shared")


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strides(pkg, pairs, off):
    """Heads in the middle of wider rows, at any alignment; nothing beside them is written."""
    x, p = _inputs(50, 6, 64, 2, BF)
    wide = torch.full((50, 9, 80), 7.0, dtype=BF, device="cuda")
    part = wide[:, 2:8, off:off + 64]
    part.copy_(x)
    _check(pkg.rotary(part, p, (16, 16), pairs=pairs), x, p, (16, 16), pairs)
    rest = torch.full((50, 9, 80), 3.0, dtype=BF, device="cuda")
    pkg.rotary(x, p, (16, 16), pairs=pairs, out=rest[:, 2:8, off:off + 64])
    _check(rest[:, 2:8, off:off + 64], x, p, (16, 16), pairs)
    rest[:, 2:8, off:off + 64] = 3.0
    assert bool((rest == 3.0).all())
    pkg.rotary(part, p, (16, 16), pairs=pairs, out=part)   # in place
    _check(part, x, p, (16, 16), pairs)


def test_heads_before_tokens(pkg):
    x, p = _inputs(40, 6, 64, 1, FF)
    y = x.transpose(0, 1).contiguous().transpose(0, 1)
    got = pkg.rotary(y, p[:, 0].contiguous(), (32,))
    _check(got, x, p, (32,))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_far_positions(pkg, dtype):
    """The whole-number turn against the same product in rational arithmetic."""
    far = [0, 1, -1, 2 ** 31 - 1, -2 ** 31] + ([] if dtype is torch.int32 else [2 ** 40 + 1, -2 ** 45])
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    n = 16
    x = torch.ones(len(far), 1, 2 * n, device="cuda")
    p = torch.tensor(far, dtype=dtype, device="cuda")
    got = pkg.rotary(x, p, (n,), pairs="interleaved").double().cpu()
    for t, pos in enumerate(far):
        for i in range(n):
            f = Fraction(10000.0 ** (-i / n))
            turn = f * pos / (2 * pi)
            a = float((turn - math.floor(turn)) * 2 * pi)
            tol = 2 * (2.0 ** -20 + abs(float(f * pos)) * 2.0 ** -51) + 2.0 ** -22
            assert abs(float(got[t, 0, 2 * i]) - (math.cos(a) - math.sin(a))) <= tol
            assert abs(float(got[t, 0, 2 * i + 1]) - (math.cos(a) + math.sin(a))) <= tol


def test_given_frequencies_and_scales(pkg):
    x, p = _inputs(9, 4, 64, 2, FF)
    axis, freq = ref.ladder64((10, 22), base=500.0, scales=(0.25, 1.5))
    got = pkg.rotary(x, p, (10, 22), base=500.0, scales=(0.25, 1.5))
    _check(got, x, p, (10, 22), base=500.0, scales=(0.25, 1.5))
    assert torch.equal(got, pkg.rotary(x, p, (10, 22), frequencies=freq))
    still = pkg.rotary(x, p, (10, 22), frequencies=[0.0] * 32)
    assert torch.equal(still, x)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_gradient(pkg, pairs):
    """The inverse is the transpose: the formula's gradient, and differences."""
    x, p = _inputs(6, 2, 80, 2, FF)
    w = torch.randn_like(x)
    got = pkg.rotary(w, p, (9, 20), pairs=pairs, inverse=True)
    axis, freq = ref.ladder64((9, 20))
    leaf = x.double().requires_grad_()
    n = 29
    ang = p.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    ia = torch.arange(n, device="cuda") * (2 if pairs == "interleaved" else 1)
    ib = ia + (1 if pairs == "interleaved" else n)
    a, b = leaf[..., ia], leaf[..., ib]
    rest = torch.ones(80, dtype=torch.bool, device="cuda")
    rest[ia] = rest[ib] = False
    loss = ((a * c - b * s) * w[..., ia] + (b * c + a * s) * w[..., ib]).sum() + (
        leaf * w)[..., rest].sum()
    loss.backward()
    _, tol = ref.rotary64(w, p, axis, freq, pairs == "interleaved", True)
    ref.check(got, leaf.grad, tol)
    # one element moved by h moves the loss by h times its gradient (a linear map)
    for e in (0, 17, 58, 79):
        up, down = x.clone(), x.clone()
        up[3, 1, e] += 1.0
        down[3, 1, e] -= 1.0
        d = [(pkg.rotary(v, p, (9, 20), pairs=pairs).double() * w.double())[3, 1].sum() for v in (up, down)]
        slack = 80 * 2.0 ** -19 * float(w[3, 1].abs().max()) * float(up[3, 1].abs().max() + 1)
        assert abs(float(d[0] - d[1]) / 2 - float(got[3, 1, e])) <= slack


def test_nothing_to_do_and_nan(pkg):
    p = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert pkg.rotary(torch.zeros(0, 4, 64, dtype=BF, device="cuda"), p, (4, 4)).shape == (0, 4, 64)
    x, p = _inputs(3, 2, 64, 1, BF)
    x[1, 0, 5] = float("nan")
    y = pkg.rotary(x, p, (16,))
    bad = torch.isnan(y).nonzero().tolist()
    assert bad == [[1, 0, 5], [1, 0, 21]]


def test_stream_and_graph(pkg):
    x, p = _inputs(200, 8, 128, 3, BF)
    want = pkg.rotary(x, p, (16, 24, 24))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.rotary(x, p, (16, 24, 24), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.rotary(x, p, (16, 24, 24), out=out)
    p += 3
    x.mul_(0.5)
    graph.replay()
    _check(out, x, p, (16, 24, 24))


def test_refusals(pkg):
    x, p = _inputs(4, 2, 64, 2, BF)
    for bad in (dict(sections=(40, 10)), dict(sections=()), dict(sections=(0, 0)), dict(sections=(-1, 4)),
                dict(sections=(4,)), dict(sections=(4, 4, 4)), dict(pairs="other"), dict(ladder="other"),
                dict(base=0.0), dict(frequencies=[1.0]), dict(scales=(1.0,)),
                dict(frequencies=[float("inf")] * 8)):
        kw = dict(sections=(4, 4))
        kw.update(bad)
        with pytest.raises((ValueError, TypeError, pkg.ConvError)):
            pkg.rotary(x, p, **kw)
    with pytest.raises(TypeError):
        pkg.rotary(x, p.float(), (4, 4))
    with pytest.raises(TypeError):
        pkg.rotary(x.to(torch.int8), p, (4, 4))
    with pytest.raises(ValueError):
        pkg.rotary(x, p[:3], (4, 4))
    with pytest.raises(ValueError):
        pkg.rotary(x, p, (4, 4), out=torch.empty(4, 2, 32, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        pkg.rotary(x.transpose(1, 2), p, (1, 0))
