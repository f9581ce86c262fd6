"""paged_attention under caps of all sizes that it accepts: a cap far above the scores
changes nothing, one far below them takes their sign, and scores in between keep their
relative accuracy."""
import pytest
import torch

import _attention_ref as ref
from _capped_ref import capped64

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _problem(lengths, heads, kv, width, cache, dtype, spread, page=16):
    g = torch.Generator(device="cuda").manual_seed(width + len(lengths))
    per = -(-max(lengths) // page)
    table = torch.randperm(per * len(lengths), generator=g, device="cuda").view(len(lengths), per).int()
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    q = (draw(len(lengths), heads, width) * spread).to(dtype)
    shape = (per * len(lengths), kv, page, width)
    pools, scales, held, coarse = [], {}, [], None
    for name in ("k", "v"):
        if cache in (I8, E4):
            t = (draw(*shape) * 40).clamp(-127, 127).to(cache)
            s = 0.025 * (0.2 + torch.rand(*shape[:3], generator=g, device="cuda"))
            scales[name + "_scale"] = s
            full = t.double() * s.double()[..., None]
            coarse = float(s.max()) * 127
        else:
            t = draw(*shape).to(cache)
            full = t.double()
        pools.append(t)
        held.append([full[table[b].long()].transpose(1, 2).reshape(-1, kv, width)[:n] for b, n in enumerate(lengths)])
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return q, held, coarse, lambda pkg, **kw: pkg.paged_attention(q, *pools, table, n, **scales, **kw)


CAPS = [1e-20, 1e-6, 0.5, 3.0, 30.0, 1e3, 1e6, 1e9, 1e30, 3.4e38]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("cache,dtype", [(I8, BF), (E4, HF), (BF, BF), (HF, HF)])
@pytest.mark.parametrize("width,heads", [(64, 4), (128, 24)])
def test_caps(pkg, cap, cache, dtype, width, heads):
    lengths = [700, 90, 17, 1]
    q, held, coarse, run = _problem(lengths, heads, 2, width, cache, dtype, 3.0)
    got = run(pkg, cap=cap)
    for b in range(len(lengths)):
        want, tol = capped64(q[b:b + 1], held[0][b], held[1][b], cap, BF if cache is BF else HF, coarse=coarse)
        ref.check(got[b:b + 1], want, tol)


@pytest.mark.parametrize("cap", [20.0, 1e4])
def test_scores_about_the_cap(pkg, cap):
    """Rows whose scores lie below, next to and above the cap, side by side."""
    lengths = [300, 300, 300]
    q, held, _, run = _problem(lengths, 8, 2, 64, HF, HF, 1.0)
    q.mul_(torch.tensor([0.2, 0.5, 1.0, 3.0, 0.1, 0.6, 2.0, 4.0], device="cuda")[None, :, None])
    scale = cap / 12
    got = run(pkg, cap=cap, scale=scale)
    for b in range(len(lengths)):
        want, tol = capped64(q[b:b + 1], held[0][b], held[1][b], cap, HF, scale=scale)
        ref.check(got[b:b + 1], want, tol)


def test_zero_queries(pkg):
    """Scores of 0 stay 0 under any cap: the mean of the values."""
    q, held, _, run = _problem([100, 33], 4, 2, 64, BF, BF, 0.0)
    for cap in (1e-20, 1e-3, 50.0, 3.4e38):
        for scale in (0.125, 1e30):
            got = run(pkg, cap=cap, scale=scale)
            for b in range(2):
                want, tol = capped64(q[b:b + 1], held[0][b], held[1][b], cap, BF)
                ref.check(got[b:b + 1], want, tol)
