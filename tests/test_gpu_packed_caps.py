"""packed_attention under caps of all sizes that it accepts, in tiles that are seen
whole and in part, next to rows and keys that would ask for another form of the cap, and
beside paged_attention of the same tokens."""
import pytest
import torch

import _attention_ref as ref
from _capped_ref import capped64

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


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


def _rows(n, heads, kv, width, dtype, spread=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n + width)
    draw = lambda h: torch.randn(n, h, width, generator=g, device="cuda")   # noqa: E731
    return (draw(heads) * spread).to(dtype), draw(kv).to(dtype), draw(kv).to(dtype)


def _check(got, q, k, v, cap, rows=None, **kw):
    want, tol = capped64(q, k, v, cap, q.dtype, **kw)
    rows = slice(None) if rows is None else rows
    ref.check(got[rows], want[rows], tol[rows])


CAPS = [1e-20, 1e-6, 0.5, 3.0, 50.0, 1e3, 1e6, 1e9, 1e30, 3.4e38]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [False, True])
def test_caps(pkg, cap, dtype, causal):
    for lens, heads, width in (([300, 99], 4, 64), ([1300, 700], 40, 128)):   # one query tile a job, two
        q, k, v = _rows(sum(lens), heads, 2, width, dtype, 3.0)
        off = _ints([0, lens[0], sum(lens)])
        got = pkg.packed_attention(q, k, v, off, causal=causal, cap=cap)
        a = 0
        for n in lens:
            for h in (0, heads - 1):
                g = h // (heads // 2)
                _check(got[a:a + n, h:h + 1], q[a:a + n, h:h + 1], k[a:a + n, g:g + 1], v[a:a + n, g:g + 1], cap,
                       causal=causal)
            a += n


@pytest.mark.parametrize("cap", [1e-6, 1e-20, 3.4e38])
@pytest.mark.parametrize("scale", [0.125, 1e30])
def test_zero_queries(pkg, cap, scale):
    """Scores of 0 stay 0 under any cap: the mean of the values."""
    q, k, v = _rows(300, 2, 2, 64, BF, 0.0)
    got = pkg.packed_attention(q, k, v, _ints([0, 300]), cap=cap, scale=scale)
    _check(got, q, k, v, cap, causal=False)


@pytest.mark.parametrize("cap", [20.0, 1e4, 3e5])
def test_scores_about_the_cap(pkg, cap):
    """Rows whose scores lie below, next to and above the cap, side by side."""
    q, k, v = _rows(400, 2, 1, 64, HF)
    q.mul_(torch.tensor([0.2, 0.5, 1.0, 3.0, 0.1, 0.6, 2.0, 4.0], device="cuda").repeat(50)[:, None, None])
    for causal in (False, True):
        got = pkg.packed_attention(q, k, v, _ints([0, 400]), causal=causal, cap=cap, scale=cap / 12)
        _check(got, q, k, v, cap, causal=causal, scale=cap / 12)


@pytest.mark.parametrize("cap", [1e6, 1e8])
@pytest.mark.parametrize("what", ["query", "key"])
def test_beside_large_scores(pkg, cap, what):
    """A row, or a later key, whose scores are above the cap leaves the others as they are."""
    n, at = 384, 200
    q, k, v = _rows(n, 2, 2, 64, BF, 3.0)
    (q if what == "query" else k)[at] *= cap
    got = pkg.packed_attention(q, k, v, _ints([0, n]), causal=True, cap=cap)
    if what == "query":
        rest = torch.arange(n, device="cuda") != at
        _check(got, q, k, v, cap, rows=rest)
    else:
        _check(got[:at], q[:at], k[:at], v[:at], cap)


@pytest.mark.parametrize("cap", [30.0, 1e5, 1e7])
def test_rows_that_are_computed_again(pkg, cap):
    """Rows next to values that are not finite, which they do not see."""
    q, k, v = _rows(300, 2, 2, 64, HF, 3.0)
    v[250] = float("nan")
    got = pkg.packed_attention(q, k, v, _ints([0, 300]), causal=True, cap=cap)
    _check(got[:250], q[:250], k[:250], v[:250], cap)


@pytest.mark.parametrize("cap", [30.0, 1e6, 1e9])
def test_the_token_path_agrees(pkg, cap):
    """The last query of a document, and the same token over a cache."""
    n, heads, kv, width, page = 500, 8, 2, 64, 20
    q, k, v = _rows(n, heads, kv, width, BF, 3.0)
    pools = [t.view(n // page, page, kv, width).transpose(1, 2).contiguous() for t in (k, v)]
    table = torch.arange(n // page, device="cuda").int()[None]
    one = pkg.paged_attention(q[-1:], *pools, table, _ints([n]), cap=cap)
    all_ = pkg.packed_attention(q, k, v, _ints([0, n]), causal=True, cap=cap)
    want, tol = capped64(q[-1:], k, v, cap, BF)
    ref.check(one, want, tol)
    ref.check(all_[-1:], want, tol)
