"""packed_attention against its definition in 64 bits: document lengths from none and
one to long ones, both forms of the kernel, widths, head layouts, masks, caps,
distances, what lies in unseen places, rows in no document, strides, graphs."""
import pytest
import torch

import _attention_ref as ref

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


def _offsets(lens):
    return _ints([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist())


class Problem:
    def __init__(self, nq, heads, kv, width, dtype, nk=None, seed=0, spread=1.0, behind=5):
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * width + sum(nq))
        self.nq, self.nk = nq, nq if nk is None else nk
        draw = lambda n, h: torch.randn(n, h, width, generator=g, device="cuda")   # noqa: E731
        # rows behind the last document hold anything
        self.q = (draw(sum(nq) + behind, heads) * spread).to(dtype)
        self.k, self.v = (draw(sum(self.nk) + behind, kv).to(dtype) for _ in range(2))
        for t, n in ((self.q, nq), (self.k, self.nk), (self.v, self.nk)):
            t[sum(n):] = float("nan")

    def run(self, pkg, **kw):
        ko = None if self.nk is self.nq else _offsets(self.nk)
        if ko is None and self.q.shape[0] != self.k.shape[0]:
            ko = _offsets(self.nk)
        kw.setdefault("out", torch.full_like(self.q, 7.0))
        return pkg.packed_attention(self.q, self.k, self.v, _offsets(self.nq), ko, **kw)

    def check(self, got, prefix=None, **kw):
        a = b = 0
        for s, (n, m) in enumerate(zip(self.nq, self.nk)):
            want, tol = ref.attention64(self.q[a:a + n], self.k[b:b + m], self.v[b:b + m],
                                        prefix=0 if prefix is None else prefix[s], weights=self.q.dtype, **kw)
            ref.check(got[a:a + n], want, tol)
            a, b = a + n, b + m
        assert bool((got[a:] == 7.0).all())   # rows in no document are left


# one tile a CTA, and two (documents of 1024 and more, with CTAs for all SMs)
SHORT, LONG = [256, 1, 0, 127, 128, 129, 300, 77], [5000, 1700, 1]


@pytest.mark.parametrize("width", [8, 16, 64, 72, 80, 96, 120, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [False, True])
def test_widths(pkg, width, dtype, causal):
    p = Problem(SHORT, 4, 2, width, dtype)
    p.check(p.run(pkg, causal=causal), causal=causal)


@pytest.mark.parametrize("width", [40, 64, 80, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [False, True])
def test_long_documents(pkg, width, dtype, causal):
    p = Problem(LONG, 8, 4, width, dtype)
    p.check(p.run(pkg, causal=causal), causal=causal)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (12, 4), (40, 8)])
def test_heads(pkg, heads, kv):
    p = Problem([200, 31], heads, kv, 64, BF)
    p.check(p.run(pkg, causal=True), causal=True)


@pytest.mark.parametrize("lens", [[1], [2], [0], [0, 0, 5], [1] * 300, [(31 * i) % 150 for i in range(140)],
                                  [0] * 200 + [130] + [0] * 70 + [3]])
def test_lengths(pkg, lens):
    p = Problem(lens, 3, 3, 64, HF)
    p.check(p.run(pkg), causal=False)


MASKS = [dict(causal=True, window=1), dict(causal=False, window=1), dict(causal=True, window=100),
         dict(causal=False, window=100), dict(causal=True, window=513), dict(causal=True, prefix=True),
         dict(causal=False, window=60, prefix=True), dict(causal=True, window=33, prefix=True),
         dict(causal=True, window=10 ** 9)]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("long", [False, True])
def test_masks(pkg, mask, long):
    lens = [3000, 1500] if long else SHORT
    mask = dict(mask)
    prefix = [(97 * i * i) % 700 for i in range(len(lens))] if mask.pop("prefix", False) else None
    p = Problem(lens, 16 if long else 2, 2, 64, BF)
    kw = dict(mask, prefix=None if prefix is None else _ints(prefix))
    p.check(p.run(pkg, **kw), prefix=prefix, **mask)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("long", [False, True])
def test_queries_are_the_last_tokens(pkg, causal, window, long):
    """More keys than queries (a chunk after a cache), fewer, none."""
    nq, nk = ([2000, 1300, 1100], [2600, 1300, 700]) if long else ([100, 1, 60, 300, 5, 0, 260], [400, 333, 0, 130, 5, 9, 100])
    p = Problem(nq, 16 if long else 4, 4, 80, HF, nk=nk)
    p.check(p.run(pkg, causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("cap", [0.0, 0.7, 50.0])
@pytest.mark.parametrize("sloped", [False, True])
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_caps_and_distances(pkg, cap, sloped, long, dtype):
    p = Problem([2100, 1400] if long else [260, 99], 16, 4, 64, dtype, spread=3.0)
    slopes = torch.linspace(0.0001, 0.3, 16, device="cuda") if sloped else None
    for causal in (False, True):
        got = p.run(pkg, causal=causal, cap=cap, slopes=slopes, scale=0.2)
        p.check(got, causal=causal, cap=cap, slopes=slopes, scale=0.2)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_scales(pkg, scale):
    p = Problem([300, 10], 2, 1, 64, BF, spread=4.0)
    p.check(p.run(pkg, scale=scale), causal=False, scale=scale)


def test_rising_scores(pkg):
    """Each tile of keys outweighs the ones before by far: O is rescaled at each."""
    for lens, heads in (([1500], 2), ([2600, 1100], 16)):
        p = Problem(lens, heads, 1, 64, HF)
        p.q.copy_(p.q.abs())
        ramp = torch.arange(p.k.shape[0], device="cuda").float() / 128
        p.k.copy_((p.k.float().abs() * (1 + ramp[:, None, None])).nan_to_num().to(HF))
        p.check(p.run(pkg, scale=0.3), causal=False, scale=0.3)


def test_values_that_are_not_finite_where_unseen(pkg):
    """NaN and infinities in other documents, behind the last key, in later tokens and
    outside the window reach no row that does not see them."""
    for lens, heads in (([200, 90, 300], 2), ([1500, 1200, 1800], 16)):
        for bad in (float("nan"), float("inf")):
            p = Problem(lens, heads, 2, 64, BF)
            first = lens[0]
            p.k[:first], p.v[:first] = bad, bad                     # a whole document
            last = sum(lens) - 1
            p.v[last], p.k[last] = bad, bad                         # its last token
            for kw in (dict(causal=True), dict(causal=True, window=40)):
                got = p.run(pkg, **kw)
                assert not torch.isfinite(got[:first]).any()
                a = first
                for n, cut in ((lens[1], lens[1]), (lens[2], lens[2] - 1)):
                    want, tol = ref.attention64(p.q[a:a + cut], p.k[a:a + cut], p.v[a:a + cut],
                                                weights=BF, **kw)
                    ref.check(got[a:a + cut], want, tol)
                    a += n
                assert not torch.isfinite(got[last]).any()


def test_seen_nan_spoils_its_rows_only(pkg):
    p = Problem([140, 150], 4, 2, 64, HF)
    p.v[150, 1, 7] = float("nan")     # document 1, token 10, key head 1
    p.q[3, 0, 0] = float("nan")
    got = p.run(pkg, causal=True)
    bad = torch.isnan(got[:290])
    want = torch.zeros_like(bad)
    want[150:, 2:, 7] = True
    want[3, 0, :] = True
    assert torch.equal(bad, want)


def test_strides(pkg):
    """Parts of one projection's rows, an output at any alignment."""
    p = Problem([200, 77], 4, 2, 64, BF, behind=0)
    want = p.run(pkg)
    rows = torch.zeros(277, 10, 72, dtype=BF, device="cuda")
    q, k, v = rows[:, 1:5, :64], rows[:, 5:7, :64], rows[:, 7:9, :64]
    q.copy_(p.q), k.copy_(p.k), v.copy_(p.v)
    out = torch.full((277, 6, 67), 7.0, dtype=BF, device="cuda")
    got = pkg.packed_attention(q, k, v, _offsets([200, 77]), out=out[:, 1:5, 3:67])
    assert torch.equal(got, want)
    out[:, 1:5, 3:67] = 7.0
    assert bool((out == 7.0).all())
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (p.q, p.k, p.v)]
    assert torch.equal(pkg.packed_attention(*heads_first, _offsets([200, 77])), want)
    assert torch.equal(pkg.packed_attention(p.q, p.k, p.v, _offsets([200, 77])), want)   # deterministic


def test_far_rows(pkg):
    """Packed rows past 2^31 elements."""
    n = 2 ** 31 // (32 * 128) + 300
    big = torch.zeros(n, 32, 128, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    big[-260:] = torch.randn(260, 32, 128, generator=g, device="cuda").to(BF)
    off = _ints([0, 0, n - 260, n])[1:]
    out = torch.zeros_like(big)
    pkg.packed_attention(big, big, big, _ints([n - 260, n]), out=out)
    want, tol = ref.attention64(big[-260:], big[-260:], big[-260:], causal=False, weights=BF)
    ref.check(out[-260:], want, tol)
    assert off.numel() == 3 and not out[:-260].any()


def test_stream_and_graph(pkg):
    p = Problem([300, 20, 260], 4, 2, 64, BF, behind=100)
    p.q.nan_to_num_(), p.k.nan_to_num_(), p.v.nan_to_num_()
    off = _offsets([300, 20, 260])
    out = torch.full_like(p.q, 7.0)
    graph = torch.cuda.CUDAGraph()
    pkg.packed_attention(p.q, p.k, p.v, off, causal=True, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkg.packed_attention(p.q, p.k, p.v, off, causal=True, out=out)
    for lens in ([300, 20, 260], [1, 600, 0], [0, 0, 0]):
        off.copy_(_offsets(lens))
        out.fill_(7.0)
        graph.replay()
        p.nq = p.nk = lens
        p.check(out, causal=True)
    side = torch.cuda.Stream()
    p.nq = p.nk = [300, 20, 260]
    p.out = torch.full_like(p.q, 7.0)
    torch.cuda.synchronize()
    got = p.run(pkg, stream=side, out=p.out)
    side.synchronize()
    p.check(got, causal=False)


def test_refusals(pkg):
    p = Problem([10, 20], 4, 2, 64, BF, behind=0)
    off = _offsets([10, 20])
    good = dict(q=p.q, k=p.k, v=p.v, q_offsets=off)
    pkg.packed_attention(**good)
    wide = torch.zeros(30, 4, 136, dtype=BF, device="cuda")
    flat = torch.zeros(30 * 4 * 64 + 1, dtype=BF, device="cuda")[1:].view(30, 4, 64)
    for bad in (dict(q=p.q.float()), dict(k=p.k.to(HF), v=p.v.to(HF)), dict(v=p.v[:, :1]), dict(k=p.k[..., :32], v=p.v[..., :32]),
                dict(q=p.q[:, :3]), dict(q=p.q[:20]), dict(q=wide, k=wide, v=wide), dict(q=p.q[..., :20], k=p.k[..., :20], v=p.v[..., :20]),
                dict(q=flat), dict(q_offsets=off.long()), dict(q_offsets=off.cpu()), dict(k_offsets=off[:2]),
                dict(prefix=_ints([1])), dict(slopes=torch.ones(2, device="cuda")), dict(cap=-1.0), dict(window=-1),
                dict(scale=float("nan")), dict(out=torch.empty(30, 4, 64, device="cuda")), dict(q=p.q.cpu())):
        with pytest.raises((ValueError, TypeError, pkg.ConvError)):
            pkg.packed_attention(**{**good, **bad})
    none = pkg.packed_attention(p.q[:0], p.k, p.v, _ints([0]), _ints([0]))
    assert none.shape == (0, 4, 64)
    alone = pkg.packed_attention(p.q, p.k[:0], p.v[:0], off, _ints([0, 0, 0]))
    assert not alone.any()
