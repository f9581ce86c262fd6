"""paged_attention against its definition in 64 bits: cache types, head layouts,
widths, lengths of zero and one to long ones, page sizes, masks, caps, distances,
what lies in unseen places, pages that are not there, strides, streams and graphs."""
import pytest
import torch

import _attention_ref as ref

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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Problem:
    """Caches whose unseen places hold NaN, in shuffled pages; `values` are the seen rows."""

    def __init__(self, lengths, heads, kv, width, cache, dtype, page=16, seed=0, spread=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed + 17 * width + len(lengths))
        self.lengths, self.page = lengths, page
        per = max(1, -(-max(lengths) // page))
        pages = per * len(lengths) + 2
        self.table = torch.randperm(pages, generator=g, device="cuda")[:per * len(lengths)].view(-1, per).to(torch.int32)
        shape = (pages, kv, page, width)
        draw = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
        self.q = (draw(len(lengths), heads, width) * spread).to(dtype)
        codes = cache in (I8, E4)
        self.scales = {}
        self.pools = []
        for name in ("k", "v"):
            if codes:
                if cache == I8:
                    t = torch.randint(-127, 128, shape, generator=g, device="cuda").to(I8)
                    s = 0.02 * (0.2 + torch.rand(*shape[:3], generator=g, device="cuda"))
                else:
                    t = (draw(*shape) * 100).clamp(-448, 448).to(E4)
                    s = 0.01 * (0.2 + torch.rand(*shape[:3], generator=g, device="cuda"))
                self.scales[name + "_scale"] = s
            else:
                t, s = draw(*shape).to(cache), None
            self.pools.append((t, s))
        self.values = []
        for t, s in self.pools:
            full = t.double() if s is None else t.double() * s.double()[..., None]
            self.values.append([
                full[self.table[b].long()].transpose(1, 2).reshape(-1, kv, width)[:n] for b, n in enumerate(lengths)])
            hide = torch.ones(shape[:3], dtype=torch.bool, device="cuda")
            for b, n in enumerate(lengths):
                for j in range(per):
                    left = min(max(n - j * page, 0), page)
                    hide[self.table[b, j].long(), :, :left] = False
            if s is None:
                t[hide] = float("nan")
            else:
                s[hide] = float("nan")
        self.coarse = max(float((t.double().abs() * s.double()[..., None]).nan_to_num().max()) for t, s in self.pools
                          ) if codes else None
        self.weights = BF if cache == BF else HF
        if codes:
            self.coarse = float(self.scales["v_scale"].nan_to_num().max()) * (127 if cache == I8 else 448)

    def run(self, pkg, **kw):
        (k, _), (v, _) = self.pools
        return pkg.paged_attention(self.q, k, v, self.table, _ints(self.lengths), **self.scales, **kw)

    def check(self, got, window=0, prefix=None, **kw):
        for b, n in enumerate(self.lengths):
            want, tol = ref.attention64(
                self.q[b:b + 1], self.values[0][b], self.values[1][b], window=window,
                prefix=0 if prefix is None else prefix[b], weights=self.weights, coarse=self.coarse, **kw)
            ref.check(got[b:b + 1], want, tol)


CACHES = [(I8, BF), (E4, BF), (I8, HF), (E4, HF), (BF, BF), (HF, HF)]


@pytest.mark.parametrize("cache,dtype", CACHES)
@pytest.mark.parametrize("width", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("heads,kv", [(4, 4), (8, 2), (32, 2)])
def test_types_and_heads(pkg, cache, dtype, width, heads, kv):
    p = Problem([1, 0, 15, 16, 17, 300, 129], heads, kv, width, cache, dtype)
    p.check(p.run(pkg))


@pytest.mark.parametrize("heads,kv", [(1, 1), (7, 1), (9, 1), (16, 1), (17, 1), (33, 1), (40, 1), (14, 2), (48, 3)])
@pytest.mark.parametrize("width", [64, 256])
def test_groups(pkg, heads, kv, width):
    p = Problem([257, 40], heads, kv, width, E4, BF)
    p.check(p.run(pkg))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 32, 128, 1000])
@pytest.mark.parametrize("cache", [I8, BF])
def test_page_sizes(pkg, page, cache):
    p = Problem([5, 333, 1000, 128], 8, 2, 64, cache, BF, page=page)
    p.check(p.run(pkg))
    p.check(p.run(pkg, window=100), window=100)


@pytest.mark.parametrize("lengths", [[1], [2], [5000], [20001], [0], [0, 0, 0], [1] * 700,
                                     [(37 * i) % 400 for i in range(333)], [9000, 1, 0, 30, 2500, 1]])
@pytest.mark.parametrize("cache", [E4, HF])
def test_lengths(pkg, lengths, cache):
    p = Problem(lengths, 8, 4, 128, cache, HF)
    got = p.run(pkg)
    p.check(got)
    assert torch.equal(got, p.run(pkg))   # the split and its join do not depend on timing


@pytest.mark.parametrize("window,prefix", [(1, None), (16, None), (100, None), (5000, None), (7, [0, 3, 40, 9000]),
                                           (300, [20, 17, 250, 1]), (0, [3, 3, 3, 3])])
@pytest.mark.parametrize("cache", [I8, BF])
def test_masks(pkg, window, prefix, cache):
    p = Problem([3, 500, 1111, 0], 6, 3, 64, cache, BF)
    kw = dict(window=window, prefix=None if prefix is None else _ints(prefix))
    p.check(p.run(pkg, **kw), window=window, prefix=prefix)


@pytest.mark.parametrize("cap", [0.5, 30.0])
@pytest.mark.parametrize("sloped", [False, True])
@pytest.mark.parametrize("cache,dtype", CACHES)
def test_caps_and_distances(pkg, cap, sloped, cache, dtype):
    p = Problem([77, 900], 12, 2, 80, cache, dtype, spread=3.0)
    slopes = torch.linspace(0.001, 0.5, 12, device="cuda") if sloped else None
    p.check(p.run(pkg, cap=cap, slopes=slopes, scale=0.2), cap=cap, slopes=slopes, scale=0.2)


def test_large_scores(pkg):
    """Exponents far beyond fp32's, and one that outweighs all others."""
    p = Problem([600, 50], 8, 2, 64, HF, HF, spread=200.0)
    p.check(p.run(pkg, scale=1.0), scale=1.0)


def test_scales_of_all_sizes(pkg):
    """Values' scales over 60 powers of two, in rows of zeros and next to the largest."""
    p = Problem([700, 90], 8, 2, 64, I8, BF)
    s = p.scales["v_scale"]
    e = torch.randint(-30, 31, s.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    s.mul_(torch.ldexp(torch.ones_like(s), e))
    p.values[1] = [(p.pools[1][0].double() * s.double()[..., None])[p.table[b].long()].transpose(1, 2)
                   .reshape(-1, 2, 64)[:n] for b, n in enumerate(p.lengths)]
    p.coarse = float(s.nan_to_num().max()) * 127
    p.check(p.run(pkg))
    s.fill_(0.0)   # values that count as zeros
    assert not p.run(pkg).any()


def test_queries_of_all_sizes(pkg):
    """bf16 queries beyond fp16's range, and tiny ones, over 8-bit keys."""
    for size in (1e30, 1e-30, 3e5):
        p = Problem([200], 8, 2, 64, E4, BF, spread=size)
        p.check(p.run(pkg, scale=0.1 / size), scale=0.1 / size)
    p.q.zero_()
    p.check(p.run(pkg))


def test_pages_that_are_not_there(pkg):
    """A missing page spoils the sequences that see it, and no others; a length past the
    table spoils its sequence; unseen pages may be anything."""
    for cache in (E4, BF):
        p = Problem([100, 100, 100, 100, 100], 4, 2, 64, cache, BF)
        p.table[1, 3], p.table[2, 0], p.table[3, 0] = -1, 2 ** 31 - 1, -5
        got = p.run(pkg)
        assert bool(torch.isnan(got[1:4]).all()) and bool(torch.isfinite(got[0]).all() & torch.isfinite(got[4]).all())
        got = p.run(pkg, window=60)
        assert bool(torch.isnan(got[1]).all()) and bool(torch.isfinite(got[[0, 2, 3, 4]]).all())
        p.table[1:4] = p.table[0]
        p.lengths = [100, 113, 2 ** 31 - 1, 10 ** 6, -7]
        got = p.run(pkg)
        assert bool(torch.isfinite(got[0]).all()) and bool(torch.isnan(got[1:4]).all()) and not got[4].any()


def test_nan_and_inf_where_they_are_seen(pkg):
    for cache in (E4, HF):
        p = Problem([60, 60, 60], 4, 2, 64, cache, HF)
        p.q[1, 2, 5] = float("nan")
        got = p.run(pkg)
        assert bool(torch.isnan(got[1, 2]).all()) and not torch.isnan(got[1, [0, 1, 3]]).any()
        assert not torch.isnan(got[[0, 2]]).any()
    s = Problem([60, 60], 4, 2, 64, I8, HF)
    s.scales["k_scale"][s.table[0, 1].long(), 1, 3] = float("nan")   # key head 1: query heads 2, 3
    got = s.run(pkg)
    assert bool(torch.isnan(got[0, 2:]).all()) and not torch.isnan(got[0, :2]).any() and not torch.isnan(got[1]).any()


def test_strides_and_given_buffers(pkg):
    p = Problem([130, 1, 77], 6, 2, 64, I8, BF)
    want = p.run(pkg)
    wide = torch.zeros(3, 11, 72, dtype=BF, device="cuda")
    wide[:, 2:8, 1:65] = p.q
    p.q = wide[:, 2:8, 1:65]
    out = torch.full((3, 11, 72), 5.0, dtype=BF, device="cuda")
    table = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    table[:, 4:4 + p.table.shape[1]] = p.table
    p.table = table[:, 4:4 + p.table.shape[1]]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    got = p.run(pkg, out=out[:, 2:8, 3:67], workspace=ws)
    assert torch.equal(got, want)
    out[:, 2:8, 3:67] = 5.0
    assert bool((out == 5.0).all())


def test_cache_of_other_strides(pkg):
    """Keys and values of a page side by side, heads behind tokens."""
    p = Problem([200, 45], 4, 2, 64, E4, BF)
    want = p.run(pkg)
    (k, ks), (v, vs) = p.pools
    both = torch.empty(k.shape[0], 16, 2, 2, 64, dtype=torch.uint8, device="cuda").view(E4)
    both.view(torch.uint8)[:, :, 0] = k.view(torch.uint8).transpose(1, 2)
    both.view(torch.uint8)[:, :, 1] = v.view(torch.uint8).transpose(1, 2)
    size = torch.stack([ks, vs], 1)
    got = pkg.paged_attention(p.q, both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2), p.table,
                              _ints(p.lengths), k_scale=size[:, 0], v_scale=size[:, 1])
    assert torch.equal(got, want)


def test_far_pages(pkg):
    """Rows past 2^31 bytes."""
    pages = 30000
    k = torch.zeros(pages, 2, 128, 512 // 2, dtype=HF, device="cuda")   # 3.9 GB
    v = torch.zeros_like(k)
    table = _ints([[pages - 1, 7, pages - 2]])
    for t in (pages - 1, 7, pages - 2):
        k[t], v[t] = torch.randn(2, 128, 256, device="cuda").to(HF), torch.randn(2, 128, 256, device="cuda").to(HF)
    q = torch.randn(1, 4, 256, device="cuda").to(HF)
    got = pkg.paged_attention(q, k, v, table, _ints([300]))
    at = table[0].long()
    kk, vv = (t[at].transpose(1, 2).reshape(-1, 2, 256)[:300] for t in (k, v))
    want, tol = ref.attention64(q, kk, vv, weights=HF)
    ref.check(got, want, tol)


def test_streams_and_graphs(pkg):
    """Two captured graphs with workspaces of their own, replayed at once; new lengths
    and pages between replays."""
    ps = [Problem([300, 700, 1], 8, 2, 128, E4, BF, seed=s) for s in (1, 2)]
    lens = [_ints(p.lengths) for p in ps]
    graphs, outs = [], []
    for p, n in zip(ps, lens):
        (k, _), (v, _) = p.pools
        run = lambda: pkg.paged_attention(p.q, k, v, p.table, n, **p.scales)   # noqa: E731
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    for lengths in ([300, 700, 1], [1, 699, 0], [17, 0, 1]):
        for n in lens:
            n.copy_(_ints(lengths))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for p, o in zip(ps, outs):
            vals = p.values
            p.lengths, p.values = lengths, [[t[:n] for t, n in zip(x, lengths)] for x in vals]
            p.check(o)
            p.values = vals
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = Problem([999], 8, 2, 64, I8, BF)
    side.wait_stream(torch.cuda.current_stream())
    got = p.run(pkg, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    p.check(got)


def test_refusals(pkg):
    p = Problem([10, 20], 4, 2, 64, I8, BF)
    (k, ks), (v, vs) = p.pools
    good = dict(q=p.q, k_cache=k, v_cache=v, page_table=p.table, lengths=_ints([10, 20]), k_scale=ks, v_scale=vs)
    pkg.paged_attention(**good)
    for bad in (dict(q=p.q.float()), dict(q=p.q[:, :3]), dict(q=p.q[:1]), dict(q=p.q[..., :32]), dict(k_scale=None),
                dict(lengths=_ints([1])), dict(lengths=torch.tensor([1, 2], device="cuda")), dict(cap=-1.0),
                dict(cap=float("nan")), dict(window=-1), dict(scale=float("inf")), dict(prefix=_ints([1])),
                dict(slopes=torch.ones(3, device="cuda")), dict(slopes=torch.ones(4, dtype=HF, device="cuda")),
                dict(out=torch.empty(2, 4, 64, dtype=HF, device="cuda")),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[1:]),
                dict(page_table=p.table[:1]), dict(q=p.q.cpu())):
        with pytest.raises((ValueError, TypeError, pkg.ConvError)):
            pkg.paged_attention(**{**good, **bad})
    e = pkg.paged_attention(p.q[:0], k, v, p.table[:0], _ints([]), k_scale=ks, v_scale=vs)
    assert e.shape == (0, 4, 64)
