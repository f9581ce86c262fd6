"""kv_cache_write and kv_cache_read against their definitions: types, widths, page
sizes, ragged sequences, padding, pages that are not there, rows behind the last
sequence, strides, streams and graphs."""
import pytest
import torch

import _token_ref as tref

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
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


def _raw(t):
    return t.view(torch.uint8) if t.dtype == E4 else t


class Cache:
    """A pool with marked contents, and each sequence's pages in shuffled order."""

    def __init__(self, seqs, per, heads, page, width, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        pages = seqs * per + 2
        self.k, self.v = (torch.full((pages, heads, page, width), 7, device="cuda").to(dtype) for _ in range(2))
        q = dtype in (I8, E4)
        self.ks, self.vs = (torch.full((pages, heads, page), 0.5, device="cuda") if q else None for _ in range(2))
        self.table = torch.randperm(pages, generator=g, device="cuda")[:seqs * per].view(seqs, per).to(torch.int32)
        self.page, self.scales = page, dict(k_scale=self.ks, v_scale=self.vs)

    def at(self, s, pos):
        return int(self.table[s, pos // self.page]), pos % self.page

    def places(self, starts, counts):
        rows = [self.at(s, a + i) for s, (a, n) in enumerate(zip(starts, counts)) for i in range(n)]
        pages, offs = zip(*rows) if rows else ((), ())
        return torch.tensor(pages, dtype=torch.long, device="cuda"), torch.tensor(offs, dtype=torch.long, device="cuda")


def _rows(tokens, heads, width, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(tokens, heads, width, generator=g, device="cuda") for _ in range(2))
    if tokens > 2:
        k[1], v[2] = 0.0, 0.0
        k[2, 0, 3] = float("inf")
    return k.to(dtype), (v * 1e-3).to(dtype)


def _check_written(c, rows, codes, scale, pages, offs):
    got, size = codes[pages, :, offs], None if scale is None else scale[pages, :, offs]
    if size is None:
        assert torch.equal(got, rows)
        return
    bad = ~torch.isfinite(rows.float()).all(-1)
    assert bool(torch.isnan(size[bad]).all()) and not _raw(got)[bad].any()
    ok = ~bad
    tref.check_quant(rows[ok].double(), got[ok], size[ok], 2.0 ** -23)


@pytest.mark.parametrize("width", [16, 48, 64, 80, 128, 176, 256])
@pytest.mark.parametrize("dtype,rows", [(I8, BF), (E4, BF), (E4, HF), (I8, FF), (BF, BF), (HF, HF)])
@pytest.mark.parametrize("page", [16, 40, 1])
def test_write_then_read(pkg, width, dtype, rows, page):
    starts, counts = [0, 3, 30, 17], [5, 0, 41, 1]
    c = Cache(4, -(-80 // page), 3, page, width, dtype, seed=width)
    n = sum(counts)
    k, v = _rows(n, 3, width, rows, width)
    before = [None if t is None else _raw(t).clone() for t in (c.k, c.v, c.ks, c.vs)]
    off = torch.tensor([0] + counts).cumsum(0).tolist()
    pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints(starts), offsets=_ints(off), **c.scales)
    pages, offs = c.places(starts, counts)
    _check_written(c, k, c.k, c.ks, pages, offs)
    _check_written(c, v, c.v, c.vs, pages, offs)
    # nothing else was touched
    for now, was in zip((c.k, c.v, c.ks, c.vs), before):
        if now is not None:
            a = _raw(now).clone()
            a[pages, :, offs] = was[pages, :, offs]
            assert torch.equal(a, was)
    # and back, each sequence from its first new token, and with a row behind the last
    for out in (BF, FF, HF):
        ko, vo = (torch.full((n + 3, 3, width), 9.0, dtype=out, device="cuda") for _ in range(2))
        pkg.kv_cache_read(c.k, c.v, c.table, _ints(off), starts=_ints(starts), k_out=ko, v_out=vo, **c.scales)
        for got, codes, scale in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
            want = codes[pages, :, offs].double()
            if scale is not None:
                want = want * scale[pages, :, offs].double()[..., None]
            assert bool((got[n:] == 9.0).all())
            got = got[:n]
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan)
            fine = torch.isfinite(want)   # an infinity of an unquantised cache stays one
            assert torch.equal(got.double()[~fine & ~nan], want[~fine & ~nan])
            tref.check_rounded(got[fine], want[fine], 2.0 ** -24 * want[fine].abs())


@pytest.mark.parametrize("dtype", [I8, E4, BF])
@pytest.mark.parametrize("seqs", [1, 5, 300])
def test_one_token_each(pkg, dtype, seqs):
    """A decoding step: no offsets; sequences that are not running are negative."""
    c = Cache(seqs, 4, 2, 16, 128, dtype)
    k, v = _rows(seqs, 2, 128, BF, seqs)
    starts = [(7 * s) % 64 for s in range(seqs)]
    if seqs > 3:
        starts[3] = -1
        starts[4] = 64   # past the table
    pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints(starts), **c.scales)
    live = [s for s in range(seqs) if 0 <= starts[s] < 64]
    at = [c.at(s, starts[s]) for s in live]
    pages, offs = (torch.tensor(t, device="cuda") for t in zip(*at))
    _check_written(c, k[live], c.k, c.ks, pages, offs)
    _check_written(c, v[live], c.v, c.vs, pages, offs)
    written = _raw(c.k).clone()
    written[pages, :, offs] = _raw(torch.full((1,), 7, device="cuda").to(dtype))[0]
    assert bool((written == _raw(torch.full((1,), 7, device="cuda").to(dtype))[0]).all())


@pytest.mark.parametrize("dtype", [I8, HF])
def test_pages_that_are_not_there(pkg, dtype):
    """A page outside the pool is neither written nor read: its tokens read as NaN."""
    c = Cache(2, 3, 2, 16, 64, dtype)
    was_k = c.k.clone()
    c.table[0, 1], c.table[1, 0], c.table[1, 2] = -1, c.k.shape[0], 2 ** 31 - 1
    k, v = _rows(96, 2, 64, HF, 1)
    k, v = k.nan_to_num(posinf=2.0), v
    pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints([0, 0]), offsets=_ints([0, 48, 96]), **c.scales)
    ko, vo = pkg.kv_cache_read(c.k, c.v, c.table, _ints([0, 60, 120]), tokens=120, dtype=FF, **c.scales)
    gone = torch.zeros(120, dtype=torch.bool, device="cuda")
    gone[16:32] = gone[48:76] = gone[92:] = True   # 48..59 and 108..119: past the table
    for t in (ko, vo):
        assert torch.equal(torch.isnan(t).all(-1).all(-1), gone)
        assert torch.equal(torch.isnan(t).any(-1).any(-1), gone)
    held = {int(c.table[0, 0]), int(c.table[0, 2]), int(c.table[1, 1])}
    for page in range(c.k.shape[0]):
        assert torch.equal(c.k[page], was_k[page]) == (page not in held)


def test_strides_and_alignment(pkg):
    """Rows inside a projection's, at any alignment, and a cache that keeps keys and
    values of a page side by side."""
    for off in (0, 1):
        c = Cache(2, 2, 2, 16, 64, I8)
        pool = torch.zeros(6, 2, 2, 16, 64, dtype=I8, device="cuda")
        scale = torch.zeros(6, 2, 2, 16, device="cuda")
        k, v = _rows(20, 2, 64, BF, 3)
        k = k.nan_to_num(posinf=1.0)
        wide = torch.zeros(20, 5, 66, dtype=BF, device="cuda")
        kk, vv = wide[:, :2, off:off + 64], wide[:, 2:4, off:off + 64]
        kk.copy_(k), vv.copy_(v)
        args = dict(k_scale=scale[:, 0], v_scale=scale[:, 1])
        pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints([3, 0]), offsets=_ints([0, 9, 20]), **c.scales)
        pkg.kv_cache_write(kk, vv, pool[:, 0], pool[:, 1], c.table, _ints([3, 0]), offsets=_ints([0, 9, 20]), **args)
        pages, offs = c.places([3, 0], [9, 11])
        for a, b in ((c.k, pool[:, 0]), (c.v, pool[:, 1]), (c.ks, scale[:, 0]), (c.vs, scale[:, 1])):
            assert torch.equal(a[pages, :, offs], b[pages, :, offs])
        out = torch.zeros(20, 5, 66, dtype=BF, device="cuda")
        pkg.kv_cache_read(pool[:, 0], pool[:, 1], c.table, _ints([0, 9, 20]), starts=_ints([3, 0]),
                          k_out=out[:, :2, off:off + 64], v_out=out[:, 2:4, off:off + 64], **args)
        ko, vo = pkg.kv_cache_read(c.k, c.v, c.table, _ints([0, 9, 20]), tokens=20, starts=_ints([3, 0]), **c.scales)
        assert torch.equal(out[:, :2, off:off + 64], ko) and torch.equal(out[:, 2:4, off:off + 64], vo)
        out[:, :4, off:off + 64] = 0
        assert not out.any()


def test_far_pages(pkg):
    """Offsets past 2^31 bytes and elements."""
    pages = 40000
    k = torch.empty(pages, 4, 128, 128, dtype=I8, device="cuda")   # 2.6e9 elements
    v, s = torch.empty_like(k), torch.empty(pages, 4, 128, device="cuda")
    vs = torch.empty_like(s)
    table = _ints([[pages - 1, 5]])
    a, b = _rows(200, 4, 128, BF, 8)
    a = a.nan_to_num(posinf=1.0)
    pkg.kv_cache_write(a, b, k, v, table, _ints([0]), offsets=_ints([0, 200]), k_scale=s, v_scale=vs)
    small = Cache(1, 2, 4, 128, 128, I8)
    pkg.kv_cache_write(a, b, small.k, small.v, small.table, _ints([0]), offsets=_ints([0, 200]), **small.scales)
    got = pkg.kv_cache_read(k, v, table, _ints([0, 200]), tokens=200, k_scale=s, v_scale=vs)
    want = pkg.kv_cache_read(small.k, small.v, small.table, _ints([0, 200]), tokens=200, **small.scales)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_codes_are_act_quants(pkg):
    k, v = _rows(64, 4, 128, BF, 5)
    for q in (I8, E4):
        c = Cache(1, 4, 4, 16, 128, q)
        pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints([0]), offsets=_ints([0, 64]), **c.scales)
        codes, scale = pkg.act_quant(k.reshape(256, 128), qdtype=q)
        pages, offs = c.places([0], [64])
        assert torch.equal(_raw(c.k[pages, :, offs]).reshape(256, 128), _raw(codes))
        assert torch.equal(c.ks[pages, :, offs].reshape(-1).view(torch.int32), scale.view(torch.int32))


def test_many_sequences_and_empty_ones(pkg):
    """Offsets found among thousands of sequences, most of them empty."""
    seqs = 3000
    counts = [(s * 7919 % 11 == 0) * (1 + s % 3) for s in range(seqs)]
    c = Cache(seqs, 1, 1, 16, 64, E4)
    n = sum(counts)
    k, v = _rows(n, 1, 64, BF, 2)
    k = k.nan_to_num(posinf=1.0)
    off = _ints([0] + torch.tensor(counts).cumsum(0).tolist())
    pkg.kv_cache_write(k, v, c.k, c.v, c.table, _ints([2] * seqs), offsets=off, **c.scales)
    pages, offs = c.places([2] * seqs, counts)
    _check_written(c, k, c.k, c.ks, pages, offs)
    got, _ = pkg.kv_cache_read(c.k, c.v, c.table, off, tokens=n, starts=_ints([2] * seqs), dtype=FF, **c.scales)
    want = c.k[pages, :, offs].float() * c.ks[pages, :, offs][..., None]
    assert torch.equal(got, want)


def test_nothing_to_do(pkg):
    c = Cache(2, 1, 2, 16, 64, I8)
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    pkg.kv_cache_write(e, e, c.k, c.v, c.table, _ints([0, 0]), offsets=_ints([0, 0, 0]), **c.scales)
    assert pkg.kv_cache_read(c.k, c.v, c.table, _ints([0, 0, 0]), tokens=0, **c.scales)[0].shape == (0, 2, 64)
    none = c.table[:0]
    pkg.kv_cache_write(e, e, c.k, c.v, none, _ints([]), **c.scales)


def test_graph(pkg):
    c = Cache(3, 2, 2, 16, 64, E4)
    k, v = _rows(3, 2, 64, BF, 1)
    k = k.nan_to_num(posinf=1.0)
    starts, off = _ints([0, 5, 31]), _ints([0, 1, 7, 39])
    graph = torch.cuda.CUDAGraph()
    pkg.kv_cache_write(k, v, c.k, c.v, c.table, starts, **c.scales)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkg.kv_cache_write(k, v, c.k, c.v, c.table, starts, **c.scales)
        ko, vo = pkg.kv_cache_read(c.k, c.v, c.table, off, tokens=39, **c.scales)
        starts += 1
    starts.copy_(_ints([0, 0, 0]))
    for i in range(3):
        k.mul_(0.5)
        graph.replay()
        at = [c.at(s, i) for s in range(3)]
        pages, offs = (torch.tensor(t, device="cuda") for t in zip(*at))
        _check_written(c, k, c.k, c.ks, pages, offs)
        want, _ = pkg.kv_cache_read(c.k, c.v, c.table, off, tokens=39, **c.scales)
        assert torch.equal(ko, want)


def test_refusals(pkg):
    c = Cache(2, 1, 2, 16, 64, I8)
    k, v = _rows(2, 2, 64, BF, 1)
    good = dict(k=k, v=v, k_cache=c.k, v_cache=c.v, page_table=c.table, starts=_ints([0, 0]), **c.scales)
    pkg.kv_cache_write(**good)
    half = torch.zeros(4, 2, 16, 64, dtype=HF, device="cuda")
    narrow = torch.zeros(4, 2, 16, 24, dtype=I8, device="cuda")
    odd = torch.zeros(4 * 2 * 16 * 64 + 1, dtype=I8, device="cuda")[1:].view(4, 2, 16, 64)
    for bad in (dict(k=k[:1]), dict(v=v.float()), dict(k=k[:, :1], v=v[:, :1]), dict(k_scale=None),
                dict(v_scale=c.vs.double()), dict(k_scale=c.ks[:2]), dict(v_cache=c.v[:2]),
                dict(v_cache=half), dict(k_cache=half, v_cache=half),
                dict(k_cache=half, v_cache=half, k_scale=None, v_scale=None),   # bf16 rows, fp16 cache
                dict(page_table=c.table.long()), dict(page_table=c.table[:1]), dict(starts=_ints([0])),
                dict(starts=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(starts=_ints([0, 0]).cpu()),
                dict(offsets=_ints([0, 1])), dict(k_cache=narrow, v_cache=narrow), dict(k_cache=odd, v_cache=odd),
                dict(k=k.cpu(), v=v.cpu())):
        with pytest.raises((ValueError, TypeError, pkg.ConvError)):
            pkg.kv_cache_write(**{**good, **bad})
    read = dict(k_cache=c.k, v_cache=c.v, page_table=c.table, offsets=_ints([0, 1, 2]), **c.scales)
    for bad in (dict(), dict(tokens=2, k_out=k, v_out=v), dict(k_out=k), dict(tokens=2, dtype=I8),
                dict(k_out=k[:, :1], v_out=v[:, :1]), dict(tokens=2, offsets=_ints([0, 2]))):
        with pytest.raises((ValueError, TypeError, pkg.ConvError)):
            pkg.kv_cache_read(**{**read, **bad})
