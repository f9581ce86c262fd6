"""The cache's forms for many rows (several rows or runs of elements a lane): what was
written against the rows, what is read against what the cache holds, at every width of
lanes, for heads that fill a lane's rows and heads that do not."""
import pytest
import torch

import _token_ref as tref

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
I8, E4 = torch.int8, torch.float8_e4m3fn
PAGE = 24


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


def _case(heads, width, dtype, rows, odd):
    """Rows of ragged sequences (empty ones among them), in no sequence at both ends, for a
    pool with marked contents; where each sequence's row lies."""
    g = torch.Generator(device="cuda").manual_seed(heads * 1000 + width)
    # every launch far beyond the switch to several rows a lane
    tokens = max(3000, 2_600_000 // (heads * width))
    cuts = sorted(int(c) for c in torch.randint(0, tokens, (11,), generator=g, device="cuda"))
    counts = [b - a for a, b in zip([0] + cuts, cuts + [tokens])] + [0]
    starts = [(37 * s) % 50 for s in range(len(counts))]
    per = -(-(max(counts) + 50) // PAGE)
    pages = per * len(counts) + 1
    table = torch.randperm(pages, generator=g, device="cuda")[:per * len(counts)].view(len(counts), per).int()
    pos = torch.cat([torch.arange(n, device="cuda") + a for n, a in zip(counts, starts)])
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
    page, off = table[seq, pos // PAGE].long(), pos % PAGE
    pad = 8 if not odd else 7
    k, v = (torch.randn(tokens + 5, heads, width + pad, generator=g, device="cuda").to(rows)[..., odd:odd + width]
            for _ in range(2))
    k[40] = 0.0
    v[41, 0, 3], v[42, heads - 1, width - 1] = float("nan"), float("-inf")
    k[43, 0] *= 1e-30 if rows is not HF else 1e-4
    mark = torch.full((pages, heads, PAGE, width), 7, device="cuda").to(dtype)
    pool = [mark.clone(), mark.clone()]
    scales = [torch.full((pages, heads, PAGE), 0.5, device="cuda") if dtype in (I8, E4) else None for _ in range(2)]
    offsets = _ints([0] + torch.tensor(counts).cumsum(0).tolist()) + 2      # rows 0, 1 and the last three: none
    return tokens, k, v, pool, scales, table, _ints(starts), offsets, page, off


KINDS = [(I8, BF), (I8, FF), (E4, HF), (E4, FF), (E4, BF), (BF, BF), (HF, HF)]


@pytest.mark.parametrize("heads", [1, 2, 5, 6, 8, 11])
@pytest.mark.parametrize("width", [64, 80, 128, 256, 48])
@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("odd", [0, 1])
def test_write_then_read(pkg, heads, width, dtype, rows, odd):
    tokens, k, v, pool, scales, table, starts, offsets, page, off = _case(heads, width, dtype, rows, odd)
    kw = dict(k_scale=scales[0], v_scale=scales[1])
    was = [None if t is None else t.clone() for t in pool + scales]
    pkg.kv_cache_write(k, v, *pool, table, starts, offsets=offsets, **kw)
    for x, codes, scale in ((k, pool[0], scales[0]), (v, pool[1], scales[1])):
        x, got = x[2:2 + tokens], codes[page, :, off]
        if scale is None:
            assert torch.equal(got.view(torch.int16), x.contiguous().view(torch.int16))
            continue
        size = scale[page, :, off]
        bad = ~torch.isfinite(x.float()).all(-1)
        assert bool(torch.isnan(size[bad]).all()) and not _raw(got)[bad].any()
        tref.check_quant(x[~bad].double(), got[~bad], size[~bad], 2.0 ** -23)
    for now, before in zip(pool + scales, was):      # nothing else was touched
        if now is not None:
            rest = _raw(now).clone()
            rest[page, :, off] = _raw(before)[page, :, off]
            assert torch.equal(rest, _raw(before))
    for out in ((rows, BF) if rows is not BF else (BF, HF, FF)):
        wide = [torch.full((tokens + 5, heads, width + 8), 9.0, dtype=out, device="cuda") for _ in range(2)]
        ko, vo = (t[..., odd:odd + width] for t in wide)
        pkg.kv_cache_read(*pool, table, offsets, starts=starts, k_out=ko, v_out=vo, **kw)
        for got, codes, scale in ((ko, pool[0], scales[0]), (vo, pool[1], scales[1])):
            want = codes[page, :, off].double()
            if scale is not None:
                want = want * scale[page, :, off].double()[..., None]
            assert bool((got[:2] == 9.0).all() & (got[2 + tokens:] == 9.0).all())
            got = got[2:2 + tokens]
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan)
            fine = torch.isfinite(want)
            assert torch.equal(got.double()[~fine & ~nan], want[~fine & ~nan])
            tref.check_rounded(got[fine], want[fine], 2.0 ** -24 * want[fine].abs())
        for t in wide:
            t[..., odd:odd + width] = 9.0
            assert bool((t == 9.0).all())


@pytest.mark.parametrize("dtype", [I8, BF])
@pytest.mark.parametrize("heads", [1, 8])
def test_one_token_of_many_sequences(pkg, dtype, heads):
    """No offsets: every row a sequence of its own, some of them not running."""
    seqs, width = 20000 // heads, 128
    g = torch.Generator(device="cuda").manual_seed(heads)
    table = torch.randperm(seqs, generator=g, device="cuda").int()[:, None]
    k, v = (torch.randn(seqs, heads, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool = [torch.zeros(seqs, heads, PAGE, width, device="cuda").to(dtype) for _ in range(2)]
    scales = [torch.zeros(seqs, heads, PAGE, device="cuda") if dtype is I8 else None for _ in range(2)]
    starts = torch.randint(-3, PAGE + 3, (seqs,), generator=g, device="cuda").int()
    pkg.kv_cache_write(k, v, *pool, table, starts, k_scale=scales[0], v_scale=scales[1])
    live = (starts >= 0) & (starts < PAGE)
    page, off = table[live, 0].long(), starts[live].long()
    for x, codes, scale in ((k, pool[0], scales[0]), (v, pool[1], scales[1])):
        got = codes[page, :, off]
        if scale is None:
            assert torch.equal(got, x[live])
        else:
            tref.check_quant(x[live].double(), got, scale[page, :, off], 2.0 ** -23)
        codes[page, :, off] = 0
        assert not codes.any()


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("heads", [1, 8])
def test_pages_that_are_not_there(pkg, dtype, heads):
    width, per, seqs = 128, 400, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    n = per * PAGE
    table = torch.randperm(seqs * per, generator=g, device="cuda").view(seqs, per).int()
    gone = torch.rand(seqs, per, generator=g, device="cuda") < 0.2
    bad = table.clone()
    bad[gone] = torch.tensor([-1, seqs * per, 2 ** 31 - 1], dtype=torch.int32, device="cuda")[
        torch.randint(0, 3, (int(gone.sum()),), generator=g, device="cuda")]
    k, v = (torch.randn(seqs * n, heads, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool = [torch.zeros(seqs * per, heads, PAGE, width, device="cuda").to(dtype) for _ in range(2)]
    scales = [torch.zeros(seqs * per, heads, PAGE, device="cuda") if dtype is E4 else None for _ in range(2)]
    kw = dict(k_scale=scales[0], v_scale=scales[1])
    off = _ints([0, n, 2 * n, 3 * n])
    pkg.kv_cache_write(k, v, *pool, bad, _ints([0, 0, 0]), offsets=off, **kw)
    missing = gone.reshape(-1).repeat_interleave(PAGE)
    for codes in pool:
        assert not _raw(codes)[table[gone].long()].any()
    ko, vo = pkg.kv_cache_read(*pool, bad, off, tokens=seqs * n, dtype=FF, **kw)
    for got, x in ((ko, k), (vo, v)):
        assert torch.equal(torch.isnan(got).all(-1).all(-1), missing)
        assert bool(torch.isfinite(got[~missing]).all())
        near = (got[~missing] - x[~missing].float()).abs()
        top = x[~missing].float().abs().amax(-1, keepdim=True)
        # codes are within half a step: 2^-4 of themselves, and 2^-10 where e4m3 is subnormal (of a top of 448)
        assert bool((near <= (0 if dtype is BF else 2.0 ** -4 + 2.0 ** -20) * x[~missing].float().abs() + top * 2.0 ** -17).all())
