"""The attention operators as they are used together: the tokens of a video's patch
embedding, frame by frame, turned by their positions, cached in 8 bits, attended to as
a chunk over all that is cached, and one token at a time; the one-token step captured
in a graph and replayed with everything advancing on the device."""
import math

import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SECTIONS = (8, 12, 12)


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


def _cache(pages, heads, page, width, dtype):
    k, v = (torch.zeros(pages, heads, page, width, device="cuda").to(dtype) for _ in range(2))
    s = [torch.full((pages, heads, page), float("nan"), device="cuda") for _ in range(2)] if k.element_size() == 1 else [None] * 2
    return dict(k_cache=k, v_cache=v, k_scale=s[0], v_scale=s[1])


def _held(cache, table, n):
    """The cache's values as they stand, 64 bits."""
    out = []
    for name in "kv":
        c = cache[name + "_cache"][table.long()].double()
        if cache[name + "_scale"] is not None:
            c = c * cache[name + "_scale"][table.long()].double()[..., None]
        out.append(c.transpose(1, 2).reshape(-1, c.shape[1], c.shape[3])[:n])
    return out


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8, BF])
def test_frames_after_a_patch_embedding(pkg, dtype):
    heads, kv, width, page, side, frames = 8, 4, 64, 16, 9, 4
    hidden, n = heads * width, side * side
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    patch = (draw(hidden, 1, 14, 14, 3) / math.sqrt(588)).bfloat16()
    project = (draw((heads + 2 * kv) * width, hidden) / math.sqrt(hidden)).bfloat16()
    cache = _cache(2 * 24 + 1, kv, page, width, dtype)
    table = torch.randperm(49, generator=g, device="cuda")[:48].view(2, 24).int()
    where = torch.arange(n, device="cuda")
    grid = torch.stack([where * 0, where // side, where % side], 1).int()
    axis, freq = ref.ladder64(SECTIONS)
    for t in range(frames):
        pixels = draw(2, 1, side * 14, side * 14, 3).bfloat16()          # two videos
        tokens = pkg.conv_fwd(pixels, patch, (1, 14, 14), 0, 1).view(2 * n, hidden)
        qkv = torch.matmul(tokens.float(), project.float().t()).bfloat16().view(2 * n, heads + 2 * kv, width)
        pos = (grid + _ints([t, 0, 0])).repeat(2, 1)
        turned = qkv[:, :heads + kv]
        want, tol = ref.rotary64(turned, pos, axis, freq)
        pkg.rotary(turned, pos, SECTIONS, out=turned)                    # in place, queries and keys
        ref.check(turned, want, tol)
        pkg.kv_cache_write(qkv[:, heads:heads + kv], qkv[:, heads + kv:], page_table=table,
                           starts=_ints([t * n, t * n]), offsets=_ints([0, n, 2 * n]), **cache)
        all_ = (t + 1) * n
        k, v = pkg.kv_cache_read(page_table=table, offsets=_ints([0, all_, 2 * all_]), tokens=2 * all_, **cache)
        y = pkg.packed_attention(qkv[:, :heads], k, v, _ints([0, n, 2 * n]), _ints([0, all_, 2 * all_]))
        z = pkg.paged_attention(qkv[n - 1::n, :heads], page_table=table, lengths=_ints([all_, all_]), **cache)
        for s in range(2):
            q = qkv[s * n:(s + 1) * n, :heads]
            want, tol = ref.attention64(q, k[s * all_:(s + 1) * all_], v[s * all_:(s + 1) * all_], causal=False, weights=BF)
            ref.check(y[s * n:(s + 1) * n], want, tol)
            hk, hv = _held(cache, table[s], all_)
            codes = dtype is not BF
            coarse = float(cache["v_scale"].nan_to_num().max()) * 448 if codes else None
            want, tol = ref.attention64(q[-1:], hk, hv, weights=torch.float16 if codes else BF, coarse=coarse)
            ref.check(z[s:s + 1], want, tol)


def test_one_token_steps_in_a_graph(pkg):
    """Rotation in place, the write and the attention of one token of each sequence,
    captured once; lengths and positions advance on the device."""
    seqs, heads, kv, width, page = 5, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    start = [0, 15, 100, 33, 16]
    cache = _cache(seqs * 10, kv, page, width, torch.float8_e4m3fn)
    table = torch.randperm(seqs * 10, generator=g, device="cuda").view(seqs, 10).int()
    old = [torch.randn(sum(start), kv, width, generator=g, device="cuda").bfloat16() for _ in range(2)]
    off = _ints([0] + torch.tensor(start).cumsum(0).tolist())
    pkg.kv_cache_write(*old, page_table=table, starts=_ints([0] * seqs), offsets=off, **cache)
    twin = {k: v.clone() for k, v in cache.items()}
    qkv = torch.zeros(seqs, heads + 2 * kv, width, dtype=BF, device="cuda")
    lengths, at = _ints([n + 1 for n in start]), _ints(start)
    out = torch.empty(seqs, heads, width, dtype=BF, device="cuda")

    def step(x, c, n, p, o):
        pos = torch.stack([p, p * 0 + 3, p % 7], 1).int()
        pkg.rotary(x[:, :heads + kv], pos, (16, 24, 24), out=x[:, :heads + kv])
        pkg.kv_cache_write(x[:, heads:heads + kv], x[:, heads + kv:], page_table=table, starts=p, **c)
        return pkg.paged_attention(x[:, :heads], page_table=table, lengths=n, out=o, **c)

    step(qkv.clone(), {k: v.clone() for k, v in cache.items()}, lengths, at, out)   # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qkv, cache, lengths, at, out)
        lengths += 1
        at += 1
    n2, at2 = lengths.clone(), at.clone()
    for i in range(6):
        new = torch.randn(seqs, heads + 2 * kv, width, generator=g, device="cuda").bfloat16()
        qkv.copy_(new)
        graph.replay()
        want = step(new, twin, n2, at2, torch.empty_like(out))
        n2 += 1
        at2 += 1
        assert torch.equal(out, want), i
    for a, b in zip(cache.values(), twin.values()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, BF])
@pytest.mark.parametrize("pages", [23, 24, 25])
@pytest.mark.parametrize("seqs", [1, 7, 300])
def test_tables_that_are_split_or_not(pkg, seqs, pages, dtype):
    """Tables of up to and beyond the tokens that one CTA takes alone, batches of up to and
    beyond those that run at once, sequences that see nothing or more than there is."""
    heads, kv, width, page = 8, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(seqs + pages)
    most = pages * page
    lengths = [(0, most, 1, most - 1, 17, -3, 130)[i % 7] if i else most for i in range(seqs)]
    cache = _cache(seqs * pages, kv, page, width, dtype)
    table = torch.randperm(seqs * pages, generator=g, device="cuda").view(seqs, pages).int()
    kept = [max(n, 0) for n in lengths]
    off = _ints([0] + torch.tensor(kept).cumsum(0).tolist())
    rows = [torch.randn(sum(kept), kv, width, generator=g, device="cuda").bfloat16() for _ in range(2)]
    pkg.kv_cache_write(*rows, page_table=table, starts=_ints([0] * seqs), offsets=off, **cache)
    q = torch.randn(seqs, heads, width, generator=g, device="cuda").bfloat16()
    got = pkg.paged_attention(q, page_table=table, lengths=_ints(lengths), **cache)
    need = pkg.paged_attention_workspace_size(seqs, heads, kv, width, page, pages)
    assert (need == 0) == (pages < 25 and seqs < 300)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(got, pkg.paged_attention(q, page_table=table, lengths=_ints(lengths), workspace=ws, **cache))
    codes = dtype is not BF
    coarse = float(cache["v_scale"].nan_to_num().max()) * 448 if codes else None
    for s in sorted(set(range(min(seqs, 8))) | {seqs - 1}):
        if lengths[s] <= 0:
            assert not got[s].any()
            continue
        hk, hv = _held(cache, table[s], lengths[s])
        want, tol = ref.attention64(q[s:s + 1], hk, hv, weights=torch.float16 if codes else BF, coarse=coarse)
        ref.check(got[s:s + 1], want, tol)
    if seqs == 7:
        lengths[3] = most + 1     # past the table
        got = pkg.paged_attention(q, page_table=table, lengths=_ints(lengths), **cache)
        assert bool(got[3].isnan().all()) and not got[:3].isnan().any() and not got[4:].isnan().any()
