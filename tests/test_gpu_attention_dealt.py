"""packed_attention over long documents whose jobs are dealt to CTAs that ask: every row
is computed whatever the documents' lengths, order and number, next to buffers that are
mostly unused, in replayed graphs and with two calls at once."""
import random

import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _offsets(lens):
    return torch.tensor([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist(),
                        dtype=torch.int32, device="cuda")


def _rows(n, heads, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, heads, width, generator=g, device="cuda").bfloat16()


def _check(out, q, k, v, lens, causal, heads=(0, -1)):
    a = 0
    group = q.shape[1] // k.shape[1]
    for n in lens:
        for h in heads:   # (all heads of a job's documents go the same way)
            h %= q.shape[1]
            want, tol = ref.attention64(q[a:a + n, h:h + 1], k[a:a + n, h // group:h // group + 1],
                                        v[a:a + n, h // group:h // group + 1], causal=causal, weights=BF)
            ref.check(out[a:a + n, h:h + 1], want, tol)
        a += n
    assert bool((out[a:] == 7.0).all())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("lens", [
    [1500, 0, 0, 2100, 1, 900], [0] * 5 + [3000] + [0] * 3, [2500, 130, 128, 127, 1, 2000, 700],
    [random.Random(4).randint(300, 900) for _ in range(20)]])
def test_lengths(pkg, lens, width, causal):
    heads, kv = 24, 8
    n = sum(lens)
    q, k, v = _rows(n + 3, heads, width, 1), _rows(n + 3, kv, width, 2), _rows(n + 3, kv, width, 3)
    out = torch.full_like(q, 7.0)
    pkg.packed_attention(q, k, v, _offsets(lens), causal=causal, out=out)
    _check(out, q, k, v, lens, causal)


def test_many_documents_with_rows(pkg):
    """More documents than are looked through at a time, long on the whole."""
    r = random.Random(5)
    lens = [r.choice((0, 1, 70, 1100, 1300)) for _ in range(300)]
    n = sum(lens)
    assert n // 300 > 384
    q, k, v = (_rows(n + 3, 2, 64, s) for s in (1, 2, 3))
    out = torch.full_like(q, 7.0)
    pkg.packed_attention(q, k, v, _offsets(lens), causal=True, out=out)
    _check(out, q, k, v, lens, True)


def test_mostly_unused_buffers(pkg):
    """Offsets on the device say how much of the buffers is in use: a replayed graph."""
    rows, heads = 40000, 16
    q, k, v = (_rows(rows, heads, 64, s) for s in (1, 2, 3))
    off, out = _offsets([700, 900]), torch.full_like(q, 7.0)
    pkg.packed_attention(q, k, v, off, causal=True, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.packed_attention(q, k, v, off, causal=True, out=out)
    for lens in ([700, 900], [0, 0], [3000, 5], [1, 0], [20000, 2]):
        off.copy_(_offsets(lens))
        out.fill_(7.0)
        graph.replay()
        if lens[0] < 20000:
            _check(out, q, k, v, lens, True)
        else:   # its last rows
            want, tol = ref.attention64(q[19900:20000, :1], k[:20000, :1], v[:20000, :1], causal=True, weights=BF)
            ref.check(out[19900:20000, :1], want, tol)
            assert bool((out[20002:] == 7.0).all()) and bool((out[:20002] != 7.0).any(-1).all())


def test_two_calls_at_once(pkg):
    lens = [[2600, 900, 1400], [1200, 3000, 500]]
    ps = [[_rows(sum(n), h, 128, 7 + i) for i, h in enumerate((16, 4, 4))] for n in lens]
    offs = [_offsets(n) for n in lens]
    want = [pkg.packed_attention(*p, o, causal=True) for p, o in zip(ps, offs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for _ in range(5):
        got.append([pkg.packed_attention(*p, o, causal=True, stream=s) for p, o, s in zip(ps, offs, streams)])
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)


def test_calls_that_take_one_anothers_output(pkg):
    """Launches may begin before the one ahead of them has ended, but see all of it."""
    lens = [2300, 600, 1500]
    q, k, v = (_rows(sum(lens), h, 128, 11 + i) for i, h in enumerate((16, 16, 16)))
    off = _offsets(lens)
    args = dict(q_offsets=off, causal=True)
    outs = [torch.empty_like(q) for _ in range(6)]

    def chain(wait):
        x = q
        for o in outs:
            x = pkg.packed_attention(x, k, x, out=o, **args)   # values from the call before
            if wait:
                torch.cuda.synchronize()
        return [o.clone() for o in outs]

    want = chain(True)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    got = chain(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for o in outs:
        o.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = chain(False)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
