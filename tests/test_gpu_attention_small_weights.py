"""fp16 weights of many keys that one key outweighs by far: what they add up to is kept.

One key's score lies 17.4 above all others', so that each of those has a weight of
2^-25.1 of the largest, below half of fp16's smallest step of it; 200000 of them hold
0.55% of the mass, over ten times fp16's own half step.  Tolerance: ``attention64``'s with
the largest weight at 2^15 (paged) or 2^7 (packed) in fp16, so that its absolute step,
2^-25, is 2^-36 or 2^-32 of the largest weight."""
import math

import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I8, E4 = torch.int8, torch.float8_e4m3fn
N, WIDTH, ABOVE = 200000, 64, 17.4


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


def _keys(at, dtype=HF):
    """Keys and a query with scores of 0 and, of key `at`, ABOVE; values that share a sign."""
    g = torch.Generator(device="cuda").manual_seed(at + 1)
    k = torch.zeros(N, 1, WIDTH, device="cuda")
    k[at, 0, 0] = 1.0
    v = 1 + torch.rand(N, 1, WIDTH, generator=g, device="cuda")
    v[at] = 0.0
    q = torch.zeros(1, 1, WIDTH, device="cuda")
    q[0, 0, 0] = ABOVE
    return q.to(dtype), k.to(HF), v.to(HF)


def _check(got, q, k, v, kept, coarse=None):
    want, tol = ref.attention64(q, k, v, weights=HF, scale=1.0, causal=False, coarse=coarse)
    total = 1 + (N - 1) * math.exp(-float(q[0, 0, 0]))
    largest = float(v.double().abs().max()) if coarse is None else coarse
    tol = tol - (2.0 ** -25 - kept) * N * largest / total
    assert float((tol / want).max()) < 0.75      # all of the others' part is 1
    ref.check(got, want, tol)


@pytest.mark.parametrize("at", [0, 77777, N - 1])
def test_packed(pkg, at):
    q, k, v = _keys(at)
    got = pkg.packed_attention(q.expand(130, 1, WIDTH).contiguous(), k, v, _ints([0, 130]), _ints([0, N]), scale=1.0)
    for row in (0, 129):
        _check(got[row:row + 1], q, k, v, 2.0 ** -32)


@pytest.mark.parametrize("at", [0, 77777, N - 1])
@pytest.mark.parametrize("cache,dtype", [(HF, HF), (I8, BF), (E4, HF)])
@pytest.mark.parametrize("seqs", [1, 400])
def test_paged(pkg, at, cache, dtype, seqs):
    """One sequence, split over all CTAs, and as many as there are CTAs (on the same pages)."""
    q, k, v = _keys(at, dtype)
    scales, coarse = {}, None
    if cache is not HF:
        # codes with one scale: 0 or 1, and whole numbers
        s = torch.full((N // 16, 1, 16), 2.0 ** -4, device="cuda")
        scales = dict(k_scale=s, v_scale=s)
        k, v = k, (v.float() * 16).round().to(HF) / 16
        pools = [(t.float() * 16).to(cache) for t in (k, v)]
        coarse = (127 if cache is I8 else 448) / 16
        if cache is E4:
            v = (pools[1].float() / 16).to(HF)
    else:
        pools = [k, v]
    pools = [t.view(N // 16, 16, 1, WIDTH).transpose(1, 2) for t in pools]
    table = torch.arange(N // 16, device="cuda").int()[None].repeat(seqs, 1)
    got = pkg.paged_attention(q.repeat(seqs, 1, 1), *pools, table, _ints([N] * seqs), scale=1.0, **scales)
    for row in (0, seqs // 2, seqs - 1):
        _check(got[row:row + 1], q, k, v, 2.0 ** -36, coarse)
