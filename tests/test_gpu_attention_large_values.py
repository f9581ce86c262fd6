"""bf16 values next to the type's largest and smallest magnitudes: a weighted mean of
finite values is finite, although sums of weights times values are not; and small values
keep their bits.  Tolerances are ``attention64``'s, relative to the values, and beside them
2^-125 for each of a row's products of 16 tokens: sums of values times 2^-24 times weights
are in fp32, in steps of 2^-149, and the sum of weights is 2^-24 at least."""
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


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(n, heads, kv, width, power, rising, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + n + width)
    q, k = (torch.randn(n, h, width, generator=g, device="cuda") for h in (heads, kv))
    v = (0.5 + 0.5 * torch.rand(n, kv, width, generator=g, device="cuda"))
    v *= torch.where(torch.arange(width, device="cuda") % 3 > 0, 1.0, -1.0)   # columns of one sign
    if rising:   # scores that grow slowly: weights stay above what they are relative to
        q, k = q.abs(), k.abs() * (1 + torch.arange(n, device="cuda")[:, None, None] / n)
    # (through 64 bits: v * 2^128 may be the type's largest)
    v = (v.double() * 2.0 ** power).clamp(-3.38e38, 3.38e38).to(BF)
    assert bool(torch.isfinite(v).all())
    return q.to(BF), k.to(BF), v


def _check(got, q, k, v, causal):
    want, tol = ref.attention64(q, k, v, causal=causal, weights=BF)
    assert bool(torch.isfinite(got).all())
    ref.check(got, want, tol + 2.0 ** -125 * (k.shape[0] / 16 + 32))


@pytest.mark.parametrize("power", [128, 124, 119, -100, -112])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_packed(pkg, power, rising, causal):
    for lens, heads, width in (([300, 99], 2, 64), ([2000, 1300], 30, 128)):
        q, k, v = _rows(sum(lens), heads, 1, width, power, rising)
        got = pkg.packed_attention(q, k, v, _ints([0, lens[0], sum(lens)]), causal=causal)
        a = 0
        for n in lens:
            _check(got[a:a + n, :1], q[a:a + n, :1], k[a:a + n], v[a:a + n], causal)
            a += n


@pytest.mark.parametrize("power", [128, 124, 119, -100, -112])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("width", [64, 256])
def test_paged(pkg, power, rising, width):
    n, page = 4000, 16
    q, k, v = _rows(n, 3, 1, width, power, rising)
    pools = [t.view(n // page, page, 1, width).transpose(1, 2) for t in (k, v)]
    table = torch.arange(n // page, device="cuda").int()[None].repeat(2, 1)
    got = pkg.paged_attention(q[-2:], *pools, table, _ints([n, 333]))
    _check(got[:1], q[-2:-1], k, v, False)
    _check(got[1:], q[-1:], k[:333], v[:333], False)
