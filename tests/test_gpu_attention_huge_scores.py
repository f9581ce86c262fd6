"""fp16 and 8-bit attention with scores that fp32 holds in steps of 4 and more: weights that
lag behind the maximum they are relative to stay within f16.  Scores are sums of 2^25 and a
whole multiple of 4 that grows from tile to tile, so that they are exact in fp32; what
follows (log2 e times a score, in steps of 4) is off by 2 at most for each key, which leaves
results within the range of the values, and a key that outweighs all others by far alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I8 = torch.int8


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


def _rows(n, step, block):
    g = torch.Generator(device="cuda").manual_seed(step + block)
    q, k = torch.zeros(1, 1, 64, device="cuda"), torch.zeros(n, 1, 64, device="cuda")
    q[0, 0, 0], q[0, 0, 1] = 8192.0, 4.0
    k[:, 0, 0] = 4096.0
    k[:, 0, 1] = (torch.arange(n, device="cuda") // block) * step
    v = 1 + torch.rand(n, 1, 64, generator=g, device="cuda")
    return q.to(HF), k.to(HF), v.to(HF)


@pytest.mark.parametrize("step", [0, 1, 2, 3])
@pytest.mark.parametrize("block", [128, 16, 1])
def test_packed(pkg, step, block):
    n = 1000
    q, k, v = _rows(n, step, block)
    got = pkg.packed_attention(q.expand(130, 1, 64).contiguous(), k, v, _ints([0, 130]), _ints([0, n]), scale=1.0).float()
    assert bool(((got >= 0.99) & (got <= 2.01)).all())
    if block == 1:    # the last key's score is 64 above the next: 2^92 of the weight
        k[-1, 0, 1] += 16
        got = pkg.packed_attention(q, k, v, _ints([0, 1]), _ints([0, n]), scale=1.0).float()
        assert bool((got - v[-1].float()).abs().max() <= 2.0 ** -9)


@pytest.mark.parametrize("step", [0, 1, 2, 3])
@pytest.mark.parametrize("block", [128, 16, 1])
@pytest.mark.parametrize("cache", [HF, I8])
def test_paged(pkg, step, block, cache):
    n, page = 960, 16
    q, k, v = _rows(n, step, block)
    scales = {}
    if cache is I8:      # 8192 * (64 * 64), 4 * code * 64 / 64
        s = torch.full((n // page, 1, page), 64.0, device="cuda")
        scales = dict(k_scale=s, v_scale=s / 4096)
        k[:, 0, 0], q[0, 0, 1] = 64.0, 1 / 16
        k[:, 0, 1].clamp_(max=127)
        k, v = k.to(I8), (v.float() * 64).round().clamp(max=127).to(I8)
    pools = [t.view(n // page, page, 1, 64).transpose(1, 2) for t in (k, v)]
    table = torch.arange(n // page, device="cuda").int()[None]
    got = pkg.paged_attention(q, *pools, table, _ints([n]), scale=1.0, **scales).float()
    assert bool(((got >= 0.98) & (got <= 2.02)).all())
