"""Calls on a given stream while the current one is busy with memory that it has
already freed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _busy_with_freed(shapes):
    """Tensors written late on the current stream and freed before that."""
    torch.cuda.empty_cache()
    blocks = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in shapes]
    torch.cuda._sleep(100_000_000)      # 50 ms or so
    for b in blocks:
        b.fill_(85)


@pytest.mark.parametrize("q", [I8, E4])
def test_results_are_not_written_over(pkg, q):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randn(1030, 2051, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    w = (torch.randn(1500, 2051, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
    want = pkg.linear_w8a8(x, w)
    t = torch.randn(1030, 2051, generator=g, device="cuda").bfloat16()
    norm = pkg.rms_norm_quant(t, residual=t, qdtype=q)
    act = pkg.act_quant(t, act="silu", qdtype=q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        # blocks of the sizes that the calls allocate: output, staged operands, codes
        _busy_with_freed([want.numel() * 2, 2064 * (1030 + 1500), 1030 * 2051, 1030 * 2051 * 2,
                          1030 * 4])
        got = pkg.linear_w8a8(x, w, stream=side)
        got_norm = pkg.rms_norm_quant(t, residual=t, qdtype=q, stream=side)
        got_act = pkg.act_quant(t, act="silu", qdtype=q, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for a, b in zip((*got_norm, *got_act), (*norm, *act)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
