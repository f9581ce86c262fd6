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


def test_products_and_convolutions_side_by_side(pkg):
    """Kernels that hold an SM's tensor memory, in clusters of several sizes, on four
    streams at once: each gives what it gives alone."""
    g = torch.Generator(device="cuda").manual_seed(8)
    work = []
    for q, m, n, k in ((I8, 40, 1024, 4096), (E4, 64, 512, 8192), (E4, 128, 2048, 1024),
                       (I8, 300, 1280, 1280), (E4, 1200, 2560, 640), (I8, 1200, 2560, 640)):
        x = (torch.randn(m, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
        w = (torch.randn(n, k, generator=g, device="cuda") * 30).clamp(-127, 127).to(q)
        work.append(lambda s, x=x, w=w: pkg.linear_w8a8(x, w, stream=s))
    xc = torch.randn(1, 4, 24, 24, 256, generator=g, device="cuda").bfloat16()
    wc = torch.randn(256, 3, 3, 3, 256, generator=g, device="cuda").bfloat16()
    work.append(lambda s: pkg.conv_fwd(xc, wc, 1, 1, 1, stream=s))
    want = [f(None) for f in work]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for turn in range(20):
        for i in range(len(work)):
            j = (turn + i) % len(work)
            got.append((j, work[j](streams[(turn * 3 + i) % 4])))
    torch.cuda.synchronize()
    for j, y in got:
        assert torch.equal(y, want[j]), j


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("tokens", [1, 7, 16, 40])
def test_chains_over_the_same_buffers(pkg, q, tokens):
    """Blocks back to back, in a graph, over the same buffers: kernels that start
    while the ones before them run read what those write, not what they read there
    a few kernels ago."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    width, inner = 256, 512
    layers = []
    for _ in range(6):
        up, sup = pkg.act_quant(torch.randn(2 * inner, width, generator=g, device="cuda") / 16, qdtype=q)
        down, sdown = pkg.act_quant(torch.randn(width, inner, generator=g, device="cuda") / 16, qdtype=q)
        layers.append((up, sup, down, sdown))
    new = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")   # noqa: E731
    a, sa, b, sb = new(tokens, width, t=q), new(tokens, t=torch.float32), \
        new(tokens, inner, t=q), new(tokens, t=torch.float32)
    h, y, res = new(tokens, 2 * inner), new(tokens, width), new(tokens, width)

    def chain(sync):
        for up, sup, down, sdown in layers * 5:
            pkg.rms_norm_quant(y, residual=res, out=a, scale_out=sa, residual_out=res)
            sync()
            pkg.linear_w8a8(a, up, sa, sup, out=h)
            sync()
            pkg.act_quant(h, "silu", gated=True, out=b, scale_out=sb)
            sync()
            pkg.linear_w8a8(b, down, sb, sdown, out=y)
            sync()

    start = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()

    def reset():
        y.copy_(start)
        res.copy_(start)

    reset()
    chain(torch.cuda.synchronize)
    want = y.clone(), res.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for run in range(10):
        reset()
        if run % 2:
            chain(lambda: None)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(res, want[1]), run
