"""rotary records its gradient, the inverse rotation: against the formula's by torch's own
differentiation in 64 bits, through a chain of operations, with accumulation, and not
where none is asked for."""
import pytest
import torch

import _attention_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


def _inputs(dtype, tokens=37, heads=3, width=80, axes=2, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens)
    x = torch.randn(tokens, heads, width, generator=g, device="cuda").to(dtype)
    w = torch.randn(tokens, heads, width, generator=g, device="cuda").to(dtype)
    return x, w, torch.randint(-500, 500, (tokens, axes), generator=g, device="cuda").int()


@pytest.mark.parametrize("dtype", [BF, HF, FF])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient(pkg, dtype, pairs, inverse):
    x, w, p = _inputs(dtype)
    kw = dict(pairs=pairs, base=500.0, scales=(0.5, 2.0), inverse=inverse)
    leaf = x.clone().requires_grad_()
    y = pkg.rotary(leaf, p, (9, 20), **kw)
    assert y.requires_grad and torch.equal(y.detach(), pkg.rotary(x, p, (9, 20), **kw))
    y.backward(w)
    axis, freq = ref.ladder64((9, 20), 500.0, scales=(0.5, 2.0))
    want, tol = ref.rotary64(w, p, axis, freq, pairs == "interleaved", not inverse)
    assert leaf.grad.dtype is dtype
    ref.check(leaf.grad, want, tol)
    before = leaf.grad.clone()
    pkg.rotary(leaf, p, (9, 20), **kw).backward(w)     # accumulates
    assert torch.equal(leaf.grad, 2 * before)


def test_chain(pkg):
    """Heads of a projection's rows, a gradient that is broadcast (strides of 0), two uses."""
    x, w, p = _inputs(FF)
    leaf = torch.cat([x, w], 1).requires_grad_()
    y = pkg.rotary(leaf[:, :3], p, (9, 20)) * 2 + pkg.rotary(leaf[:, 3:], p, (9, 20), inverse=True)
    y.sum().backward()
    axis, freq = ref.ladder64((9, 20))
    ones = torch.ones_like(x)
    for part, inverse, times in ((leaf.grad[:, :3], True, 2), (leaf.grad[:, 3:], False, 1)):
        want, tol = ref.rotary64(ones, p, axis, freq, False, inverse)
        ref.check(part, want * times, tol * times)


def test_differences(pkg):
    """One element moved by h moves the loss by h times its gradient (a linear map)."""
    x, w, p = _inputs(FF, tokens=4, heads=2)
    leaf = x.clone().requires_grad_()
    (pkg.rotary(leaf, p, (9, 20)) * w).sum().backward()
    for e in (0, 17, 40, 58, 79):
        up, down = x.clone(), x.clone()
        up[3, 1, e] += 1.0
        down[3, 1, e] -= 1.0
        d = [(pkg.rotary(t, p, (9, 20)).double() * w.double())[3, 1].sum() for t in (up, down)]
        # two elements of a pair take part; their products' roundings (2^-19 with the sines')
        slack = 80 * 2.0 ** -19 * float(w[3, 1].abs().max()) * float(up[3, 1].abs().max() + 1)
        assert abs(float(d[0] - d[1]) / 2 - float(leaf.grad[3, 1, e])) <= slack


def test_only_where_it_is_asked_for(pkg):
    x, w, p = _inputs(BF)
    assert not pkg.rotary(x, p, (9, 20)).requires_grad
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        assert not pkg.rotary(leaf, p, (9, 20)).requires_grad
    out = torch.empty_like(x)
    got = pkg.rotary(leaf, p, (9, 20), out=out)      # a given output records nothing, as documented
    assert got is out and not got.requires_grad
    assert torch.equal(got, pkg.rotary(x, p, (9, 20)))


def test_gradient_of_the_gradient(pkg):
    """The map is linear: the gradient's own gradient turns the other way."""
    x, w, p = _inputs(FF, tokens=5)
    leaf, up = x.clone().requires_grad_(), w.clone().requires_grad_()
    got, = torch.autograd.grad(pkg.rotary(leaf, p, (9, 20)), leaf, up, create_graph=True)
    back, = torch.autograd.grad(got, up, x)
    axis, freq = ref.ladder64((9, 20))
    want, tol = ref.rotary64(x, p, axis, freq)
    ref.check(back, want, tol)


def test_in_a_graph(pkg):
    """Forward and backward captured; positions and gradients are other ones at the replay."""
    x, w, p = _inputs(FF)
    leaf = x.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(pkg.rotary(leaf, p, (9, 20)), leaf, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(pkg.rotary(leaf, p, (9, 20)), leaf, w)
    p += 7
    w.mul_(0.5)
    graph.replay()
    axis, freq = ref.ladder64((9, 20))
    want, tol = ref.rotary64(w, p, axis, freq, False, True)
    ref.check(got, want, tol)


def test_positions_that_change(pkg):
    """Positions changed in place before the backward pass are an error, not another gradient."""
    x, w, p = _inputs(FF)
    y = pkg.rotary(x.clone().requires_grad_(), p, (9, 20))
    p += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.backward(w)


def test_streams_and_empty(pkg):
    x, w, p = _inputs(FF)
    side = torch.cuda.Stream()
    leaf = x.clone().requires_grad_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = pkg.rotary(leaf, p, (9, 20))
        y.backward(w)
    torch.cuda.current_stream().wait_stream(side)
    axis, freq = ref.ladder64((9, 20))
    want, tol = ref.rotary64(w, p, axis, freq, False, True)
    ref.check(leaf.grad, want, tol)
    none = torch.zeros(0, 3, 80, device="cuda", requires_grad=True)
    pkg.rotary(none, p[:0], (9, 20)).sum().backward()
    assert none.grad.shape == (0, 3, 80)


def test_arguments_that_change(pkg):
    """The backward pass takes the frequencies and scales of the call, whatever became of the lists."""
    x, w, p = _inputs(FF, axes=2)
    freq, scales = [0.1 * (i + 1) for i in range(29)], [1.0, 2.0]
    leaf = x.clone().requires_grad_()
    y = pkg.rotary(leaf, p, (9, 20), frequencies=freq, scales=scales)
    want = pkg.rotary(w, p, (9, 20), frequencies=freq, scales=scales, inverse=True)
    freq[:], scales[:] = [0.0] * 29, [0.0, 0.0]
    y.backward(w)
    assert torch.equal(leaf.grad, want)
