"""Caches in other orders and with padding; dimensions of size one may have any stride."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I8 = torch.bfloat16, torch.int8


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


@pytest.mark.parametrize("dtype", [I8, BF])
@pytest.mark.parametrize("pages,heads,page", [(6, 1, 16), (1, 2, 48), (40, 3, 1), (40, 1, 1), (1, 1, 40)])
def test_strides_of_dimensions_of_one(pkg, dtype, pages, heads, page):
    """Where a dimension has one element its stride is nobody's: views that differ in
    nothing else are the same cache."""
    width, n = 32, min(pages * page, 40)
    g = torch.Generator(device="cuda").manual_seed(pages + heads)
    k, v = (torch.randn(n, heads, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, 2 * heads, width, generator=g, device="cuda").bfloat16()
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    shape = (pages, heads, page, width)

    def strange(t):
        """The same elements; strides of 5 where there is one element."""
        return t.as_strided(t.shape, [5 if n == 1 else s for n, s in zip(t.shape, t.stride())])

    results = []
    for odd in (lambda t, i: t, lambda t, i: strange(t), lambda t, i: strange(t) if i % 2 else t):
        made = [torch.zeros(shape, device="cuda").to(dtype) for _ in range(2)]
        if dtype is I8:
            made += [torch.ones(shape[:3], device="cuda") for _ in range(2)]
        c = [odd(t, i) for i, t in enumerate(made)] + ([None, None] if dtype is BF else [])
        pkg.kv_cache_write(k, v, c[0], c[1], table, _ints([0]), c[2], c[3], offsets=_ints([0, n]))
        ko, vo = pkg.kv_cache_read(c[0], c[1], table, _ints([0, n]), tokens=n, k_scale=c[2], v_scale=c[3])
        y = pkg.paged_attention(q, c[0], c[1], table, _ints([n]), k_scale=c[2], v_scale=c[3])
        assert not ko.isnan().any() and not y.isnan().any()
        results.append(made + [ko, vo, y])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    # strides that matter still have to be the same, and rows contiguous
    a, b = (torch.zeros(4, 2, 16, width * i, device="cuda").to(dtype)[..., :width] for i in (1, 2))
    s = [torch.ones(4, 2, 16, device="cuda") if dtype is I8 else None for _ in range(2)]
    four = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pkg.kv_cache_read(a, b, four, _ints([0, 4]), tokens=4, k_scale=s[0], v_scale=s[1])
    wide = torch.zeros(4, 2, 16, 2 * width, device="cuda").to(dtype)[..., ::2]
    with pytest.raises(ValueError):
        pkg.kv_cache_read(wide, wide.clone(memory_format=torch.preserve_format), four, _ints([0, 4]), tokens=4,
                          k_scale=s[0], v_scale=s[1])
    if dtype is I8:
        turned = torch.ones(4, 16, 2, device="cuda").transpose(1, 2)
        with pytest.raises(ValueError):
            pkg.kv_cache_read(a, a.clone(), four, _ints([0, 4]), tokens=4, k_scale=turned, v_scale=turned)


@pytest.mark.parametrize("dtype", [I8, BF])
@pytest.mark.parametrize("order", ["phtw", "pthw", "hptw", "tphw", "thpw", "htpw"])
@pytest.mark.parametrize("pads", [(0, 0, 0), (16, 0, 0), (0, 48, 0), (0, 0, 112), (16, 32, 80)])
def test_orders_and_padding(pkg, dtype, order, pads):
    """Pages, heads and tokens of a cache in any order in memory, with rows, and what
    follows them, padded: strides that are no multiples of one another."""
    pages, heads, page, width, n = 13, 3, 32, 48, 400
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(2, 2 * heads, width, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(n, heads, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").int()[None].repeat(2, 1)
    sizes, stride, extent = dict(p=pages, h=heads, t=page, w=width), {}, 1
    for d, pad in zip(reversed(order), (0,) + pads):
        stride[d] = extent + (pad if d != "w" else 0)
        extent = stride[d] * sizes[d]
    results = []
    for strides in (None, [stride[d] for d in "phtw"]):
        made = []
        for _ in range(2):
            if strides is None:
                made.append(torch.zeros(pages, heads, page, width, device="cuda").to(dtype))
            else:
                flat = torch.full((extent,), 9, device="cuda").to(dtype)
                made.append(flat.as_strided((pages, heads, page, width), strides))
        s = [torch.zeros(pages, heads, page, device="cuda") if dtype is I8 else None for _ in range(2)]
        pkg.kv_cache_write(k, v, *made, table[:1], _ints([0]), *s, offsets=_ints([0, n]))
        ko, vo = pkg.kv_cache_read(*made, table[:1], _ints([0, n]), tokens=n, k_scale=s[0], v_scale=s[1])
        y = pkg.paged_attention(q, *made, table, _ints([n, 77]), k_scale=s[0], v_scale=s[1])
        assert not y.isnan().any()
        results.append([ko, vo, y])
    for a, b in zip(*results):
        assert torch.equal(a, b)
