"""Seeded problems of the token operators in slices of larger buffers: whatever
lies beside an operand is NaN (or the largest code) and must not be read into a
result, whatever lies beside an output must stay."""
import math
import random

import pytest
import torch

import _token_ref as ref

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.float8_e4m3fn
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import implicit_gemm_convolution_conv3d_gb300 as p
    p.load_library()
    yield p
    assert p.conv_get_device_status() == 0


class _Slice:
    """[rows, width] of `dtype` inside a buffer of 0x7F bytes (NaN in e4m3, bf16 and
    fp16, 127 in int8, 3.4e38 in fp32)."""

    def __init__(self, rng, rows, width, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        unit = rng.choice([1, 1, 4, 16 // size if size < 16 else 1, 8])
        left, more = rng.randrange(0, 4) * unit, rng.randrange(0, 4) * unit
        stride = width + more
        if rng.random() < 0.5:      # rows on 16 bytes, of any length
            stride = -(-stride * size // 16) * 16 // size
        self.bytes = torch.full(((left + rows * stride + 64) * size,), 0x7F, dtype=torch.uint8,
                                device="cuda")
        flat = self.bytes.view(dtype)
        self.at = torch.as_strided(flat, (rows, width), (stride, 1), left)
        mark = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
        torch.as_strided(mark, (rows, width), (stride, 1), left).fill_(False)
        self.beside = mark.repeat_interleave(size)

    def put(self, values):
        self.at.copy_(values)
        return self

    def check(self):
        assert (self.bytes[self.beside] == 0x7F).all(), "written beside the rows"


def _size(rng, hi):
    v = int(math.exp(rng.uniform(0, math.log(hi))))
    return max(1, v // 16 * 16 if rng.random() < 0.4 else v)


@pytest.mark.parametrize("seed", range(60))
def test_norm(pkg, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, width = _size(rng, 400), _size(rng, 36000)
    x_type = rng.choice([BF, HF, FF])
    r_type = rng.choice([None, x_type, FF])
    w_type = rng.choice([None, x_type, FF])
    q = rng.choice([I8, E4])
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x = _Slice(rng, rows, width, x_type).put(randn(rows, width) * 3)
    res = None if r_type is None else _Slice(rng, rows, width, r_type).put(randn(rows, width))
    w = None if w_type is None else _Slice(rng, 1, width, w_type).put(1 + 0.3 * randn(1, width))
    codes, scale = _Slice(rng, rows, width, q), _Slice(rng, 1, rows, FF)
    in_place = res is not None and rng.random() < 0.3
    ro = None if res is None else res if in_place else _Slice(rng, rows, width, r_type)
    eps = rng.choice([1e-6, 1e-5, 0.0])
    weight = None if w is None else w.at[0]
    h, v = ref.norm64(x.at, weight, eps, None if res is None else res.at.clone())
    pkg.rms_norm_quant(x.at, weight, eps, residual=None if res is None else res.at, out=codes.at,
                       scale_out=scale.at[0],
                       residual_out=None if ro is None else res.at if in_place else ro.at)
    ref.check_quant(v, codes.at, scale.at[0], (width / 32 + 64) * 2.0 ** -24)
    if ro is not None:
        ref.check_rounded(ro.at, h, 2.0 ** -24 * h.abs())
    for s in (x, res, w, codes, scale, ro):
        if s is not None:
            s.check()


@pytest.mark.parametrize("seed", range(60))
def test_act(pkg, seed):
    rng = random.Random(1000 + seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, width = _size(rng, 400), _size(rng, 36000)
    gated, act = rng.random() < 0.5, rng.choice(["none", "relu", "silu", "gelu"])
    x_type, q = rng.choice([BF, HF, FF]), rng.choice([I8, E4])
    values = torch.randn(rows, 2 * width if gated else width, generator=g, device="cuda") * 2
    values[:, 0] = values[:, 0].abs() + 0.5      # no row lies in the tail alone
    x = _Slice(rng, rows, values.shape[1], x_type).put(values)
    codes, scale = _Slice(rng, rows, width, q), _Slice(rng, 1, rows, FF)
    pkg.act_quant(x.at, act=act, gated=gated, out=codes.at, scale_out=scale.at[0])
    xd = x.at.double()
    v = ref.act64(xd[:, :width], act)
    ref.check_quant(v * xd[:, width:] if gated else v, codes.at, scale.at[0], 2.0 ** -19)
    for s in (x, codes, scale):
        s.check()


@pytest.mark.parametrize("seed", range(120))
def test_linear(pkg, seed):
    rng = random.Random(2000 + seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n, k = _size(rng, 3000), _size(rng, 9000), _size(rng, 3000)
    q, out_type = rng.choice([I8, E4]), rng.choice([BF, HF, FF])
    act = rng.choice(["none", "none", "relu", "silu", "gelu"])
    make = lambda r: _Slice(rng, r, k, q).put(   # noqa: E731
        (torch.randn(r, k, generator=g, device="cuda") * 40).clamp(-127, 127).to(q))
    x, w = make(m), make(n)
    vec = lambda c, f: _Slice(rng, 1, c, FF).put(   # noqa: E731
        torch.rand(1, c, generator=g, device="cuda") * f + 0.001)
    sx = vec(m, 0.02) if rng.random() < 0.8 else None
    sw = vec(n, 0.02 / math.sqrt(k))
    bias = vec(n, 1.0) if rng.random() < 0.5 else None
    out = _Slice(rng, m, n, out_type)
    row = lambda s: None if s is None else s.at[0]   # noqa: E731
    pkg.linear_w8a8(x.at, w.at, row(sx), row(sw), bias=row(bias), act=act, out=out.at)
    for s in (x, w, sx, sw, bias, out):
        if s is not None:
            s.check()
    y = ref.linear64(x.at, w.at, row(sx), row(sw), row(bias), act)[0]
    if out_type != HF or float(y.abs().max()) < 6e4:   # beyond: infinities in fp16
        ref.check_linear(out.at, x.at, w.at, row(sx), row(sw), row(bias), act)
