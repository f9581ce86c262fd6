"""The token operators (rms_norm_quant, act_quant, linear_w8a8) against their
definitions in 64 bits: types, odd sizes, strides, alignment, empty and
non-finite rows, in-place residuals, streams and graphs."""
import math

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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=FF):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _codes(g, rows, width, q):
    if q == I8:
        return torch.randint(-128, 128, (rows, width), generator=g, device="cuda").to(I8)
    return (torch.randn(rows, width, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4)


def _unaligned(t, pad, off):
    """The same values as a row-strided view that starts `off` elements in."""
    rows, width = t.shape
    flat = torch.zeros(rows * (width + pad) + off, dtype=t.dtype, device=t.device)
    v = flat[off:].view(rows, width + pad)[:, :width]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ rms_norm_quant

NORM_WIDTHS = [1, 2, 7, 8, 31, 64, 100, 127, 256, 641, 768, 1000, 1001, 1024, 1280, 2048, 2056,
               4096, 5120, 8191, 8192, 16384, 20001, 32768, 40000]


def _norm_case(pkg, tokens, width, x_type, res_type, w_type, q, seed=0, strided=False):
    g = _gen(1000 * seed + width)
    x = _randn(g, tokens, width, dtype=x_type)
    x[:, width // 2] *= 9
    res = None if res_type is None else _randn(g, tokens, width, dtype=res_type)
    w = None if w_type is None else (1 + 0.3 * _randn(g, width)).to(w_type)
    if tokens > 2:
        x[1] = 0
        if res is not None:
            res[1] = 0
    if strided:
        x = _unaligned(x, 3, 1)
        res = None if res is None else _unaligned(res, 5, 1)
    codes, scale, res_out = pkg.rms_norm_quant(x, w, 1e-6, residual=res, qdtype=q)
    h, v = ref.norm64(x, w, 1e-6, res)
    assert codes.dtype == q
    ref.check_quant(v, codes, scale, (width / 32 + 64) * 2.0 ** -24)
    if res is None:
        assert res_out is None
    else:
        assert res_out.dtype == res_type
        ref.check_rounded(res_out, h, 2.0 ** -24 * h.abs())
    if tokens > 2:
        assert float(scale[1]) == 1.0 and not codes[1].view(torch.uint8).any()


@pytest.mark.parametrize("width", NORM_WIDTHS)
@pytest.mark.parametrize("tokens,q", [(1, I8), (5, E4)])
def test_norm_widths(pkg, width, tokens, q):
    _norm_case(pkg, tokens, width, BF, BF, BF, q)


@pytest.mark.parametrize("x_type,res_type,w_type", [
    (BF, None, None), (BF, None, FF), (BF, FF, BF), (BF, FF, FF), (BF, BF, FF), (HF, HF, HF),
    (HF, FF, HF), (HF, None, FF), (FF, FF, FF), (FF, None, None)])
@pytest.mark.parametrize("width", [640, 999, 4096, 12288])
@pytest.mark.parametrize("q", [I8, E4])
def test_norm_types(pkg, width, x_type, res_type, w_type, q):
    _norm_case(pkg, 9, width, x_type, res_type, w_type, q, seed=3)


@pytest.mark.parametrize("width", [8, 33, 1280, 2048, 8192, 33000])
@pytest.mark.parametrize("x_type", [BF, FF])
def test_norm_strided_rows(pkg, width, x_type):
    _norm_case(pkg, 6, width, x_type, x_type, x_type, I8, seed=5, strided=True)


@pytest.mark.parametrize("tokens", [1, 2, 151, 153, 1217, 5000])
@pytest.mark.parametrize("width", [640, 1280, 2048])
def test_norm_token_counts(pkg, tokens, width):
    _norm_case(pkg, tokens, width, BF, BF, BF, E4, seed=7)


@pytest.mark.parametrize("width", [96, 1280, 2048, 5000, 9000, 36000])
def test_norm_residual_in_place(pkg, width):
    g = _gen(width)
    x, res = _randn(g, 300, width, dtype=BF), _randn(g, 300, width, dtype=BF)
    want = pkg.rms_norm_quant(x, None, residual=res)
    again = res.clone()
    got = pkg.rms_norm_quant(x, None, residual=again, residual_out=again)
    assert got[2] is again
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_norm_leading_dims_and_given_outputs(pkg):
    g = _gen(1)
    x = _randn(g, 2, 3, 5, 640, dtype=BF)
    codes, scale, _ = pkg.rms_norm_quant(x)
    assert codes.shape == x.shape and scale.shape == (2, 3, 5)
    wide = torch.zeros(30, 700, dtype=I8, device="cuda")
    s2 = torch.empty(30, device="cuda")
    c2, _, _ = pkg.rms_norm_quant(x.view(30, 640), out=wide[:, 10:650], scale_out=s2)
    assert torch.equal(c2, codes.view(30, 640)) and torch.equal(s2, scale.view(30))
    assert not wide[:, :10].any() and not wide[:, 650:].any()   # nothing beside the rows


@pytest.mark.parametrize("width", [40, 1280, 2048, 9000, 36000])
@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_norm_not_finite_rows(pkg, width, q, what):
    """A NaN or infinity spoils its own row only, and visibly."""
    g = _gen(2)
    x = _randn(g, 4, width, dtype=BF)
    clean = pkg.rms_norm_quant(x, qdtype=q)
    bad = x.clone()
    bad[2, width - 1] = what
    codes, scale, _ = pkg.rms_norm_quant(bad, qdtype=q)
    assert math.isnan(float(scale[2])) and not codes[2].view(torch.uint8).any()
    for r in (0, 1, 3):
        assert float(scale[r]) == float(clean[1][r])
        assert torch.equal(codes[r].view(torch.uint8), clean[0][r].view(torch.uint8))


@pytest.mark.parametrize("width", [640, 2048, 40000])
def test_norm_mean_square_beyond_fp32(pkg, width):
    """Finite rows whose mean square overflows are marked like rows that are not
    finite; those whose sum of squares alone would are not."""
    x = torch.full((3, width), 1e15, device="cuda")
    x[1] = 3e19
    x[2] = 1.5e19
    codes, scale, _ = pkg.rms_norm_quant(x)
    assert math.isnan(float(scale[1])) and not codes[1].any()
    for r in (0, 2):
        assert abs(float(scale[r]) * 127 - 1) < 1e-5 and (codes[r] == 127).all()


@pytest.mark.parametrize("mag", [1e-30, 1e-20, 1e18])
def test_norm_magnitudes(pkg, mag):
    """eps decides below, the squares stay within fp32 above."""
    x = _randn(_gen(3), 3, 1280) * mag
    codes, scale, _ = pkg.rms_norm_quant(x, eps=1e-6)
    _, v = ref.norm64(x, None, 1e-6, None)
    ref.check_quant(v, codes, scale, (1280 / 32 + 64) * 2.0 ** -24)


def test_quant_of_subnormal_rows(pkg):
    """Rows far below the codes' reach of a normal scale: finite, within a step."""
    x = torch.zeros(2, 64, device="cuda")
    x[0, 3] = 1e-42
    x[1, 5] = 1e-37
    codes, scale = pkg.act_quant(x)
    assert torch.isfinite(scale).all() and (scale > 0).all()
    back = codes.double() * scale.double()[:, None]
    assert ((back - x.double()).abs() <= 0.5 * scale.double()[:, None] * (1 + 1e-6)).all()


# ------------------------------------------------------------------ act_quant

@pytest.mark.parametrize("width", [1, 3, 8, 100, 640, 1023, 2048, 4096, 5120, 8192, 11008, 16384,
                                   28672, 33001, 70000])
@pytest.mark.parametrize("act,gated", [("silu", True), ("gelu", False), ("none", False),
                                       ("gelu", True), ("relu", False), ("none", True)])
def test_act_widths(pkg, width, act, gated):
    g = _gen(width)
    for tokens, x_type, q in ((1, BF, I8), (7, BF, E4), (3, HF, I8), (4, FF, E4)):
        x = _randn(g, tokens, 2 * width if gated else width, dtype=x_type) * 2
        x[:, 0] = x[:, 0].abs() + 0.5
        codes, scale = pkg.act_quant(x, act=act, gated=gated, qdtype=q)
        xd = x.double()
        v = ref.act64(xd[:, :width], act)
        if gated:
            v = v * xd[:, width:]
        ref.check_quant(v, codes, scale, 2.0 ** -19)


@pytest.mark.parametrize("tokens", [1, 150, 1300, 6000])
def test_act_token_counts_and_strides(pkg, tokens):
    g = _gen(tokens)
    x = _unaligned(_randn(g, tokens, 2 * 1000, dtype=BF), 7, 3)
    codes, scale = pkg.act_quant(x, act="silu", gated=True, qdtype=E4)
    xd = x.double()
    ref.check_quant(ref.act64(xd[:, :1000], "silu") * xd[:, 1000:], codes, scale, 2.0 ** -19)


@pytest.mark.parametrize("width", [24, 4096, 40000])
@pytest.mark.parametrize("act,gated", [("silu", True), ("gelu", False), ("none", False),
                                       ("relu", False)])
def test_act_not_finite_rows(pkg, width, act, gated):
    x = _randn(_gen(9), 3, 2 * width if gated else width, dtype=BF)
    clean = pkg.act_quant(x, act=act, gated=gated)
    x[1, width // 2] = math.nan
    x[2, width // 3] = math.inf
    codes, scale = pkg.act_quant(x, act=act, gated=gated)
    assert torch.isnan(scale[1:]).all() and not codes[1:].any()
    assert float(scale[0]) == float(clean[1][0]) and torch.equal(codes[0], clean[0][0])


def test_zero_rows_and_zero_tokens(pkg):
    codes, scale = pkg.act_quant(torch.zeros(3, 50, device="cuda", dtype=BF), qdtype=E4)
    assert (scale == 1).all() and not codes.view(torch.uint8).any()
    codes, scale = pkg.act_quant(torch.zeros(0, 50, device="cuda"))
    assert codes.shape == (0, 50) and scale.shape == (0,)
    codes, scale, res = pkg.rms_norm_quant(torch.zeros(0, 4, 50, device="cuda"),
                                           residual=torch.zeros(0, 4, 50, device="cuda"))
    assert codes.shape == (0, 4, 50) and scale.shape == (0, 4) and res.shape == (0, 4, 50)


# ------------------------------------------------------------------ linear_w8a8

def _linear_case(pkg, m, n, k, q, out_dtype=BF, bias=False, act="none", seed=0, x=None, w=None):
    g = _gen(7 * m + 31 * n + k + seed)
    x = _codes(g, m, k, q) if x is None else x
    w = _codes(g, n, k, q) if w is None else w
    sx = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.001
    sw = (torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001) / math.sqrt(k)
    b = _randn(g, n) if bias else None
    got = pkg.linear_w8a8(x, w, sx, sw, bias=b, act=act, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    ref.check_linear(got, x, w, sx, sw, b, act)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("m", [1, 2, 3, 8, 9, 16, 17, 31, 32, 33, 48, 64, 65, 100, 127, 128, 129,
                               200, 256, 257, 400, 640])
def test_linear_token_counts(pkg, m, q):
    _linear_case(pkg, m, 384, 512, q)
    _linear_case(pkg, m, 1000, 272, q, out_dtype=FF, bias=True)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 32, 48, 63, 64, 65, 112, 127, 128, 129, 144,
                               255, 256, 400, 1000, 1024, 1283, 2064, 4096, 8192])
@pytest.mark.parametrize("m", [1, 5, 70, 300])
def test_linear_widths(pkg, k, m, q):
    _linear_case(pkg, m, 200, k, q)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 31, 64, 100, 127, 128, 129, 255, 256, 257, 500,
                               1003, 2304])
@pytest.mark.parametrize("m", [1, 20, 333])
def test_linear_outputs(pkg, n, m, q):
    _linear_case(pkg, m, n, 320, q, out_dtype=FF, bias=True)
    _linear_case(pkg, m, n, 320, q, out_dtype=BF)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("m,n,k", [(3, 700, 1152), (2500, 1280, 640), (9500, 1280, 1280),
                                   (4100, 2056, 2048), (40000, 520, 272)])
@pytest.mark.parametrize("out_dtype,bias,act", [(BF, True, "gelu"), (HF, True, "relu"),
                                                (FF, True, "silu"), (FF, False, "gelu"),
                                                (BF, False, "silu")])
def test_linear_epilogues(pkg, m, n, k, q, out_dtype, bias, act):
    _linear_case(pkg, m, n, k, q, out_dtype, bias, act)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("m", [1, 4, 30, 150, 700])
@pytest.mark.parametrize("px,ox,pw,ow", [(3, 0, 0, 0), (0, 1, 0, 0), (0, 0, 5, 2), (7, 3, 1, 9),
                                         (16, 16, 32, 0)])
def test_linear_strided_and_unaligned_rows(pkg, m, q, px, ox, pw, ow):
    g = _gen(m + px + ow)
    k, n = 656, 330
    x = _unaligned(_codes(g, m, k, q).view(torch.uint8), px, ox).view(q)
    w = _unaligned(_codes(g, n, k, q).view(torch.uint8), pw, ow).view(q)
    _linear_case(pkg, m, n, k, q, x=x, w=w)


@pytest.mark.parametrize("m", [1, 6, 40, 129, 600])
@pytest.mark.parametrize("out_dtype", [BF, FF])
def test_linear_writes_only_its_rows(pkg, m, out_dtype):
    """A row-strided output: the columns beside it and the row after it stay."""
    g = _gen(m)
    x, w = _codes(g, m, 160, I8), _codes(g, 77, 160, I8)
    buf = torch.full((m + 1, 100), 3.0, dtype=out_dtype, device="cuda")
    got = pkg.linear_w8a8(x, w, out=buf[:m, 5:82])
    assert torch.equal(got, pkg.linear_w8a8(x, w, out_dtype=out_dtype))
    assert (buf[:, :5] == 3).all() and (buf[:, 82:] == 3).all() and (buf[m] == 3).all()


@pytest.mark.parametrize("m", [1, 3, 16, 64, 200, 512, 3000])
@pytest.mark.parametrize("k", [16, 1024])
def test_linear_int8_is_exact(pkg, m, k):
    """Up to 1024 products the fp32 sums hold every int8 result exactly, at the
    type's limits too."""
    g = _gen(m + k)
    x, w = _codes(g, m, k, I8), _codes(g, 260, k, I8)
    x[0], w[0], w[1] = -128, -128, 127
    got = pkg.linear_w8a8(x, w, out_dtype=FF)
    assert torch.equal(got.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("k", [8192, 50000])
def test_linear_int8_long_sums(pkg, m, k):
    """Every product at the limit and of one sign: beyond 2^24 the sum rounds."""
    x = torch.full((m, k), 127, dtype=I8, device="cuda")
    w = torch.full((150, k), 127, dtype=I8, device="cuda")
    got = pkg.linear_w8a8(x, w, out_dtype=FF)
    ref.check_linear(got, x, w)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("m", [5, 150, 700])
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_linear_not_finite_scales(pkg, m, q, act):
    """A row of scale NaN is NaN throughout (relu too), the others as before."""
    g = _gen(m)
    x, w = _codes(g, m, 256, q), _codes(g, 140, 256, q)
    sx, sw = torch.full((m,), 0.01, device="cuda"), torch.full((140,), 0.01, device="cuda")
    clean = pkg.linear_w8a8(x, w, sx, sw, act=act)
    sx[2] = math.nan
    got = pkg.linear_w8a8(x, w, sx, sw, act=act)
    assert torch.isnan(got[2]).all()
    keep = torch.arange(m, device="cuda") != 2
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("m", [4, 100, 600])
def test_linear_e4m3_nan_codes(pkg, m):
    g = _gen(m)
    x, w = _codes(g, m, 192, E4), _codes(g, 130, 192, E4)
    clean = pkg.linear_w8a8(x, w)
    x.view(torch.uint8)[1, 191] = 0x7F
    w.view(torch.uint8)[129, 0] = 0xFF
    got = pkg.linear_w8a8(x, w)
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, 129]).all()
    keep = torch.arange(m, device="cuda") != 1
    assert torch.equal(got[keep][:, :129], clean[keep][:, :129])


def test_linear_empty(pkg):
    x, w = torch.zeros(0, 32, dtype=I8, device="cuda"), torch.zeros(5, 32, dtype=I8, device="cuda")
    assert pkg.linear_w8a8(x, w).shape == (0, 5)
    assert pkg.linear_w8a8(w, x).shape == (5, 0)


@pytest.mark.parametrize("q", [I8, E4])
def test_linear_same_bits_every_time(pkg, q):
    for m, n, k in ((4, 2048, 8192), (100, 1280, 5120), (600, 640, 4096), (3000, 2048, 1024)):
        g = _gen(m)
        x, w = _codes(g, m, k, q), _codes(g, n, k, q)
        first = pkg.linear_w8a8(x, w, out_dtype=FF)
        for _ in range(3):
            assert torch.equal(first, pkg.linear_w8a8(x, w, out_dtype=FF))


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("m", [520, 700, 1024])
def test_linear_waiting_for_its_weights(pkg, m, q):
    """Few token tiles and weights larger than the L2 cache: the products wait for
    the weights while the tokens run ahead; back to back, and the same bits
    each time."""
    g = _gen(m)
    n = k = 8192
    x, w = _codes(g, m, k, q), _codes(g, n, k, q)
    outs = [pkg.linear_w8a8(x, w, out_dtype=FF) for _ in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    ref.check_linear(outs[0][:, :512], x, w[:512])
    ref.check_linear(outs[0][:, -300:], x, w[-300:])


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("wx,ww", [(1, 0), (0, 1), (1, 1)])
def test_linear_workspace_follows_each_operand(pkg, q, wx, ww):
    """The workspace's size depends on either operand's alignment."""
    g = _gen(5)
    x, w = _codes(g, 40, 656, q), _codes(g, 100, 656, q)
    for ox, ow in ((wx, 0), (0, ww), (wx, ww), (0, 0)):
        a = _unaligned(x.view(torch.uint8), 0, ox).view(q)
        b = _unaligned(w.view(torch.uint8), 0, ow).view(q)
        _linear_case(pkg, 40, 100, 656, q, x=a, w=b)


@pytest.mark.parametrize("q", [I8, E4])
def test_linear_past_32_bits(pkg, q):
    """An output of more than 2^32 bytes and 2^31 elements, and token rows that
    lie more than 2^32 bytes apart: sampled rows."""
    g = _gen(11)
    m, n, k = 300000, 8192, 64
    x, w = _codes(g, m, k, q), _codes(g, n, k, q)
    got = pkg.linear_w8a8(x, w)
    rows = torch.tensor([0, 1, 127, 128, 131071, 131072, 262143, 262144, 262145, m - 129, m - 1],
                        device="cuda")
    ref.check_linear(got[rows], x.view(torch.uint8)[rows].view(q), w)
    del got
    wide = torch.zeros(5, 1 << 30, dtype=torch.uint8, device="cuda").view(q)[:, :k]
    wide.copy_(x[:5])
    ref.check_linear(pkg.linear_w8a8(wide, w), x[:5], w)


def test_norm_and_act_past_32_bits(pkg):
    g = _gen(12)
    rows, width = 1200000, 2048          # 2.46e9 elements
    x = torch.empty(rows, width, dtype=BF, device="cuda")
    x.normal_(generator=g)
    codes, scale, _ = pkg.rms_norm_quant(x, qdtype=E4)
    at = torch.tensor([0, 1, 1048575, 1048576, 1048577, rows - 1], device="cuda")
    pick = lambda t: t[at]                                                   # noqa: E731
    _, v = ref.norm64(pick(x), None, 1e-6, None)
    ref.check_quant(v, pick(codes.view(torch.uint8)).view(E4), pick(scale), 128 * 2.0 ** -24)
    codes, scale = pkg.act_quant(x, act="silu", gated=True, out=codes[:, :1024])
    xd = pick(x).double()
    ref.check_quant(ref.act64(xd[:, :1024], "silu") * xd[:, 1024:],
                    codes.view(torch.uint8)[at].view(E4), pick(scale), 2.0 ** -19)


# ------------------------------------------------------------------ together

def _mlp(pkg, x, res, p, q, stream=None):
    a, sa, res = pkg.rms_norm_quant(x, p["gain"], residual=res, qdtype=q, stream=stream)
    h = pkg.linear_w8a8(a, p["up"], sa, p["sup"], stream=stream)
    b, sb = pkg.act_quant(h, act="silu", gated=True, qdtype=q, stream=stream)
    return pkg.linear_w8a8(b, p["down"], sb, p["sdown"], stream=stream), res


def _mlp_params(pkg, g, width, inner, q):
    up, sup = pkg.act_quant(_randn(g, 2 * inner, width) / math.sqrt(width), qdtype=q)
    down, sdown = pkg.act_quant(_randn(g, width, inner) / math.sqrt(inner), qdtype=q)
    return dict(gain=(1 + 0.1 * _randn(g, width)).to(BF), up=up, sup=sup, down=down, sdown=sdown)


@pytest.mark.parametrize("q", [I8, E4])
@pytest.mark.parametrize("tokens", [1, 50, 400, 4000])
def test_block_follows_the_unquantised_one(pkg, tokens, q):
    """The chain against the same block without quantisation, in 64 bits: each
    8-bit rounding is at most amax/254 (int8) or 2^-4 relative (e4m3), about 1%
    (2.5%) rms per operand of a product, uncorrelated: 10% bounds four of them."""
    g = _gen(tokens)
    width, inner = 640, 1280
    wu, wd = _randn(g, 2 * inner, width) / math.sqrt(width), _randn(g, width, inner) / math.sqrt(inner)
    up, sup = pkg.act_quant(wu, qdtype=q)
    down, sdown = pkg.act_quant(wd, qdtype=q)
    p = dict(gain=(1 + 0.1 * _randn(g, width)).to(BF), up=up, sup=sup, down=down, sdown=sdown)
    x, res = _randn(g, tokens, width, dtype=BF), _randn(g, tokens, width, dtype=BF)
    y, _ = _mlp(pkg, x, res, p, q)
    _, v = ref.norm64(x, p["gain"], 1e-6, res)
    u = v @ wu.double().t()
    want = (ref.act64(u[:, :inner], "silu") * u[:, inner:]) @ wd.double().t()
    assert float((y.double() - want).norm() / want.norm()) < 0.10


@pytest.mark.parametrize("q", [I8, E4])
def test_given_stream_owns_what_it_allocates(pkg, q):
    """Calls on a given stream whose tensors come from the current stream's pool:
    what is dropped between the calls (workspaces, codes) is not handed to the
    current stream's work while the given stream still reads it."""
    g = _gen(21)
    side = torch.cuda.Stream()
    x, w = _codes(g, 1030, 2051, q), _codes(g, 1500, 2051, q)   # staged operands
    want = pkg.linear_w8a8(x, w)
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        got.append(pkg.linear_w8a8(x, w, stream=side))
        junk = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")   # the pool's next user
        del junk
    side.synchronize()
    for y in got:
        assert torch.equal(y, want)


@pytest.mark.parametrize("tokens", [1, 37, 700])
def test_block_on_another_stream_and_in_a_graph(pkg, tokens):
    """Everything runs on the stream it is given, and a captured block replayed
    on new inputs gives what the calls give."""
    g = _gen(tokens)
    p = _mlp_params(pkg, g, 640, 1024, I8)
    xs = [_randn(g, tokens, 640, dtype=BF) for _ in range(3)]
    rs = [_randn(g, tokens, 640, dtype=BF) for _ in range(3)]
    want = [_mlp(pkg, x, r, p, I8) for x, r in zip(xs, rs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [_mlp(pkg, x, r, p, I8) for x, r in zip(xs, rs)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x, r = xs[0].clone(), rs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ro = _mlp(pkg, x, r, p, I8)
    for i in range(3):
        x.copy_(xs[i])
        r.copy_(rs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(ro, want[i][1])


# ------------------------------------------------------------------ refusals

def test_refusals(pkg):
    x = torch.zeros(4, 32, device="cuda", dtype=BF)
    c = torch.zeros(4, 32, device="cuda", dtype=I8)
    s = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        pkg.rms_norm_quant(x.double())
    with pytest.raises(TypeError):
        pkg.rms_norm_quant(x, qdtype=torch.uint8)
    with pytest.raises(TypeError):
        pkg.rms_norm_quant(x, torch.ones(32, device="cuda", dtype=HF))
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x, torch.ones(31, device="cuda"))
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x.t())
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x, residual=x[:2])
    with pytest.raises(pkg.ConvError):
        pkg.rms_norm_quant(x, residual=x.half())
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x, residual_out=x)
    with pytest.raises(pkg.ConvError):
        pkg.rms_norm_quant(x, eps=-1.0)
    with pytest.raises(pkg.ConvError):
        pkg.rms_norm_quant(x, eps=math.nan)
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x, out=c[:, :30])
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x, scale_out=s[:3])
    with pytest.raises(TypeError):
        pkg.rms_norm_quant(x, scale_out=s.to(BF))
    with pytest.raises(ValueError):
        pkg.rms_norm_quant(x.cpu())
    with pytest.raises(pkg.ConvError):
        pkg.rms_norm_quant(torch.zeros(3, 0, device="cuda"))
    with pytest.raises(ValueError):
        pkg.act_quant(x, act="tanh")
    with pytest.raises(ValueError):
        pkg.act_quant(x[:, :31], gated=True)
    with pytest.raises(pkg.ConvError):
        pkg.act_quant(x[:1].expand(4, 32))
    with pytest.raises(TypeError):
        pkg.linear_w8a8(c, c.view(torch.uint8).view(E4))
    with pytest.raises(TypeError):
        pkg.linear_w8a8(x, x)
    with pytest.raises(ValueError):
        pkg.linear_w8a8(c, c[:, :16])
    with pytest.raises(ValueError):
        pkg.linear_w8a8(c, c, scale_x=s[:3])
    with pytest.raises(TypeError):
        pkg.linear_w8a8(c, c, scale_x=s.half())
    with pytest.raises(ValueError):
        pkg.linear_w8a8(c, c, bias=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        pkg.linear_w8a8(c, c, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        pkg.linear_w8a8(c, c, out=torch.zeros(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        pkg.linear_w8a8(c, c, act="swish")


# ------------------------------------------------------------------ the example

@pytest.mark.parametrize("dtype", ["int8", "e4m3"])
@pytest.mark.parametrize("images", [1, 4])
def test_patch_mlp_example(pkg, dtype, images):
    """The patch embedding and two blocks in a graph: each block adds at most the
    10% of test_block_follows_the_unquantised_one to a stream that keeps its
    unquantised part."""
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "patch_mlp_w8a8", os.path.join(root, "examples", "patch_mlp_w8a8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    error, ms = mod.run(images=images, blocks=2, dtype=dtype, width=640, inner=1280)
    assert error < 0.10 and ms > 0
