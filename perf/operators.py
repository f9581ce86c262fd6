"""Cases of the 8-bit token operators that follow a convolutional patch embedding:
the root-mean-square norm with the residual's addition and an 8-bit output, the
(gated) activation with an 8-bit output, and the matrix product of 8-bit operands
with a scale per token and per output channel.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, by the library's
operators.  8-bit results come back as the values they stand for: e4m3 codes as
float8 tensors beside their row scales, int8 codes multiplied by their row scale
in bf16, beside the scales.
"""
import math

import torch

own = False

EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}
FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token through the first norm of a block: latency only
        dict(name="norm_one_token", op="norm", t=1, h=2048, x="bf16", res="bf16", q="int8"),
        # a ragged batch of tokens with an odd width in fp16, no residual yet
        dict(name="norm_ragged", op="norm", t=777, h=1001, x="fp16", res="none", q="int8"),
        # the tokens of the 9500-image patch embedding (1280 wide), 32-bit residual stream
        dict(name="norm_patches", op="norm", t=9500, h=1280, x="bf16", res="fp32", q="e4m3"),
        # the positions of the 15 x 120 x 120 video grid, 2048 channels
        dict(name="norm_video", op="norm", t=216000, h=2048, x="bf16", res="bf16", q="e4m3"),
        # one token between the two products of a gated block
        dict(name="act_one_token", op="act", t=1, f=8192, x="bf16", act="silu", gated=True,
             q="int8"),
        # the 16384 tokens of 64 images in 14 x 14 patches, gated, four times 1024 wide
        dict(name="act_gated_patches", op="act", t=16384, f=4096, x="bf16", act="silu",
             gated=True, q="e4m3"),
        # the 9500 patch tokens after an ordinary GELU product, four times 1280 wide
        dict(name="act_gelu_patches", op="act", t=9500, f=5120, x="bf16", act="gelu",
             gated=False, q="int8"),
        # one token through a block's first product: the weights are all there is to read
        dict(name="linear_one_token", op="linear", m=1, n=8192, k=2048, q="int8", bias=False,
             act="none", out="bf16"),
        # a batch of 16 single tokens through the product back
        dict(name="linear_16_tokens", op="linear", m=16, n=2048, k=8192, q="e4m3", bias=False,
             act="none", out="bf16"),
        # odd in every size: rows that are not 16-byte aligned, 32-bit logits with a bias
        dict(name="linear_ragged", op="linear", m=333, n=1003, k=1283, q="int8", bias=True,
             act="none", out="fp32"),
        # the 16384 patch tokens into gate and value halves at once
        dict(name="linear_gated_patches", op="linear", m=16384, n=8192, k=1024, q="e4m3",
             bias=False, act="none", out="bf16"),
        # every position of the video grid through a square product
        dict(name="linear_video", op="linear", m=216000, n=2048, k=2048, q="int8", bias=True,
             act="none", out="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm; as often odd as it falls,
    or rounded to a multiple of 128, as widths mostly are."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 128:
        v = v // 128 * 128
    return 2944 if v == 3072 else max(lo, min(hi, v))


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest listed one."""
    op = rng.choice(["norm", "act", "linear", "linear"])
    q = rng.choice(["int8", "e4m3"])
    if op == "norm":
        h = _spread(rng, 64, 8192)
        return dict(op=op, t=min(_spread(rng, 1, 216000), 216000 * 2048 // h), h=h,
                    x=rng.choice(["bf16", "bf16", "fp16"]),
                    res=rng.choice(["none", "same", "same", "fp32"]), q=q)
    if op == "act":
        f = _spread(rng, 64, 28000)
        gated = rng.random() < 0.5
        return dict(op=op, t=min(_spread(rng, 1, 16384), 16384 * 8192 // (2 * f)), f=f,
                    x=rng.choice(["bf16", "bf16", "fp16"]),
                    act=rng.choice(["silu", "gelu", "none"]), gated=gated, q=q)
    n, k = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
    m = min(_spread(rng, 1, 216000), 216000 * 2048 * 2048 // (n * k), 216000 * 2048 // max(n, k))
    return dict(op=op, m=m, n=n, k=k, q=q, bias=rng.random() < 0.5,
                act=rng.choice(["none", "none", "gelu", "silu"]),
                out=rng.choice(["bf16", "bf16", "fp32"]))


def _tokens(g, t, h, dtype):
    """Activations: N(0, 1), a few channels far larger (as hidden states have), and the
    last token of a batch a padded one, all zeros."""
    x = torch.randn(t, h, generator=g, device="cuda")
    loud = torch.randint(0, h, (max(1, h // 256),), generator=g, device="cuda")
    x[:, loud] *= 12.0
    if t > 1:
        x[-1] = 0.0
    return x.to(dtype)


def _codes(v, q):
    """Rows of v as 8-bit codes with a scale each."""
    s = v.abs().amax(dim=1) / QMAX[q]
    s = torch.where(s > 0, s, torch.ones_like(s))
    c = v / s[:, None]
    c = torch.round(c) if q == "int8" else c.clamp(-448.0, 448.0)
    return c.to(CODE[q]), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        res = case["x"] if case["res"] == "same" else case["res"]
        s["data"] = _tokens(g, t, h, FLOAT[case["x"]])
        s["residual"] = None if res == "none" else _tokens(g, t, h, FLOAT[res])
        gain = 1.0 + 0.2 * torch.randn(h, generator=g, device="cuda")
        s["weight"] = gain.to(FLOAT[case["x"]])
        s["res_out"] = None if res == "none" else torch.empty_like(s["residual"])
        s["rows"], s["width"] = t, h
    elif case["op"] == "act":
        t, f = case["t"], case["f"]
        s["data"] = _tokens(g, t, 2 * f if case["gated"] else f, FLOAT[case["x"]])
        s["rows"], s["width"] = t, f
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["xq"], s["sx"] = _codes(_tokens(g, m, k, torch.float32), case["q"])
        s["wq"], s["sw"] = _codes(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k),
                                  case["q"])
        s["bias_v"] = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["out_v"] = torch.empty(m, n, dtype=FLOAT[case["out"]], device="cuda")
    if case["op"] != "linear":
        s["codes"] = torch.empty(s["rows"], s["width"], dtype=CODE[case["q"]], device="cuda")
        s["scale"] = torch.empty(s["rows"], dtype=torch.float32, device="cuda")
        s["values"] = torch.empty(s["rows"] if case["q"] == "int8" else 0, s["width"],
                                  dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ the operators' own calls

def _run_own(s):
    import implicit_gemm_convolution_conv3d_gb300 as c3d
    if s["op"] == "linear":
        return {"out": c3d.linear_w8a8(s["xq"], s["wq"], s["sx"], s["sw"], bias=s["bias_v"],
                                       act=s["act"], out=s["out_v"])}
    out = {}
    if s["op"] == "norm":
        codes, scale, res = c3d.rms_norm_quant(
            s["data"], s["weight"], EPS, residual=s["residual"], out=s["codes"],
            scale_out=s["scale"], residual_out=s["res_out"])
        if res is not None:
            out["residual"] = res
    else:
        codes, scale = c3d.act_quant(s["data"], act=s["act"], gated=s["gated"], out=s["codes"],
                                     scale_out=s["scale"])
    out["scale"] = scale
    if s["q"] == "int8":
        out["values"] = torch.mul(codes, scale[:, None], out=s["values"])
    else:
        out["codes"] = codes
    return out


# ------------------------------------------------------------------ their plain form

def _plain_act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _plain_quant(v, q, out):
    amax = v.abs().amax(dim=1)
    scale = torch.where(amax > 0, amax / QMAX[q], torch.ones_like(amax))
    c = v / scale[:, None]
    out["scale"] = scale
    if q == "int8":
        out["values"] = (torch.round(c) * scale[:, None]).to(torch.bfloat16)
    else:
        out["codes"] = c.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return out


def _run_plain(s):
    if s["op"] == "linear":
        y = torch.matmul(s["xq"].float(), s["wq"].float().t())
        y = y * s["sx"][:, None] * s["sw"]
        if s["bias_v"] is not None:
            y = y + s["bias_v"]
        return {"out": _plain_act(y, s["act"]).to(FLOAT[s["out"]])}
    out = {}
    if s["op"] == "norm":
        h = s["data"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
            out["residual"] = h.to(s["residual"].dtype)
        v = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    else:
        x = s["data"].float()
        f = s["width"]
        v = _plain_act(x[:, :f], s["act"])
        if s["gated"]:
            v = v * x[:, f:]
    return _plain_quant(v, s["q"], out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        b = BYTES[case["x"]]
        r = 0 if case["res"] == "none" else 2 * BYTES.get(case["res"], b)
        return {"bytes": t * h * (b + r + 1) + h * b + 4 * t, "flops": 8 * t * h}
    if case["op"] == "act":
        t, f = case["t"], case["f"]
        return {"bytes": t * f * (BYTES[case["x"]] * (2 if case["gated"] else 1) + 1) + 4 * t,
                "flops": 8 * t * f}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k + n * k + m * n * BYTES[case["out"]] + 4 * (m + n)
            + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definition, in 64 bits

def _e4m3_values(c):
    """The nearest e4m3 value of each element (ties to the even significand)."""
    _, e = torch.frexp(c)
    step = torch.ldexp(torch.ones_like(c), (e - 1).clamp(min=-6) - 3)
    return (torch.round(c / step) * step).clamp(-448.0, 448.0)


def _activation(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = torch.einsum("mk,nk->mn", s["xq"].double(), s["wq"].double())
        y *= torch.outer(s["sx"].double(), s["sw"].double())
        if s["bias_v"] is not None:
            y += s["bias_v"].double()
        return {"out": _activation(y, case["act"])}
    out = {}
    x = s["data"].double()
    if case["op"] == "norm":
        if s["residual"] is not None:
            x = x + s["residual"].double()
            out["residual"] = x
        rms = (torch.linalg.vector_norm(x, dim=1) ** 2 / case["h"] + EPS).sqrt()
        v = x / rms[:, None] * s["weight"].double()
    elif case["gated"]:
        a, b = x.chunk(2, dim=1)
        v = _activation(a, case["act"]) * b
    else:
        v = _activation(x, case["act"])
    top = v.abs().max(dim=1).values
    scale = (top / QMAX[case["q"]]).masked_fill(top == 0, 1.0)
    out["scale"] = scale
    c = v / scale[:, None]
    if case["q"] == "int8":
        out["values"] = c.round() * scale[:, None]
    else:
        out["codes"] = _e4m3_values(c)
    return out
