"""Cases of the attention operators on the tokens of a convolutional patch embedding:
rotary positions with several axes, writing keys and values to a paged cache in 8 bits
and reading them back, attention of one new token over such a cache, and attention
within packed documents (images, frames, prompts).

``run`` computes a case either in its plain form (elementary torch operations in
32 bits, rounded once at the end; sequences of unlike lengths are padded to the longest)
or, where ``own`` is true, by the library's operators.  8-bit caches come back as the
values they stand for: e4m3 codes as float8 tensors beside their scales, int8 codes
through the operator that reads them back.
"""
import math
import random

import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16,
         "fp16": torch.float16}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
QMAX = {"int8": 127.0, "e4m3": 448.0}
VIDEO = (15, 120, 120)   # positions of the video grid: 216000


def listed():
    return [
        # the query and key heads of one token far into a stream of frames: latency only
        dict(name="rotary_one_token", op="rotary", t=1, heads=24, d=128, sections="16,24,24",
             ladder="shared", pairs="half", x="bf16", inverse=False, at=100000),
        # the gradient of the rotated heads of every position of the 15 x 120 x 120 video grid
        dict(name="rotary_video_grad", op="rotary", t=216000, heads=32, d=128,
             sections="16,24,24", ladder="axis", pairs="interleaved", x="bf16", inverse=True,
             at=0),
        # one new token of each of 64 sequences into an e4m3 cache
        dict(name="cache_step", op="cache", do="write", b=64, start=5000, new=1, hk=8, d=128,
             page=16, x="bf16", store="e4m3", lens=1),
        # some frames' tokens joined to the ones before, and all of them read back for
        # attention: 16 heads of 80, ragged, int8
        dict(name="cache_frames", op="cache", do="append", b=12, start=9000, new=2049, hk=16,
             d=80, page=64, x="bf16", store="int8", lens=2),
        # a whole video read back from an e4m3 cache
        dict(name="cache_read_video", op="cache", do="read", b=1, start=216000, new=0, hk=8,
             d=128, page=128, x="bf16", store="e4m3", lens=3),
        # one token of one short sequence, an unquantised cache: latency only
        dict(name="paged_one_short", op="paged", b=1, most=333, hq=16, hk=16, d=64, page=16,
             x="bf16", store="bf16", cap=0.0, window=0, prefix=0, slopes=False, lens=4),
        # one token over a whole video's positions
        dict(name="paged_one_long", op="paged", b=1, most=216000, hq=32, hk=8, d=128, page=64,
             x="bf16", store="e4m3", cap=0.0, window=0, prefix=0, slopes=False, lens=5),
        # a ragged batch of single tokens, capped scores, some sequences not begun
        dict(name="paged_ragged", op="paged", b=200, most=8192, hq=32, hk=8, d=128, page=16,
             x="fp16", store="int8", cap=30.0, window=0, prefix=0, slopes=False, lens=6),
        # 64 images of 14 x 14 patches (256 each), 16 heads of 64: each image sees itself
        dict(name="packed_images", op="packed", b=64, least=256, most=256, past=0, hq=16, hk=16,
             d=64, x="bf16", causal=False, cap=0.0, window=0, prefix=0, slopes=False, lens=7),
        # images of their own sizes, 16 heads of 80, scores that fall with the distance
        dict(name="packed_ragged", op="packed", b=24, least=100, most=1403, past=0, hq=16, hk=16,
             d=80, x="fp16", causal=False, cap=0.0, window=0, prefix=0, slopes=True, lens=8),
        # two prompts after what the cache holds of them, capped; an image's tokens lead each
        dict(name="packed_prompt", op="packed", b=2, least=5001, most=7001, past=1100, hq=16,
             hk=4, d=128, x="bf16", causal=True, cap=50.0, window=0, prefix=576, slopes=False,
             lens=9),
        # one frame of 120 x 120 positions, 16 heads of 128
        dict(name="packed_frame", op="packed", b=1, least=14400, most=14400, past=0, hq=16,
             hk=16, d=128, x="bf16", causal=False, cap=0.0, window=0, prefix=0, slopes=False,
             lens=10),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest listed ones."""
    op = rng.choice(["rotary", "cache", "paged", "paged", "packed", "packed"])
    lens = rng.randrange(1 << 30)
    if op == "rotary":
        d, axes = rng.choice([64, 80, 96, 128]), rng.choice([1, 2, 3])
        n = [rng.randint(1, d // 2 // axes) for _ in range(axes)]
        if rng.random() < 0.6:
            n[-1] += d // 2 - sum(n)
        heads = _spread(rng, 1, 48)
        x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return dict(op=op, t=min(_spread(rng, 1, 216000), 216000 * 4096 * 2 // (heads * d * BYTES[x])),
                    heads=heads, d=d, sections=",".join(map(str, n)),
                    ladder=rng.choice(["axis", "shared"]), pairs=rng.choice(["half", "interleaved"]),
                    x=x, inverse=rng.random() < 0.5, at=rng.choice([0, _spread(rng, 1, 1 << 20)]))
    hk = rng.choice([1, 2, 4, 8, 16])
    if op == "cache":
        d = rng.choice([64, 80, 128])
        store = rng.choice(["int8", "e4m3", "e4m3", "bf16"])
        do = rng.choice(["append", "read"] if store == "int8" else ["write", "append", "read"])
        b = _spread(rng, 1, 128)
        room = 216000 * 1024 // (b * hk * d)
        new = 0 if do == "read" else min(_spread(rng, 1, 4096), max(1, room // 2))
        return dict(op=op, do=do, b=b, start=max(0, min(_spread(rng, 1, 216000), room - new)),
                    new=new, hk=hk, d=d, page=rng.choice([16, 16, 32, 40, 64, 128]),
                    x="bf16", store=store, lens=lens)
    g = rng.choice([1, 2, 4, 7, 8])
    hq = min(48, hk * g) // hk * hk
    case = dict(op=op, hq=hq, hk=hk, x=rng.choice(["bf16", "bf16", "fp16"]),
                cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.25, lens=lens,
                window=rng.choice([0, 0, _spread(rng, 1, 4096)]),
                prefix=rng.choice([0, 0, _spread(rng, 1, 1000)]))
    if op == "paged":
        d = rng.choice([64, 80, 128])
        b = _spread(rng, 1, 256)
        store = rng.choice(["int8", "e4m3", case["x"]])
        most = min(_spread(rng, 1, 216000), 200 * 8192 * 1024 // (b * hk * d * BYTES[store]),
                   200 * 8192 * 4096 // (b * hq * d))
        return dict(case, b=b, most=max(1, most), d=d, page=rng.choice([16, 16, 32, 40, 64, 128]),
                    store=store)
    b = _spread(rng, 1, 128)
    most = min(_spread(rng, 16, 14400), int(14400 * math.sqrt(16 / (b * hq))))
    return dict(case, b=b, least=max(1, int(most * rng.choice([1.0, 0.5, 0.1]))), most=most,
                past=rng.choice([0, 0, most // 8]), d=rng.choice([64, 72, 80, 96, 128]),
                causal=rng.random() < 0.5)


# ------------------------------------------------------------------ lengths, by the case alone

def _cache_lens(case):
    """(tokens held before, new tokens) of each sequence."""
    r = random.Random(case["lens"])
    most = case["start"]
    if case["b"] == 1:
        return [most], [case["new"]]
    start = [r.randint(most // 2, most) for _ in range(case["b"])]
    return start, [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(case["b"])]


def _paged_lens(case):
    """Tokens in the cache of each sequence, the new one among them; in larger batches some
    places are empty."""
    r = random.Random(case["lens"])
    if case["b"] == 1:
        return [case["most"]]
    n = [r.randint(1, case["most"]) for _ in range(case["b"])]
    return [0 if case["b"] > 8 and i % 16 == 5 else v for i, v in enumerate(n)]


def _packed_lens(case):
    """(queries, keys) of each document; the queries are its last tokens."""
    r = random.Random(case["lens"])
    nq = [r.randint(case["least"], case["most"]) for _ in range(case["b"])]
    return nq, [n + (r.randint(0, case["past"]) if case["past"] else 0) for n in nq]


def _prefixes(case, lens):
    """How many leading tokens of each sequence all of its tokens see."""
    r = random.Random(case["lens"] + 1)
    return [min(n, r.randint(case["prefix"] // 2, case["prefix"])) for n in lens]


# ------------------------------------------------------------------ inputs

def _tokens(g, *shape):
    """Heads of tokens: N(0, 1) with a few channels far larger, as keys have."""
    x = torch.randn(*shape, generator=g, device="cuda")
    loud = torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), generator=g, device="cuda")
    x[..., loud] *= 3.0
    return x


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _ints([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist())


def _quantise(v, store):
    """Rows of v as 8-bit codes with a scale each."""
    s = v.abs().amax(dim=-1) / QMAX[store]
    s = torch.where(s > 0, s, torch.ones_like(s))
    c = v / s[..., None]
    c = torch.round(c) if store == "int8" else c.clamp(-448.0, 448.0)
    return c.to(STORE[store]), s


def _pool(g, case, pages):
    """(codes, scales) of a pool of pages, in slices so that a large one needs little room."""
    shape = (pages, case["hk"], case["page"], case["d"])
    codes = torch.empty(shape, dtype=STORE[case["store"]], device="cuda")
    scale = torch.empty(shape[:-1], device="cuda") if case["store"] in QMAX else None
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pages, step):
        v = _tokens(g, min(step, pages - i), *shape[1:])
        if scale is None:
            codes[i:i + step] = v.to(codes.dtype)
        else:
            codes[i:i + step], scale[i:i + step] = _quantise(v, case["store"])
    return codes, scale


def _paged_state(s, case, g, lens):
    """A pool with some pages to spare, and each sequence's pages in an order of their own."""
    per = max(1, -(-max(lens) // case["page"]))
    pages = len(lens) * per + 3
    order = torch.randperm(pages, generator=g, device="cuda")[:len(lens) * per]
    s["table"] = order.view(len(lens), per).to(torch.int32)
    s["k"], s["ks"] = _pool(g, case, pages)
    s["v"], s["vs"] = _pool(g, case, pages)
    s["lens"], s["most"] = _ints(lens), max(lens)


def _blank(s, case):
    """What lies behind each sequence's last token was never written: NaN."""
    pos = torch.arange(s["table"].shape[1] * case["page"], device="cuda")
    seq, at = torch.nonzero(pos[None] >= s["lens"][:, None], as_tuple=True)
    page = s["table"].long()[seq, at // case["page"]]
    for t in ((s["ks"], s["vs"]) if s["ks"] is not None else (s["k"], s["v"])):
        t[page, :, at % case["page"]] = float("nan")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "rotary":
        t, heads, d = case["t"], case["heads"], case["d"]
        s["sec"] = tuple(int(n) for n in case["sections"].split(","))
        # the rotated heads lie next to others of the same projection
        s["data"] = _tokens(g, t, heads + 2, d).to(FLOAT[case["x"]])[:, :heads]
        at = torch.arange(t, device="cuda")
        grid = [at // (VIDEO[1] * VIDEO[2]) + case["at"], at // VIDEO[2] % VIDEO[1], at % VIDEO[2]]
        s["pos"] = torch.stack(grid[:len(s["sec"])], dim=1).to(torch.int32)
        s["out"] = torch.empty(t, heads, d, dtype=FLOAT[case["x"]], device="cuda")
    elif case["op"] == "cache":
        start, new = _cache_lens(case)
        both = [a + b for a, b in zip(start, new)]
        _paged_state(s, case, g, both)
        s["start"], s["offsets"], s["n_new"] = _ints(start), _starts(new), sum(new)
        s["kn"] = _tokens(g, sum(new), case["hk"], case["d"]).to(FLOAT[case["x"]])
        s["vn"] = torch.randn(sum(new), case["hk"], case["d"], generator=g, device="cuda").to(FLOAT[case["x"]])
        s["all_offsets"], s["n_all"] = _starts(both), sum(both)
        if case["do"] != "write":
            s["k_out"], s["v_out"] = (torch.empty(sum(both), case["hk"], case["d"],
                                                  dtype=FLOAT[case["x"]], device="cuda") for _ in range(2))
    else:
        if case["op"] == "paged":
            lens = _paged_lens(case)
            _paged_state(s, case, g, lens)
            _blank(s, case)
            s["q"] = (1.5 * _tokens(g, case["b"], case["hq"], case["d"])).to(FLOAT[case["x"]])
        else:
            nq, lens = _packed_lens(case)
            h, hk, d = case["hq"], case["hk"], case["d"]
            s["nq"], s["nk"], s["most_q"], s["most"] = _ints(nq), _ints(lens), max(nq), max(lens)
            s["q_offsets"], s["k_offsets"] = _starts(nq), _starts(lens)
            s["n_q"] = sum(nq)
            # parts of one projection's rows, or keys and values with the cache's before them
            if nq == lens:
                qkv = _tokens(g, sum(nq), h + 2 * hk, d).to(FLOAT[case["x"]])
                s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
            else:
                s["q"] = _tokens(g, sum(nq), h, d).to(FLOAT[case["x"]])
                s["k"] = _tokens(g, sum(lens), hk, d).to(FLOAT[case["x"]])
                s["v"] = torch.randn(sum(lens), hk, d, generator=g, device="cuda").to(FLOAT[case["x"]])
        s["slope_v"] = (2.0 ** (-8.0 * torch.arange(1, case["hq"] + 1, device="cuda") / case["hq"])
                        if case["slopes"] else None)
        s["prefix_v"] = _ints(_prefixes(case, lens)) if case["prefix"] else None
        s["out"] = torch.empty(s["q"].shape, dtype=FLOAT[case["x"]], device="cuda")
    return s


# ------------------------------------------------------------------ the operators' own calls

def _run_own(s):
    import implicit_gemm_convolution_conv3d_gb300 as c3d
    if s["op"] == "rotary":
        return {"out": c3d.rotary(s["data"], s["pos"], s["sec"], ladder=s["ladder"],
                                  pairs=s["pairs"], inverse=s["inverse"], out=s["out"])}
    if s["op"] == "cache":
        out = {}
        if s["do"] != "read":
            c3d.kv_cache_write(s["kn"], s["vn"], s["k"], s["v"], s["table"], s["start"],
                               k_scale=s["ks"], v_scale=s["vs"], offsets=s["offsets"])
        if s["do"] == "write":
            out["k"], out["v"] = s["k"], s["v"]
        else:
            out["k"], out["v"] = c3d.kv_cache_read(
                s["k"], s["v"], s["table"], s["all_offsets"], k_scale=s["ks"], v_scale=s["vs"],
                k_out=s["k_out"], v_out=s["v_out"])
        out["ks"], out["vs"] = s["ks"], s["vs"]
        return out
    if s["op"] == "paged":
        return {"out": c3d.paged_attention(
            s["q"], s["k"], s["v"], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"],
            cap=s["cap"], window=s["window"], prefix=s["prefix_v"], slopes=s["slope_v"],
            out=s["out"])}
    return {"out": c3d.packed_attention(
        s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], causal=s["causal"], cap=s["cap"],
        window=s["window"], prefix=s["prefix_v"], slopes=s["slope_v"], out=s["out"])}


# ------------------------------------------------------------------ their plain form

def _plain_rotary(s):
    x, n = s["data"].float(), sum(s["sec"])
    sec = torch.tensor(s["sec"], device="cuda")
    axis = torch.repeat_interleave(torch.arange(len(s["sec"]), device="cuda"), sec)
    i = torch.arange(n, device="cuda", dtype=torch.float64)
    if s["ladder"] == "axis":
        first = sec.cumsum(0) - sec
        power = (i - first[axis]) / sec[axis]
    else:
        power = i / n
    freq = 10000.0 ** -power
    angle = s["pos"].double()[:, axis] * freq       # far positions: angles in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if s["inverse"]:
        sin = -sin
    if s["pairs"] == "half":
        a, b, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)
    else:
        a, b, rest = x[..., 0:2 * n:2], x[..., 1:2 * n:2], x[..., 2 * n:]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        y = torch.cat([y, rest], dim=-1)
    return {"out": y.to(s["data"].dtype)}


def _plain_gather(codes, scale, page, off):
    v = codes[page, :, off].float()
    return v if scale is None else v * scale[page, :, off][..., None]


def _raw(t):
    """float8 tensors by their bytes, for the torch operations that do not take them."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_cache(s):
    out, table = {}, s["table"].long()
    if s["do"] != "read":
        i = torch.arange(s["n_new"], device="cuda")
        seq = torch.searchsorted(s["offsets"], i, right=True) - 1
        pos = s["start"][seq] + i - s["offsets"][seq]
        page, off = table[seq, pos // s["page"]], pos % s["page"]
        for_k, for_v = s["kn"], s["vn"]
        if s["ks"] is not None:
            for_k, k_scale = _quantise(for_k.float(), s["store"])
            for_v, v_scale = _quantise(for_v.float(), s["store"])
            s["ks"][page, :, off], s["vs"][page, :, off] = k_scale, v_scale
        _raw(s["k"])[page, :, off], _raw(s["v"])[page, :, off] = _raw(for_k), _raw(for_v)
    if s["do"] == "write":
        out["k"], out["v"] = s["k"], s["v"]
    else:
        i = torch.arange(s["n_all"], device="cuda")
        seq = torch.searchsorted(s["all_offsets"], i, right=True) - 1
        pos = i - s["all_offsets"][seq]
        page, off = table[seq, pos // s["page"]], pos % s["page"]
        out["k"] = _plain_gather(s["k"], s["ks"], page, off).to(FLOAT[s["x"]])
        out["v"] = _plain_gather(s["v"], s["vs"], page, off).to(FLOAT[s["x"]])
    out["ks"], out["vs"] = s["ks"], s["vs"]
    return out


def _plain_softmax(s, score, i, j, seen, heads):
    """Weights of the scores [b, hq, rows, keys]; i, j: the tokens' positions; seen: their mask."""
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    far = (i - j).abs()
    if s["slopes"]:
        score = score - s["slope_v"].view(heads) * far[:, None]
    inside = seen
    if s["window"]:
        inside = inside & (far < s["window"])
    if s.get("causal", True):
        inside = inside & (j <= i)
    if s["prefix"]:
        inside = inside | (seen & (j < s["prefix_v"][:, None, None]))
    score = score.masked_fill(~inside[:, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    w = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = w.sum(dim=-1, keepdim=True)
    return w / torch.where(total == 0, torch.ones_like(total), total)


def _plain_paged(s):
    b, hq, hk, d = s["b"], s["hq"], s["hk"], s["d"]
    j = torch.arange(s["most"], device="cuda")
    seen = j[None] < s["lens"][:, None]
    page, off = s["table"].long()[:, j // s["page"]], (j % s["page"])[None].expand(b, -1)
    k, v = _plain_gather(s["k"], s["ks"], page, off), _plain_gather(s["v"], s["vs"], page, off)
    k, v = (t.masked_fill_(~seen[:, :, None, None], 0.0).transpose(1, 2) for t in (k, v))
    q = s["q"].float().view(b, hk, hq // hk, d)
    score = torch.matmul(q, k.transpose(2, 3)).view(b, hq, 1, -1) / math.sqrt(d)
    w = _plain_softmax(s, score, (s["lens"] - 1)[:, None, None], j[None, None], seen[:, None],
                       (1, hq, 1, 1))
    o = torch.matmul(w.view(b, hk, hq // hk, -1), v)
    return {"out": o.view(b, hq, d).to(s["q"].dtype)}


def _pad(x, offsets, lens, most):
    """Packed rows as [b, heads, most, d], zeros behind each sequence."""
    j = torch.arange(most, device="cuda")
    there = j[None] < lens[:, None]
    row = torch.where(there, offsets[:-1, None] + j, torch.zeros_like(j))
    return x[row].float().masked_fill_(~there[:, :, None, None], 0.0).transpose(1, 2), there


def _plain_packed(s):
    b, hq, hk, d = s["b"], s["hq"], s["hk"], s["d"]
    q, q_there = _pad(s["q"], s["q_offsets"], s["nq"], s["most_q"])
    k, k_there = _pad(s["k"], s["k_offsets"], s["nk"], s["most"])
    v, _ = _pad(s["v"], s["k_offsets"], s["nk"], s["most"])
    q = q.reshape(b, hk, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)).view(b, hq, s["most_q"], -1) / math.sqrt(d)
    i = torch.arange(s["most_q"], device="cuda") + (s["nk"] - s["nq"])[:, None]
    j = torch.arange(s["most"], device="cuda")
    w = _plain_softmax(s, score, i[:, :, None], j[None, None], k_there[:, None], (1, hq, 1, 1))
    o = torch.matmul(w.view(b, hk, -1, s["most"]), v).view(b, hq, s["most_q"], d)
    return {"out": o.transpose(1, 2)[q_there].to(s["q"].dtype)}


def _run_plain(s):
    if s["op"] == "rotary":
        return _plain_rotary(s)
    if s["op"] == "cache":
        return _plain_cache(s)
    return _plain_paged(s) if s["op"] == "paged" else _plain_packed(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def _visible(nq, nk, causal, window, prefix):
    """(pairs of a query and a key that it sees, keys that any query sees) of a document."""
    pairs, keys = 0, set() if window else None
    for i in range(nk - nq, nk):
        lo, hi = 0, nk
        if window:
            lo, hi = max(0, i - window + 1), min(nk, i + window)
        if causal:
            hi = min(hi, i + 1)
        p = min(prefix, nk)
        pairs += max(0, hi - lo) + max(0, min(p, lo)) + max(0, p - max(hi, lo))
    if not window:
        return pairs, nk
    return pairs, min(nk, nq + window - 1 + min(prefix, max(0, nk - nq - window + 1)))


def work(case):
    if case["op"] == "rotary":
        n = sum(int(v) for v in case["sections"].split(","))
        t, heads, d = case["t"], case["heads"], case["d"]
        axes = case["sections"].count(",") + 1
        return {"bytes": 2 * t * heads * d * BYTES[case["x"]] + 4 * t * axes,
                "flops": 6 * t * heads * n}
    d = case["d"]
    if case["op"] == "cache":
        start, new = _cache_lens(case)
        rows = case["hk"] * 2
        held = rows * (d * BYTES[case["store"]] + (4 if case["store"] in QMAX else 0))
        given = rows * d * BYTES[case["x"]]
        n, a = sum(new), sum(new) + sum(start)
        moved = {"write": n * (held + given), "read": a * (held + given),
                 "append": n * (2 * held + given) + sum(start) * held + a * given}[case["do"]]
        tables = 4 * sum(-(-(i + j) // case["page"]) for i, j in zip(start, new))
        done = {"write": n, "read": a, "append": n + a}[case["do"]]
        return {"bytes": moved + tables, "flops": 3 * rows * d * done}
    hq, hk = case["hq"], case["hk"]
    pairs = keys = 0
    if case["op"] == "paged":
        nq, nk = [1] * case["b"], _paged_lens(case)
    else:
        nq, nk = _packed_lens(case)
    pre = _prefixes(case, nk) if case["prefix"] else [0] * len(nk)
    for a, b, p in zip(nq, nk, pre):
        if b:
            n, m = _visible(a, b, case.get("causal", True), case["window"], p)
            pairs, keys = pairs + n, keys + m
    kind = case.get("store", case["x"])
    row = d * BYTES[kind] + (4 if kind in QMAX else 0)
    return {"bytes": 2 * sum(nq) * hq * d * BYTES[case["x"]] + 2 * keys * hk * row,
            "flops": pairs * hq * (4 * d + 4)}


# ------------------------------------------------------------------ the definition, in 64 bits

def _e4m3_values(c):
    """The nearest e4m3 value of each element (ties to the even significand)."""
    _, e = torch.frexp(c)
    step = torch.ldexp(torch.ones_like(c), (e - 1).clamp(min=-6) - 3)
    return (torch.round(c / step) * step).clamp(-448.0, 448.0)


def _exact_rotary(case, s):
    y, n = s["data"].double(), sum(s["sec"])
    pair = 0
    for axis, count in enumerate(s["sec"]):
        for i in range(count):
            power = i / count if case["ladder"] == "axis" else pair / n
            turn = s["pos"][:, axis].double() * math.exp(-power * math.log(10000.0))
            z = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn)[:, None]
            a, b = (pair, pair + n) if case["pairs"] == "half" else (2 * pair, 2 * pair + 1)
            r = torch.complex(y[..., a], y[..., b]) * z
            y[..., a], y[..., b] = r.real, r.imag
            pair += 1
    return {"out": y}


def _exact_cache(case, s):
    start, new = _cache_lens(case)
    table = s["table"].tolist()
    out = {}
    for name, row, codes, scale in (("k", s["kn"], s["k"], s["ks"]), ("v", s["vn"], s["v"], s["vs"])):
        held = codes.double()
        size = None if scale is None else scale.double()
        if case["do"] != "read":
            x = row.double()
            if size is not None:
                top = x.abs().max(dim=-1).values
                sx = (top / QMAX[case["store"]]).masked_fill(top == 0, 1.0)
                x = x / sx[..., None]
                x = x.round() if case["store"] == "int8" else _e4m3_values(x)
            at, pages, offs = 0, [], []
            for b, (a, n) in enumerate(zip(start, new)):
                pages += [table[b][p // case["page"]] for p in range(a, a + n)]
                offs += [p % case["page"] for p in range(a, a + n)]
            pages, offs = torch.tensor(pages, device="cuda"), torch.tensor(offs, device="cuda")
            held[pages, :, offs] = x
            if size is not None:
                size[pages, :, offs] = sx
        out[name + "s"] = size
        if case["do"] != "write":
            if size is not None:
                held = held * size[..., None]
            parts = []
            for b, (a, n) in enumerate(zip(start, new)):
                p = -(-(a + n) // case["page"])
                seq = held[torch.tensor(table[b][:p], dtype=torch.long, device="cuda")]
                parts.append(seq.transpose(1, 2).reshape(-1, case["hk"], case["d"])[:a + n])
            held = torch.cat(parts)
        out[name] = held
    return out


def _exact_rows(case, q, k, v, first, head, slope, prefix):
    """One head's rows q [n, d], the first at position `first`, over k, v [m, d]."""
    z = torch.einsum("id,jd->ij", q, k) * case["d"] ** -0.5
    if case["cap"]:
        z = torch.special.expm1(2 * z / case["cap"]) / (torch.exp(2 * z / case["cap"]) + 1) * case["cap"]
    i = torch.arange(first, first + q.shape[0], device="cuda")[:, None]
    j = torch.arange(k.shape[0], device="cuda")[None]
    if slope is not None:
        z -= slope[head].double() * (i - j).abs()
    hide = torch.zeros_like(z, dtype=torch.bool)
    if case["window"]:
        hide |= (i - j >= case["window"]) | (j - i >= case["window"])
    if case.get("causal", True):
        hide |= j > i
    if prefix:
        hide &= j >= prefix
    z.masked_fill_(hide, -math.inf)
    return torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True)) @ v


def _exact_attention(case, s):
    paged = case["op"] == "paged"
    nq, nk = ([1] * case["b"], _paged_lens(case)) if paged else _packed_lens(case)
    prefix = _prefixes(case, nk) if case["prefix"] else [0] * len(nk)
    if sum(a * b for a, b in zip(nq, nk)) * case["hq"] * case["d"] > 3e12:
        return None
    table = s["table"].tolist() if paged else None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    row = key = 0
    for b, (n, m) in enumerate(zip(nq, nk)):
        if paged and m:
            pages = torch.tensor(table[b][:-(-m // case["page"])], dtype=torch.long, device="cuda")
            k, v = (t[pages].double() for t in (s["k"], s["v"]))
            if s["ks"] is not None:
                k, v = k * s["ks"][pages].double()[..., None], v * s["vs"][pages].double()[..., None]
            k, v = (t.transpose(1, 2).reshape(-1, case["hk"], case["d"])[:m] for t in (k, v))
        elif m:
            k, v = s["k"][key:key + m].double(), s["v"][key:key + m].double()
        for h in range(case["hq"] if m else 0):
            kh = h * case["hk"] // case["hq"]
            out[row:row + n, h] = _exact_rows(case, s["q"][row:row + n, h].double(), k[:, kh], v[:, kh],
                                              m - n, h, s["slope_v"], prefix[b])
        row, key = row + n, key + m
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    return _exact_cache(case, s) if case["op"] == "cache" else _exact_attention(case, s)
