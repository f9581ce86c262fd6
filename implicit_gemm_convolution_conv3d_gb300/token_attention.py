"""Attention on the tokens of a convolutional patch embedding, image and video
(C ABI in ``include/token_attention.h``): rotary positions with several axes, a
paged cache of keys and values in 8 (or 16) bits, attention of one new token over
that cache, and attention within documents packed in one buffer.

Heads of tokens are ``[tokens, heads, width]`` tensors whose last dimension is
contiguous; tokens and heads may have any stride from the width on, as parts of one
projection's rows have, and an output's or a cache's rows may not overlap.  A cache is a pair of ``[pages, kv_heads, page_size, width]`` tensors,
with fp32 scales ``[pages, kv_heads, page_size]`` where it is ``torch.int8`` or
``torch.float8_e4m3fn`` (value = code * scale); ``page_table`` [sequences, pages of
the longest] int32 says where token t of a sequence lies: row ``t % page_size`` of
page ``page_table[s, t // page_size]``.  Lengths, offsets and tables are device
tensors: no call waits for the GPU.  Like the other token operators these marshal
arguments only, run on the current (or the given) stream, and raise on anything
the library refuses.  They are for serving and record no gradient, but for ``rotary``,
whose gradient is the inverse rotation.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence, Tuple

import torch

from . import _check, load_library
from .token_ops import _CODE, _FLOAT, _new, _stream

_HALF = {torch.bfloat16: _FLOAT[torch.bfloat16], torch.float16: _FLOAT[torch.float16]}
_CACHE = {**_CODE, **_HALF}
_I32 = torch.int32
MAX_PAIRS, MAX_AXES = 128, 8   # ROTARY_MAX_PAIRS, ROTARY_MAX_AXES of the header

_fns = None


class _Cache(ctypes.Structure):
    """kv_cache of the header."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [("dtype", ctypes.c_int)]
                + [(n, ctypes.c_int64) for n in (
                    "pages", "heads", "page_size", "width", "page_stride", "head_stride",
                    "row_stride", "scale_page_stride", "scale_head_stride")])


def _bind():
    """The library's entry points with their argument types."""
    global _fns
    lib = load_library()
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    cache = ctypes.POINTER(_Cache)
    lib.rotary_fwd.argtypes = [vp, i32, i64, i64, vp, i32, i32, vp, vp, i32, i32, i32, i64, i64,
                               i64, vp, i64, i64, vp]
    for f in (lib.kv_cache_write, lib.kv_cache_read):
        f.argtypes = [cache, vp, vp, i32, i64, i64, i64, vp, vp, vp, i64, i64, i64, vp]
    lib.paged_attention_fwd.argtypes = [vp, i32, i64, i64, cache, vp, i64, i64, vp, vp, vp, f32,
                                        f32, i64, i64, i64, vp, i64, i64, vp, ctypes.c_size_t, vp]
    lib.paged_attention_workspace_size.argtypes = [i64] * 6
    lib.paged_attention_workspace_size.restype = ctypes.c_size_t
    lib.packed_attention_fwd.argtypes = [vp, i64, i64, vp, vp, i64, i64, i32, vp, vp, i64, i64,
                                         i64, i64, i64, i64, i32, i64, vp, vp, f32, f32, vp, i64,
                                         i64, vp]
    _fns = lib
    return lib


def _here(x: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    """One device for all of a call's tensors: the current one, which launches."""
    d = x.get_device()
    if d != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {x.device}, which is not the current device")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"all tensors of a call must be on {x.device}")


def _heads(t: torch.Tensor, types: dict, what: str) -> Tuple[int, int, int, int, int, int]:
    """(tokens, heads, width, token stride, head stride, type code) of [tokens, heads, width]."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} has dtype {t.dtype}: one of {[str(d) for d in types]}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, width]")
    tokens, heads, width = t.shape
    ts, hs, last = t.stride()
    if last != 1 and width > 1 and tokens and heads:
        raise ValueError(f"{what} must have contiguous rows")
    return tokens, heads, width, (ts if tokens > 1 else heads * width), (hs if heads > 1 else width), code


def _given(out: Optional[torch.Tensor], x: torch.Tensor, types: dict, code: int, stream,
           what: str = "out"):
    """A given or new output of x's shape and type: the tensor and its strides."""
    if out is None:
        out = _new(x.shape, x.dtype, x, stream)
        return out, x.shape[1] * x.shape[2], x.shape[2]
    _, _, _, ts, hs, oc = _heads(out, types, what)
    if out.shape != x.shape or oc != code:
        raise ValueError(f"{what} must have shape {tuple(x.shape)} and type {x.dtype}")
    return out, ts, hs


def _ints(t: Optional[torch.Tensor], n: Optional[int], what: str) -> Optional[int]:
    """Data pointer of a contiguous int32 CUDA vector of n elements."""
    if t is None:
        return None
    if t.dtype is not _I32:
        raise TypeError(f"{what} must be int32")
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA vector" + ("" if n is None else f" of {n}"))
    return t.data_ptr()


def _slopes(t: Optional[torch.Tensor], heads: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not torch.float32:
        raise TypeError("slopes must be float32")
    if t.numel() != heads or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"slopes must be a contiguous CUDA vector of {heads}")
    return t.data_ptr()


def _table(t: torch.Tensor) -> Tuple[int, int, int, int]:
    """(pointer, stride, pages, sequences) of a page table."""
    if t.dtype is not _I32:
        raise TypeError("page_table must be int32")
    if not t.is_cuda or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("page_table must be a CUDA tensor [sequences, pages] with contiguous rows")
    n, pages = t.shape
    return t.data_ptr(), (t.stride(0) if n > 1 else pages), pages, n


def _own(shape, stride) -> Tuple[int, ...]:
    """Strides in which a dimension of one element, whose stride is nobody's, has the extent
    of those behind it."""
    out, extent = [], 1
    for n, s in zip(reversed(shape), reversed(stride)):
        s = s if n > 1 else extent
        extent = max(extent, n * s)
        out.append(s)
    return tuple(reversed(out))


def _strides(a: torch.Tensor, b: torch.Tensor, what: str) -> Tuple[int, ...]:
    """The strides that two tensors of one shape share, but the last, which is contiguous."""
    shape, stride, other = a.shape, a.stride(), b.stride()
    if 1 in shape:
        stride, other = _own(shape, stride), _own(shape, other)
    if stride != other:
        raise ValueError(f"{what} must have the same strides")
    if stride[-1] != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return stride[:-1]


def _cache(k: torch.Tensor, v: torch.Tensor, k_scale, v_scale) -> _Cache:
    code = _CACHE.get(k.dtype)
    if code is None:
        raise TypeError(f"a cache has dtype {k.dtype}: one of {[str(d) for d in _CACHE]}")
    if k.dim() != 4 or not k.is_cuda or not v.is_cuda:
        raise ValueError("a cache must be CUDA tensors [pages, kv_heads, page_size, width]")
    shape = k.shape
    if v.dtype is not k.dtype or v.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape and type")
    stride = _strides(k, v, "k_cache and v_cache")
    kp = vp = None
    scale = (0, 0)
    if k.dtype in _CODE:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        for s in (k_scale, v_scale):
            if s.dtype is not torch.float32:
                raise TypeError("scales must be float32")
            if s.shape != shape[:3] or not s.is_cuda:
                raise ValueError(f"scales must be CUDA tensors {tuple(shape[:3])}")
        scale = _strides(k_scale, v_scale, "k_scale and v_scale")
        kp, vp = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("only an 8-bit cache has scales")
    return _Cache(k.data_ptr(), v.data_ptr(), kp, vp, code, *shape, *stride, *scale)


# ------------------------------------------------------------------ rotary positions

@functools.lru_cache(maxsize=256)
def _ladder(sections: Tuple[int, ...], base: float, ladder: str, scales, frequencies):
    """C arrays of each pair's axis and of its radians for each unit of position."""
    n = sum(sections)
    if not sections or len(sections) > MAX_AXES or any(
            not isinstance(s, int) or s < 0 for s in sections) or not 0 < n <= MAX_PAIRS:
        raise ValueError(f"sections must be 1 to {MAX_AXES} pair counts with a sum of 1 to {MAX_PAIRS}")
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    if frequencies is not None:
        if len(frequencies) != n:
            raise ValueError(f"frequencies must be {n} numbers")
        freq = [float(f) for f in frequencies]
    else:
        if not base > 0:
            raise ValueError("base must be above 0")
        if ladder == "axis":
            freq = [base ** (-i / s) for s in sections for i in range(s)]
        elif ladder == "shared":
            freq = [base ** (-i / n) for i in range(n)]
        else:
            raise ValueError("ladder must be 'axis' or 'shared'")
    if scales is not None:
        if len(scales) != len(sections):
            raise ValueError(f"scales must be {len(sections)} numbers")
        freq = [f * float(scales[a]) for f, a in zip(freq, axis)]
    if not all(map(math.isfinite, freq)):
        raise ValueError("frequencies must be finite")
    return n, (ctypes.c_int * n)(*axis), (ctypes.c_double * n)(*freq)


class _Rotary(torch.autograd.Function):
    """rotary of an x that wants a gradient: the inverse rotation of the result's."""

    @staticmethod
    def forward(ctx, x, positions, stream, inverse, kw):
        ctx.save_for_backward(positions)
        ctx.inverse, ctx.kw = inverse, kw
        return rotary(x, positions, inverse=inverse, stream=stream, **kw)

    @staticmethod
    def backward(ctx, grad):
        # (contiguous: a gradient that was broadcast has strides of 0; on the stream that
        # autograd runs this on)
        return (rotary(grad.contiguous(), *ctx.saved_tensors, inverse=not ctx.inverse, **ctx.kw),
                None, None, None, None)


def rotary(x: torch.Tensor, positions: torch.Tensor, sections: Sequence[int],
           base: float = 10000.0, ladder: str = "axis", pairs: str = "half",
           scales: Optional[Sequence[float]] = None,
           frequencies: Optional[Sequence[float]] = None, inverse: bool = False,
           out: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Heads x [tokens, heads, width] turned by their token's positions.

    ``positions`` [tokens, axes] (or [tokens] for one axis) are int32 or int64, as
    they are (time, height, width of a patch); ``sections`` says how many pairs of a
    head turn with each axis, in order.  Pair p turns by its axis' position times its
    frequency: with ``ladder`` "axis" base^(-i/n) for the i-th of the axis' n pairs,
    with "shared" base^(-p/N) over all N pairs; ``frequencies`` [N] gives them
    outright, and ``scales`` [axes] multiplies them (positions in other units).
    ``pairs``: "half" pairs elements (p, p + N), "interleaved" (2p, 2p + 1); elements
    from 2N on stay as they are.  Angles are exact to 2 pi |position| 2^-65, then in
    fp32, for far positions too.  ``inverse``
    turns back: the gradient with respect to x of a loss whose gradient with respect
    to the result is x; where x requires a gradient, it is recorded so (not with
    ``out``, which records nothing).  x bf16, fp16 or fp32; ``out`` may be ``x``."""
    if out is None and x.requires_grad and torch.is_grad_enabled():
        return _Rotary.apply(x, positions, stream, bool(inverse), dict(
            sections=tuple(sections), base=base, ladder=ladder, pairs=pairs,
            scales=None if scales is None else tuple(scales),
            frequencies=None if frequencies is None else tuple(frequencies)))
    lib = _fns or _bind()
    n, axis, freq = _ladder(tuple(sections), float(base), ladder,
                            None if scales is None else tuple(scales),
                            None if frequencies is None else tuple(frequencies))
    if pairs != "half" and pairs != "interleaved":
        raise ValueError("pairs must be 'half' or 'interleaved'")
    tokens, heads, width, ts, hs, code = _heads(x, _FLOAT, "x")
    axes = len(sections)
    if positions.dtype is not _I32 and positions.dtype is not torch.int64:
        raise TypeError("positions must be int32 or int64")
    if not positions.is_cuda or not positions.is_contiguous() or not (
            positions.shape == (tokens, axes) or axes == 1 and positions.shape == (tokens,)):
        raise ValueError(f"positions must be a contiguous CUDA tensor [{tokens}, {axes}]")
    if out is x:
        os_, oh = ts, hs
    else:
        out, os_, oh = _given(out, x, _FLOAT, code, stream)
    _here(x, positions, out)
    st = lib.rotary_fwd(x.data_ptr(), code, ts, hs, positions.data_ptr(), positions.element_size(),
                        axes, axis, freq, n, pairs == "interleaved", bool(inverse), tokens, heads,
                        width, out.data_ptr(), os_, oh, _stream(stream, x))
    if st:
        _check(st, "rotary_fwd")
    return out


# ------------------------------------------------------------------ the cache

def kv_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, starts: torch.Tensor,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   offsets: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """New keys and values [tokens, kv_heads, width] to the cache, in 8 bits with a
    scale per token and head, or as they are in a cache of their own type.

    Rows ``offsets[s]`` .. ``offsets[s+1]`` (int32 [sequences + 1]) are tokens
    ``starts[s]``, ``starts[s] + 1``, ... (int32 [sequences]) of sequence s; without
    offsets row s is the one new token of sequence s.  Rows in no sequence, negative
    tokens, and tokens whose page is not in the table or the pool are not written."""
    lib = _fns or _bind()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    tokens, heads, width, ts, hs, code = _heads(k, _FLOAT, "k")
    if _heads(v, _FLOAT, "v") != (tokens, heads, width, ts, hs, code):
        raise ValueError("k and v must have the same shape, type and strides")
    if heads != c.heads or width != c.width:
        raise ValueError(f"k and v must be [tokens, {c.heads}, {c.width}] for this cache")
    tp, tstride, pages, n = _table(page_table)
    if offsets is None and tokens != n:
        raise ValueError("without offsets there is one token for each sequence of page_table")
    _here(k, v, k_cache, v_cache, page_table, starts, k_scale, v_scale, offsets)
    st = lib.kv_cache_write(c, k.data_ptr(), v.data_ptr(), code, ts, hs, tokens,
                            _ints(offsets, n + 1, "offsets"), _ints(starts, n, "starts"), tp,
                            tstride, pages, n, _stream(stream, k))
    if st:
        _check(st, "kv_cache_write")


def kv_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                  offsets: torch.Tensor, tokens: Optional[int] = None,
                  starts: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                  v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                  k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cache's keys and values as packed rows [tokens, kv_heads, width], in the form
    that ``packed_attention`` takes: rows ``offsets[s]`` .. ``offsets[s+1]`` are tokens
    ``starts[s]`` (0 without starts), ... of sequence s.  Either ``tokens`` (the rows of
    new outputs, of type ``dtype``) or both outputs are given.  Rows in no sequence are
    not written; a token whose page is not in the table or the pool reads as NaN."""
    lib = _fns or _bind()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    if (k_out is None) != (v_out is None) or (k_out is None) == (tokens is None):
        raise ValueError("give tokens, or both k_out and v_out")
    if k_out is None:
        if dtype not in _FLOAT:
            raise TypeError("dtype must be bfloat16, float16 or float32")
        shape = (int(tokens), c.heads, c.width)
        k_out, v_out = (_new(shape, dtype, k_cache, stream) for _ in range(2))
    rows, heads, width, ts, hs, code = _heads(k_out, _FLOAT, "k_out")
    if _heads(v_out, _FLOAT, "v_out") != (rows, heads, width, ts, hs, code):
        raise ValueError("k_out and v_out must have the same shape, type and strides")
    if heads != c.heads or width != c.width:
        raise ValueError(f"k_out and v_out must be [tokens, {c.heads}, {c.width}] for this cache")
    tp, tstride, pages, n = _table(page_table)
    _here(k_cache, v_cache, page_table, offsets, starts, k_scale, v_scale, k_out, v_out)
    st = lib.kv_cache_read(c, k_out.data_ptr(), v_out.data_ptr(), code, ts, hs, rows,
                           _ints(offsets, n + 1, "offsets"), _ints(starts, n, "starts"), tp,
                           tstride, pages, n, _stream(stream, k_cache))
    if st:
        _check(st, "kv_cache_read")
    return k_out, v_out


# ------------------------------------------------------------------ attention

# workspace bytes by the sizes they depend on, and the device
_need_cache: dict = {}


def _paged_need(lib, device, *sizes) -> int:
    key = (device, *sizes)
    need = _need_cache.get(key)
    if need is None:
        need = lib.paged_attention_workspace_size(*sizes)
        if len(_need_cache) >= 1024:
            _need_cache.clear()
        _need_cache[key] = need
    return need


def paged_attention_workspace_size(sequences: int, heads: int, kv_heads: int, width: int,
                                   page_size: int, table_pages: int) -> int:
    """Bytes of workspace that ``paged_attention`` of these sizes takes on the current
    device; 0 where it takes none."""
    return _paged_need(_fns or _bind(), torch.cuda.current_device(), sequences, heads, kv_heads,
                       width, page_size, table_pages)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    page_table: torch.Tensor, lengths: torch.Tensor,
                    k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, cap: float = 0.0, window: int = 0,
                    prefix: Optional[torch.Tensor] = None, slopes: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of each sequence's newest token, q [sequences, heads, width] (bf16 or
    fp16), over its ``lengths[s]`` (int32) cached tokens, the new one among them ->
    [sequences, heads, width].  A sequence of length 0 gets zeros.

    ``heads`` is a multiple of the cache's; head h reads key head h // (heads //
    kv_heads).  Scores are scale * q.k (scale 1 / sqrt(width) unless given), with
    ``cap`` > 0 cap * tanh(score / cap), and with ``slopes`` [heads] less slope *
    distance.  With ``window`` > 0 only the last ``window`` tokens and the first
    ``prefix[s]`` are seen; pages of unseen tokens are not looked at.  The workspace
    (``paged_attention_workspace_size`` bytes) is taken from torch's allocator unless
    one is given (calls that may overlap need one each; where the size is 0, one of
    0 bytes, or of the size of longer tables)."""
    lib = _fns or _bind()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    n, heads, width, qs, qh, code = _heads(q, _HALF, "q")
    if width != c.width:
        raise ValueError(f"q has heads of {width} elements, the cache of {c.width}")
    tp, tstride, pages, rows = _table(page_table)
    if rows != n:
        raise ValueError("page_table must have a row for each sequence")
    out, os_, oh = _given(out, q, _HALF, code, stream)
    if workspace is None:
        need = _paged_need(lib, q.get_device(), n, heads, c.heads, width, c.page_size, pages)
        if need:
            workspace = _new((need,), torch.uint8, q, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _here(q, k_cache, v_cache, page_table, lengths, k_scale, v_scale, prefix, slopes, out, workspace)
    st = lib.paged_attention_fwd(
        q.data_ptr(), code, qs, qh, c, tp, tstride, pages, _ints(lengths, n, "lengths"),
        _ints(prefix, n, "prefix"), _slopes(slopes, heads),
        width ** -0.5 if scale is None else scale, cap, window, n, heads, out.data_ptr(), os_, oh,
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream, q))
    if st:
        _check(st, "paged_attention_fwd")
    return out


def packed_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                     k_offsets: Optional[torch.Tensor] = None, causal: bool = False,
                     scale: Optional[float] = None, cap: float = 0.0, window: int = 0,
                     prefix: Optional[torch.Tensor] = None, slopes: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention within documents packed one after the other: document s has queries
    ``q[q_offsets[s]:q_offsets[s+1]]`` and keys and values
    ``k[k_offsets[s]:k_offsets[s+1]]`` (int32 [documents + 1]; without ``k_offsets``
    they are the same), its queries being its last tokens -> [tokens, heads, width].

    A query at position i sees the keys j of its document with |i - j| < ``window``
    (if > 0) and j <= i (if ``causal``), and those below ``prefix[s]``; a query that
    sees nothing gets zeros.  Scores as in ``paged_attention``; the distance is
    |i - j|.  q, k, v bf16 or fp16, 16-byte aligned, of up to 128 elements a head (a
    multiple of 8); k and v have the same strides.  Rows in no document are not
    written."""
    lib = _fns or _bind()
    nq, heads, width, qs, qh, code = _heads(q, _HALF, "q")
    nk, kv_heads, kw, ks, kh, kc = _heads(k, _HALF, "k")
    if _heads(v, _HALF, "v") != (nk, kv_heads, kw, ks, kh, kc):
        raise ValueError("k and v must have the same shape, type and strides")
    if kc != code or kw != width:
        raise ValueError("q and k must have the same type and width")
    if q_offsets.dim() != 1 or q_offsets.shape[0] < 1:
        raise ValueError("q_offsets must be a vector of documents + 1")
    n = q_offsets.shape[0] - 1
    if k_offsets is None:
        if nk != nq:
            raise ValueError("without k_offsets q and k must have the same tokens")
        k_offsets = q_offsets
    out, os_, oh = _given(out, q, _HALF, code, stream)
    _here(q, k, v, q_offsets, k_offsets, prefix, slopes, out)
    st = lib.packed_attention_fwd(
        q.data_ptr(), qs, qh, k.data_ptr(), v.data_ptr(), ks, kh, code,
        _ints(q_offsets, n + 1, "q_offsets"), _ints(k_offsets, n + 1, "k_offsets"), n, nq, nk,
        heads, kv_heads, width, bool(causal), window, _ints(prefix, n, "prefix"),
        _slopes(slopes, heads), width ** -0.5 if scale is None else scale, cap, out.data_ptr(),
        os_, oh, _stream(stream, q))
    if st:
        _check(st, "packed_attention_fwd")
    return out
