"""Operators on rows of tokens, as they follow a convolutional patch
embedding (C ABI in ``include/token_ops.h``): the root-mean-square norm with
the residual's addition and an 8-bit output, the (gated) activation with an
8-bit output, and the matrix product of 8-bit tokens and weights.

Tokens are ``[..., width]`` tensors whose rows are contiguous; a 2-D tensor
may have any row stride (a slice of a wider matrix), more leading dimensions
have to be viewable as rows.  8-bit tensors are ``torch.int8`` or
``torch.float8_e4m3fn`` with one fp32 scale per row: value = code * scale.
Like the convolutions', these calls marshal arguments only, run on the
current (or the given) stream, and raise on anything the library refuses.
A given ``stream`` is not made to wait for anything: inputs that another
stream still writes, and results that another stream reads, are the caller's
to order (``stream.wait_stream``).  What a call allocates for a given stream
is that stream's memory.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import ACT_CODES, _check, _stream_handle, load_library
from . import _raw_current_stream as _raw_stream

CONV_DTYPE_INT8, CONV_DTYPE_F16, CONV_DTYPE_F32 = 2, 3, 4
_FLOAT = {torch.bfloat16: 0, torch.float16: CONV_DTYPE_F16, torch.float32: CONV_DTYPE_F32}
_CODE = {torch.float8_e4m3fn: 1, torch.int8: CONV_DTYPE_INT8}
_F32 = torch.float32
NO_WORKSPACE_TOKENS = 16   # LINEAR_W8A8_NO_WORKSPACE_TOKENS of the header

_fns = None


def _bind():
    """The library's token entry points with their argument types."""
    global _fns
    lib = load_library()
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.rms_norm_quant_fwd.argtypes = [vp, i32, i64, vp, i32, i64, vp, i32, ctypes.c_float, i64,
                                       i64, i32, vp, i64, vp, vp, i64, vp]
    lib.act_quant_fwd.argtypes = [vp, i32, i64, i32, i32, i64, i64, i32, vp, i64, vp, vp]
    lib.linear_w8a8_fwd.argtypes = [vp, i64, vp, i64, i32, i64, i64, i64, vp, vp, vp, i32, vp,
                                    i32, i64, vp, ctypes.c_size_t, vp]
    lib.linear_w8a8_workspace_size.argtypes = [vp, i64, vp, i64, i32, i64, i64, i64]
    lib.linear_w8a8_workspace_size.restype = ctypes.c_size_t
    _fns = lib
    return lib


def _rows(t: torch.Tensor, types: dict, what: str) -> Tuple[int, int, int, int]:
    """(rows, row length, row stride, type code) of a CUDA tensor [..., width]."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} has dtype {t.dtype}: one of {[str(d) for d in types]}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape = t.shape
    if len(shape) == 2:
        rows, width = shape
        stride, last = t.stride()
        if last != 1 and width > 1:
            raise ValueError(f"{what} must have contiguous rows")
        return rows, width, (stride if rows > 1 else width), code
    if len(shape) < 1:
        raise ValueError(f"{what} must have at least one dimension")
    width = shape[-1]
    if t.is_contiguous():
        rows = 1
        for d in shape[:-1]:
            rows *= d
        return rows, width, width, code
    try:
        return _rows(t.view(-1, width), types, what)
    except RuntimeError:
        raise ValueError(f"{what} must be viewable as rows") from None


def _vector(t: Optional[torch.Tensor], n: int, what: str, other=_F32) -> Optional[int]:
    """Data pointer of a contiguous CUDA vector of n elements, fp32 (or `other`)."""
    if t is None:
        return None
    dtype = t.dtype
    if dtype is not _F32 and dtype is not other:
        raise TypeError(f"{what} must be float32" + ("" if other is _F32 else f" or {other}"))
    if t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {n} elements")
    return t.data_ptr()


def _given_rows(t: torch.Tensor, shape, width: int, rows: int, types: dict,
                what: str) -> Tuple[int, int]:
    """(row stride, type code) of a given output for tokens of `shape`, `width` wide."""
    out_rows, out_width, stride, code = _rows(t, types, what)
    if out_width != width or out_rows != rows or (
            len(shape) != 2 and t.shape[:-1] != shape[:-1]) or t.dim() != len(shape):
        raise ValueError(f"{what} must have shape {tuple(shape[:-1]) + (width,)}")
    return stride, code


def _stream(stream: Optional[torch.cuda.Stream], x: torch.Tensor):
    return _stream_handle(stream, x.device.index) if stream is not None or _raw_stream is None \
        else _raw_stream(x.device.index)


def _new(shape, dtype, x: torch.Tensor, stream) -> torch.Tensor:
    """A tensor that the call may write at once.  With a given stream it is that
    stream's memory: a block freed on the current stream could still be in use
    there.  The caller's stream, which gets the tensor, is recorded on it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    caller = torch.cuda.current_stream(x.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=x.device)
    t.record_stream(caller)
    return t


def _codes_out(x, rows, width, qdtype, out, scale_out, stream):
    """The (given or new) code and scale tensors for rows of x: with the codes'
    row stride and type and the scales' pointer."""
    if out is None:
        code = _CODE.get(qdtype)
        if code is None:
            raise TypeError("qdtype must be torch.int8 or torch.float8_e4m3fn")
        out, stride = _new(x.shape[:-1] + (width,), qdtype, x, stream), width
    else:
        stride, code = _given_rows(out, x.shape, width, rows, _CODE, "out")
    if scale_out is None:
        scale_out = _new(x.shape[:-1], torch.float32, x, stream)
        return out, scale_out, stride, code, scale_out.data_ptr()
    return out, scale_out, stride, code, _vector(scale_out, rows, "scale_out")


def rms_norm_quant(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   residual: Optional[torch.Tensor] = None, qdtype: torch.dtype = torch.int8,
                   out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """h = x + residual; codes and row scales of h / sqrt(mean(h^2) + eps) * weight.

    ``x`` bf16, fp16 or fp32; ``residual`` (x's shape) and ``weight`` ([width])
    of x's type or fp32.  Returns (codes, scale, residual_out): ``residual_out``
    is h in the residual's type (None without a residual), and may be given as
    ``residual`` itself to update it in place.  ``out``'s type, where given,
    stands in for ``qdtype``."""
    lib = _fns or _bind()
    rows, width, xs, xc = _rows(x, _FLOAT, "x")
    out, scale_out, qs, qc, sp = _codes_out(x, rows, width, qdtype, out, scale_out, stream)
    wp = _vector(weight, width, "weight", x.dtype)
    wc = xc if weight is None or weight.dtype is x.dtype else CONV_DTYPE_F32
    rp = op = None
    rc = rs = os_ = 0
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        _, _, rs, rc = _rows(residual, _FLOAT, "residual")
        if residual_out is None:
            residual_out, os_ = _new(x.shape, residual.dtype, x, stream), width
        elif residual_out is residual:
            os_ = rs
        else:
            os_, oc = _given_rows(residual_out, x.shape, width, rows, _FLOAT, "residual_out")
            if oc != rc:
                raise ValueError("residual_out must have the residual's type")
        rp, op = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    st = lib.rms_norm_quant_fwd(x.data_ptr(), xc, xs, rp, rc, rs, wp, wc, eps, rows, width, qc,
                                out.data_ptr(), qs, sp, op, os_, _stream(stream, x))
    if st:
        _check(st, "rms_norm_quant_fwd")
    return out, scale_out, residual_out


def act_quant(x: torch.Tensor, act: str = "none", gated: bool = False,
              qdtype: torch.dtype = torch.int8, out: Optional[torch.Tensor] = None,
              scale_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Codes and row scales of act(x), or with ``gated`` of act(x[..., :F]) *
    x[..., F:] for x [..., 2F].  ``act`` is "none", "relu", "silu" or "gelu"
    (erf form).  ``act_quant(w)`` of weights [outputs, width] gives the codes
    and channel scales that ``linear_w8a8`` takes."""
    code = ACT_CODES.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACT_CODES)}")
    lib = _fns or _bind()
    rows, width, xs, xc = _rows(x, _FLOAT, "x")
    if gated:
        if width % 2:
            raise ValueError("a gated x must have an even number of columns")
        width //= 2
    out, scale_out, qs, qc, sp = _codes_out(x, rows, width, qdtype, out, scale_out, stream)
    st = lib.act_quant_fwd(x.data_ptr(), xc, xs, code, 1 if gated else 0, rows, width, qc,
                           out.data_ptr(), qs, sp, _stream(stream, x))
    if st:
        _check(st, "act_quant_fwd")
    return out, scale_out


# workspace bytes by the operands' sizes, strides and alignment
_need_cache: dict = {}


def _linear_need(lib, xp, xs, wp, ws, qc, rows, outputs, width) -> int:
    key = (xs, ws, qc, rows, outputs, width, xp & 15, wp & 15)
    need = _need_cache.get(key)
    if need is None:
        need = lib.linear_w8a8_workspace_size(xp, xs, wp, ws, qc, rows, outputs, width)
        if len(_need_cache) >= 1024:
            _need_cache.clear()
        _need_cache[key] = need
    return need


def linear_w8a8(x: torch.Tensor, w: torch.Tensor, scale_x: Optional[torch.Tensor] = None,
                scale_w: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                act: str = "none", out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """act((x @ w.T) * scale_x[:, None] * scale_w + bias) for 8-bit x [..., width]
    and w [outputs, width] of one type, with fp32 row scales (None: ones),
    fp32 bias and fp32 sums -> [..., outputs] in bf16, fp16 or fp32
    (``out``'s type, where given).  A workspace is taken from torch's
    allocator when the product needs one (int8 with many tokens, rows that are
    not 16-byte aligned) and none is given."""
    code = ACT_CODES.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACT_CODES)}")
    lib = _fns or _bind()
    rows, width, xs, qc = _rows(x, _CODE, "x")
    if w.dim() != 2:
        raise ValueError("w must be [outputs, width]")
    outputs, w_width, ws, wc = _rows(w, _CODE, "w")
    if wc != qc:
        raise TypeError("x and w must have the same dtype")
    if w_width != width:
        raise ValueError(f"x has rows of {width} elements, w of {w_width}")
    if out is None:
        oc = _FLOAT.get(out_dtype)
        if oc is None:
            raise TypeError("out_dtype must be bfloat16, float16 or float32")
        out, os_ = _new(x.shape[:-1] + (outputs,), out_dtype, x, stream), outputs
    else:
        os_, oc = _given_rows(out, x.shape, outputs, rows, _FLOAT, "out")
    xp, wp = x.data_ptr(), w.data_ptr()
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif rows > NO_WORKSPACE_TOKENS:
        need = _linear_need(lib, xp, xs, wp, ws, qc, rows, outputs, width)
        if need:
            workspace = _new((need,), torch.uint8, x, stream)
            ws_ptr, ws_bytes = workspace.data_ptr(), need
    st = lib.linear_w8a8_fwd(xp, xs, wp, ws, qc, rows, outputs, width,
                             _vector(scale_x, rows, "scale_x"),
                             _vector(scale_w, outputs, "scale_w"),
                             _vector(bias, outputs, "bias"), code, out.data_ptr(), oc, os_,
                             ws_ptr, ws_bytes, _stream(stream, x))
    if st:
        _check(st, "linear_w8a8_fwd")
    return out
