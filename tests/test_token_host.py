"""The token operators' C ABI without a GPU: exported symbols, and argument
checks that return before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

from implicit_gemm_convolution_conv3d_gb300 import build as pkg_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "token_ops.h")
BF16, E4M3, INT8, F16, F32 = 0, 1, 2, 3, 4
INVALID = 1
P = 4096   # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    import implicit_gemm_convolution_conv3d_gb300 as p
    from implicit_gemm_convolution_conv3d_gb300 import token_ops
    return token_ops._bind()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) >= {"rms_norm_quant_fwd", "act_quant_fwd", "linear_w8a8_fwd",
                          "linear_w8a8_workspace_size"}
    assert not [n for n in names if not hasattr(lib, n)]


def _norm(lib, **kw):
    a = dict(x=P, x_dtype=BF16, x_stride=64, residual=None, res_dtype=0, res_stride=0, weight=None,
             weight_dtype=0, eps=1e-6, tokens=2, width=64, q_dtype=INT8, q=P, q_stride=64, scale=P,
             residual_out=None, res_out_stride=0)
    a.update(kw)
    return lib.rms_norm_quant_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(q=None), dict(scale=None), dict(x_dtype=INT8), dict(q_dtype=BF16),
    dict(tokens=-1), dict(width=0), dict(width=1 << 31), dict(x_stride=63), dict(q_stride=10),
    dict(x=P + 1), dict(scale=P + 2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(residual=P, res_dtype=F16, res_stride=64), dict(residual=P, res_dtype=BF16, res_stride=3),
    dict(residual=P + 1, res_dtype=BF16, res_stride=64), dict(residual_out=P, res_out_stride=64),
    dict(weight=P, weight_dtype=F16), dict(weight=P + 2, weight_dtype=F32),
    dict(residual=P, res_dtype=F32, res_stride=64, residual_out=P + 2, res_out_stride=64)])
def test_norm_refuses(lib, kw):
    assert _norm(lib, **kw) == INVALID
    assert lib.conv_last_error()


def test_zero_tokens_are_valid(lib):
    assert _norm(lib, tokens=0, x=None, q=None, scale=None) == 0
    assert _act(lib, tokens=0, x=None, q=None, scale=None) == 0
    assert _linear(lib, tokens=0, x=None, out=None) == 0
    assert _linear(lib, outputs=0, w=None, out=None) == 0


def _act(lib, **kw):
    a = dict(x=P, x_dtype=BF16, x_stride=128, act=2, gated=1, tokens=2, width=64, q_dtype=INT8,
             q=P, q_stride=64, scale=P)
    a.update(kw)
    return lib.act_quant_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(q=None), dict(scale=None), dict(act=4), dict(act=-1), dict(x_dtype=E4M3),
    dict(q_dtype=F32), dict(tokens=-2), dict(width=0), dict(x_stride=127), dict(q_stride=63),
    dict(x=P + 1)])
def test_act_refuses(lib, kw):
    assert _act(lib, **kw) == INVALID


def _linear(lib, **kw):
    a = dict(x=P, x_stride=64, w=P, w_stride=64, dtype=INT8, tokens=2, outputs=8, width=64,
             scale_x=None, scale_w=None, bias=None, act=0, out=P, out_dtype=BF16, out_stride=8,
             workspace=None, workspace_bytes=0)
    a.update(kw)
    return lib.linear_w8a8_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(out=None), dict(dtype=BF16), dict(out_dtype=INT8),
    dict(act=7), dict(tokens=-1), dict(outputs=-1), dict(width=0), dict(width=1 << 31),
    dict(x_stride=63), dict(w_stride=63), dict(out_stride=7), dict(out=P + 1),
    dict(scale_x=P + 1), dict(scale_w=P + 2), dict(bias=P + 3)])
def test_linear_refuses(lib, kw):
    assert _linear(lib, **kw) == INVALID


def test_few_tokens_need_no_workspace(lib):
    """The binding's constant is the header's, and what the library answers."""
    from implicit_gemm_convolution_conv3d_gb300 import token_ops
    n = token_ops.NO_WORKSPACE_TOKENS
    assert f"#define LINEAR_W8A8_NO_WORKSPACE_TOKENS {n}" in open(HEADER).read()
    for dtype in (INT8, E4M3):
        for off in (0, 1):
            size = lambda t: lib.linear_w8a8_workspace_size(P + off, 65, P + off, 65, dtype, t, 8, 65)   # noqa: E731
            assert all(size(t) == 0 for t in (1, 2, n))
            assert size(n + 1) == 80 * (n + 1 + 8)


def test_cpu_tensors_are_refused():
    import implicit_gemm_convolution_conv3d_gb300 as p
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        p.rms_norm_quant(x)
    with pytest.raises(ValueError):
        p.act_quant(x)
    with pytest.raises(ValueError):
        p.linear_w8a8(x.to(torch.int8), x.to(torch.int8))
