"""The attention operators' C ABI without a GPU: exported symbols, argument checks that
return before anything is launched, and the binding's own."""
import ctypes
import os
import re

import pytest
import torch

from implicit_gemm_convolution_conv3d_gb300 import build as pkg_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "token_attention.h")
BF16, E4M3, INT8, F16, F32 = 0, 1, 2, 3, 4
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 4096   # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    from implicit_gemm_convolution_conv3d_gb300 import token_attention
    return token_attention._bind()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == {"rotary_fwd", "kv_cache_write", "kv_cache_read", "paged_attention_fwd",
                          "paged_attention_workspace_size", "packed_attention_fwd"}
    assert not [n for n in names if not hasattr(lib, n)]
    from implicit_gemm_convolution_conv3d_gb300 import token_attention as t
    assert f"ROTARY_MAX_PAIRS {t.MAX_PAIRS}" in open(HEADER).read()
    assert f"ROTARY_MAX_AXES {t.MAX_AXES}" in open(HEADER).read()


def _rotary(lib, axis=(0, 0, 1), frequency=(1.0, 0.5, 0.25), **kw):
    a = dict(x=P, dtype=BF16, xt=128, xh=64, positions=P, position_bytes=4, axes=2,
             axis=(ctypes.c_int * 3)(*axis), frequency=(ctypes.c_double * 3)(*frequency), pairs=3,
             interleaved=0, inverse=0, tokens=4, heads=2, width=64, out=P, ot=128, oh=64)
    a.update(kw)
    return lib.rotary_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(out=None), dict(positions=None), dict(dtype=INT8), dict(position_bytes=2),
    dict(axes=0), dict(axes=9), dict(pairs=0), dict(pairs=129), dict(pairs=33), dict(tokens=-1),
    dict(heads=-1), dict(width=0), dict(xh=63), dict(ot=63), dict(x=P + 1), dict(positions=P + 2),
    dict(axis=(0, 2, 0)), dict(axis=(0, -1, 0)), dict(frequency=(1.0, float("inf"), 0.0))])
def test_rotary_refuses(lib, kw):
    assert _rotary(lib, **kw) == INVALID and lib.conv_last_error()


def _cache(**kw):
    from implicit_gemm_convolution_conv3d_gb300.token_attention import _Cache
    a = dict(k=P, v=2 * P, k_scale=P, v_scale=2 * P, dtype=INT8, pages=4, heads=2, page_size=16, width=64,
             page_stride=2048, head_stride=1024, row_stride=64, scale_page_stride=32, scale_head_stride=16)
    a.update(kw)
    return _Cache(**a)


BAD_CACHES = [dict(k=None), dict(k_scale=None), dict(k=P + 8), dict(dtype=F32), dict(width=24), dict(width=272),
              dict(width=0), dict(row_stride=48), dict(row_stride=72), dict(head_stride=1000), dict(pages=0),
              dict(heads=0), dict(page_size=0), dict(k_scale=P + 2), dict(scale_page_stride=-1),
              dict(row_stride=1 << 27)]


def _rows(lib, write, cache, **kw):
    a = dict(k=P, v=2 * P, dtype=BF16, ts=128, hs=64, tokens=5, offsets=P, starts=P, table=P, tstride=8, tpages=8,
             sequences=3)
    a.update(kw)
    f = lib.kv_cache_write if write else lib.kv_cache_read
    return f(cache, *a.values(), None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(dtype=INT8), dict(ts=63), dict(hs=32), dict(tokens=-1), dict(sequences=-1),
    dict(table=None), dict(table=P + 2), dict(tstride=7), dict(tpages=-1), dict(offsets=P + 1), dict(starts=P + 2),
    dict(k=P + 1)])
def test_rows_refused(lib, write, kw):
    assert _rows(lib, write, _cache(), **kw) == INVALID


def test_more_refusals_of_rows(lib):
    for kw in BAD_CACHES:
        for write in (True, False):
            assert _rows(lib, write, _cache(**kw)) == INVALID, kw
    assert _rows(lib, True, _cache(), offsets=None) == INVALID           # 5 rows, 3 sequences
    assert _rows(lib, True, _cache(), starts=None) == INVALID
    assert _rows(lib, False, _cache(), offsets=None) == INVALID
    half = _cache(dtype=F16, k_scale=None, v_scale=None)
    assert _rows(lib, True, half, dtype=BF16) == INVALID                 # rows of the cache's type only
    assert _rows(lib, True, _cache(heads=1 << 20), tokens=1 << 30, ts=1 << 40) in (INVALID, UNSUPPORTED)


def _paged(lib, cache, **kw):
    a = dict(q=P, dtype=BF16, qs=256, qh=64, cache=cache, table=P, tstride=8, tpages=8, lengths=P, prefix=None,
             slopes=None, scale=0.125, cap=0.0, window=0, sequences=3, heads=4, out=P, os=256, oh=64,
             workspace=P, bytes=1 << 30)
    a.update(kw)
    return lib.paged_attention_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(lengths=None), dict(dtype=F32), dict(heads=3), dict(heads=0), dict(qh=32),
    dict(os=100), dict(q=P + 1), dict(lengths=P + 1), dict(prefix=P + 2), dict(slopes=P + 1), dict(table=None),
    dict(tstride=2), dict(sequences=-1), dict(scale=float("nan")), dict(cap=-1.0), dict(cap=1e-30),
    dict(cap=float("inf")), dict(window=-1)])
def test_paged_refuses(lib, kw):
    assert _paged(lib, _cache(), **kw) == INVALID


def test_paged_refuses_caches(lib):
    for kw in BAD_CACHES:
        assert _paged(lib, _cache(**kw)) == INVALID, kw
    assert _paged(lib, _cache(dtype=F16, k_scale=None, v_scale=None)) == INVALID   # bf16 queries
    for a in ((0, 4, 2, 64, 16, 8), (3, 5, 2, 64, 16, 8), (3, 4, 2, 512, 16, 8), (3, 4, 0, 64, 16, 8)):
        assert lib.paged_attention_workspace_size(*a) == 0


def _packed(lib, **kw):
    a = dict(q=P, qt=256, qh=64, k=P, v=P, kt=128, kh=64, dtype=BF16, qo=P, ko=P, documents=2, nq=8, nk=8,
             heads=4, kv_heads=2, width=64, causal=0, window=0, prefix=None, slopes=None, scale=0.125, cap=0.0,
             out=2 * P, ot=256, oh=64)
    a.update(kw)
    return lib.packed_attention_fwd(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(qo=None), dict(ko=None), dict(dtype=F32),
    dict(dtype=INT8), dict(width=60), dict(width=136), dict(width=0), dict(heads=3), dict(kv_heads=0), dict(qt=60),
    dict(kh=32), dict(q=P + 8), dict(v=P + 2), dict(qt=260), dict(kh=68), dict(documents=-1), dict(nq=-1),
    dict(nk=1 << 31), dict(qo=P + 2), dict(prefix=P + 1), dict(slopes=P + 2), dict(cap=-0.5), dict(window=-3),
    dict(scale=float("inf")), dict(out=P + 1)])
def test_packed_refuses(lib, kw):
    assert _packed(lib, **kw) == INVALID


def test_nothing_to_do_is_valid(lib):
    assert _rotary(lib, tokens=0, x=None, out=None, positions=None) == OK
    assert _rotary(lib, heads=0, x=None, out=None) == OK
    for write in (True, False):
        assert _rows(lib, write, _cache(), tokens=0, sequences=0, k=None, v=None, table=None, offsets=None, starts=None) == OK
    assert _paged(lib, _cache(), sequences=0, q=None, out=None, lengths=None, table=None, workspace=None) == OK
    assert _packed(lib, documents=0, q=None, out=None) == OK
    assert _packed(lib, nq=0, q=None, out=None) == OK


def test_cpu_tensors_are_refused():
    import implicit_gemm_convolution_conv3d_gb300 as p
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    pool, table = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        p.rotary(x, n, (4,))
    with pytest.raises(ValueError):
        p.kv_cache_write(x, x, pool, pool, table, n)
    with pytest.raises(ValueError):
        p.kv_cache_read(pool, pool, table, n, tokens=2)
    with pytest.raises(ValueError):
        p.paged_attention(x, pool, pool, table, n)
    with pytest.raises(ValueError):
        p.packed_attention(x, x, x, n)


def test_ladders():
    """Pairs' axes and radians: each axis its own ladder, or one over all."""
    from implicit_gemm_convolution_conv3d_gb300.token_attention import _ladder
    n, axis, freq = _ladder((2, 0, 3), 100.0, "axis", None, None)
    assert n == 5 and list(axis) == [0, 0, 2, 2, 2]
    assert list(freq) == [1.0, 100.0 ** -0.5, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)]
    _, _, freq = _ladder((2, 3), 100.0, "shared", (0.5, 2.0), None)
    assert list(freq) == [0.5 * 1.0, 0.5 * 100.0 ** -0.2] + [2.0 * 100.0 ** (-i / 5) for i in (2, 3, 4)]
    _, _, freq = _ladder((1, 1), 10.0, "axis", None, (3.0, -2.0))
    assert list(freq) == [3.0, -2.0]


def test_overlapping_outputs_and_caches(lib):
    """Rows that lie in one another are refused where they are written; heads outside
    tokens, or tokens outside heads, are not."""
    assert _rotary(lib, ot=64, oh=64) == INVALID
    assert _rotary(lib, ot=64, oh=192) == INVALID                        # 4 tokens a head: 256
    assert _rows(lib, False, _cache(), ts=64, hs=64) == INVALID
    for kw in (dict(head_stride=960), dict(head_stride=0), dict(page_stride=0), dict(page_stride=1024),
               dict(scale_head_stride=8), dict(scale_page_stride=16), dict(row_stride=96)):
        assert _rows(lib, True, _cache(**kw)) == INVALID, kw
    assert _rows(lib, True, _cache(v=P, k=P), k=P, v=2 * P) == INVALID    # one pool for both
    assert _rows(lib, False, _cache(), k=P, v=P) == INVALID
    assert _packed(lib, out=2 * P, q=2 * P, ot=256) == INVALID
    inside = _cache(row_stride=128, head_stride=64, scale_page_stride=64, scale_head_stride=32)
    assert _rows(lib, True, inside, tokens=0, sequences=0) == OK


def test_one_device(monkeypatch):
    from implicit_gemm_convolution_conv3d_gb300 import token_attention as t

    class At:
        def __init__(self, i):
            self.device = torch.device("cuda", i)

        def get_device(self):
            return self.device.index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    t._here(At(1), At(1), None)
    with pytest.raises(ValueError, match="current"):
        t._here(At(0), At(0))
    with pytest.raises(ValueError, match="all tensors"):
        t._here(At(1), None, At(0))
