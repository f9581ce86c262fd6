"""Where the token operators' tensors come from, without a GPU: what a call on a
given stream allocates is that stream's memory."""
import contextlib
import types

import pytest


class _FakeTorch:
    """Records which stream is current at each allocation."""

    def __init__(self):
        self.log, self.current = [], ["main"]
        self.cuda = types.SimpleNamespace(
            stream=self._stream, current_stream=lambda device=None: self.current[-1])

    @contextlib.contextmanager
    def _stream(self, s):
        self.current.append(s)
        yield
        self.current.pop()

    def empty(self, shape, dtype=None, device=None):
        self.log.append(("empty", self.current[-1]))
        return types.SimpleNamespace(record_stream=lambda s: self.log.append(("record", s)))


@pytest.fixture
def fake(monkeypatch):
    from implicit_gemm_convolution_conv3d_gb300 import token_ops
    f = _FakeTorch()
    monkeypatch.setattr(token_ops, "torch", f)
    return token_ops, f


X = types.SimpleNamespace(device="cuda:0")


def test_current_stream_allocates_from_its_own_pool(fake):
    ops, f = fake
    ops._new((4,), None, X, None)
    assert f.log == [("empty", "main")]


def test_given_stream_allocates_from_its_own_pool(fake):
    """Memory that was freed on the current stream may still be in use there: the
    given stream must not get it; and the caller's stream, which the result is
    handed to, is recorded."""
    ops, f = fake
    ops._new((4,), None, X, "side")
    assert f.log == [("empty", "side"), ("record", "main")]
    assert f.current == ["main"]
