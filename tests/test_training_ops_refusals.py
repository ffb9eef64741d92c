"""The training operators refuse what they cannot do, on the host, before
anything is enqueued. No GPU is used: the addresses are never dereferenced."""
import ctypes
import math

import pytest
import torch

import gradient_compression_quantize_amd as gcq
from test_binding import FakeDev, FakeStream

FAKE = 0x10000
S = FakeStream()


@pytest.fixture(scope="module")
def lib():
    return gcq.load()


@pytest.mark.parametrize("p", [-0.1, 1.5, math.nan, math.inf])
def test_dropout_refuses_p(lib, p):
    assert lib.dropout(FAKE, None, 16, 0, p, 0, 0, 0, None, FAKE, None) == gcq.GC_EINVAL
    assert b"p must" in lib.gc_last_error()
    assert lib.dropout_backward(FAKE, 16, 0, p, 0, 0, 0, None, FAKE, None) == gcq.GC_EINVAL


def test_dropout_refuses_buffers_types_and_ranges(lib):
    def call(x=FAKE, r=None, n=16, dt=0, off=0, step=None, out=FAKE):
        return lib.dropout(x, r, n, dt, 0.5, 0, 0, off, step, out, None)
    for bad in (dict(x=None), dict(out=None), dict(x=FAKE + 2), dict(out=FAKE + 1, dt=1), dict(r=FAKE + 2),
                dict(dt=3), dict(dt=-1), dict(off=2 ** 64 - 8), dict(step=FAKE + 4)):
        assert call(**bad) == gcq.GC_EINVAL, bad
    assert call(n=0, x=None, out=None) == gcq.GC_OK


def test_dropout_binding_checks():
    with pytest.raises(ValueError, match="differ in size"):
        gcq.dropout(FakeDev(8), 0.5, 0, 0, FakeDev(9), stream=S)
    with pytest.raises(ValueError, match="differ in size"):
        gcq.dropout_backward(FakeDev(8), 0.5, 0, 0, FakeDev(7), stream=S)
    with pytest.raises(TypeError, match="out: expected"):
        gcq.dropout(FakeDev(8, torch.bfloat16), 0.5, 0, 0, FakeDev(8), stream=S)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        gcq.dropout(FakeDev(8, torch.float64), 0.5, 0, 0, FakeDev(8, torch.float64), stream=S)
    with pytest.raises(ValueError, match="worker"):
        gcq.dropout(FakeDev(8), 0.5, 0, -1, FakeDev(8), stream=S)
    with pytest.raises(ValueError, match="offset"):
        gcq.dropout(FakeDev(8), 0.5, 0, 0, FakeDev(8), offset=-4, stream=S)
    with pytest.raises(ValueError, match="step must hold one"):
        gcq.dropout(FakeDev(8), 0.5, 0, 0, FakeDev(8), step=FakeDev(2, torch.int64), stream=S)
    with pytest.raises(TypeError, match="int64"):
        gcq.dropout(FakeDev(8), 0.5, 0, 0, FakeDev(8), step=FakeDev(1), stream=S)
    with pytest.raises(TypeError, match="contiguous"):
        gcq.dropout(FakeDev(8, contiguous=False), 0.5, 0, 0, FakeDev(8), stream=S)
