"""layer_norm and layer_norm_grad refuse what they cannot do, on the host,
before anything is enqueued. No GPU is used: the addresses are never
dereferenced."""
import ctypes
import math

import pytest
import torch

import gradient_compression_quantize_amd as gcq
from test_binding import FakeStream
from test_training_ops_refusals import FakeShape

FAKE = 0x10000
S = FakeStream()


@pytest.fixture(scope="module")
def lib():
    return gcq.load()


def norm(lib, **kw):
    a = dict(x=FAKE, y=FAKE, dt=0, rows=4, d=8, gain=FAKE, bias=FAKE, eps=1e-5, p=0.0, step=None, z=FAKE, h=FAKE,
             mean=FAKE, rstd=FAKE) | kw
    return lib.layer_norm(a["x"], a["y"], a["dt"], a["rows"], a["d"], a["gain"], a["bias"], a["eps"], a["p"], 0, 0,
                          a["step"], a["z"], a["h"], a["mean"], a["rstd"], None)


def test_layer_norm_refusals(lib):
    for bad in (dict(x=None), dict(h=None), dict(y=None), dict(d=0), dict(dt=3), dict(dt=-1), dict(eps=-1.0),
                dict(eps=math.nan), dict(p=-0.1), dict(p=1.5), dict(p=math.nan), dict(x=FAKE + 2), dict(y=FAKE + 1),
                dict(z=FAKE + 2), dict(h=FAKE + 2), dict(gain=FAKE + 2), dict(bias=FAKE + 1), dict(mean=FAKE + 2),
                dict(rstd=FAKE + 3), dict(step=FAKE + 4), dict(dt=1, h=FAKE + 1)):
        assert norm(lib, **bad) == gcq.GC_EINVAL, bad
        assert b"layer_norm" in lib.gc_last_error()
    assert norm(lib, d=16385) == gcq.GC_EUNSUPPORTED
    assert norm(lib, rows=2 ** 41) == gcq.GC_EUNSUPPORTED
    assert norm(lib, rows=0) == gcq.GC_OK


def norm_grad(lib, size=None, **kw):
    a = dict(z=FAKE, dh=FAKE, dz=FAKE, dt=0, rows=4, d=8, gain=FAKE, p=0.0, step=None, mean=FAKE, rstd=FAKE, dx=FAKE,
             dy=FAKE, dgain=FAKE, dbias=FAKE, ws=FAKE) | kw
    n = ctypes.c_size_t(1 << 30 if size is None else size)
    rc = lib.layer_norm_grad(a["z"], a["dh"], a["dz"], a["dt"], a["rows"], a["d"], a["gain"], a["p"], 0, 0, a["step"],
                             a["mean"], a["rstd"], a["dx"], a["dy"], a["dgain"], a["dbias"], a["ws"], ctypes.byref(n),
                             None)
    return rc, n.value


def test_layer_norm_grad_refusals(lib):
    for bad in (dict(z=None), dict(dh=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(d=0), dict(dt=7),
                dict(p=2.0), dict(step=FAKE + 2), dict(z=FAKE + 2), dict(dz=FAKE + 1), dict(dy=FAKE + 2),
                dict(dgain=FAKE + 2), dict(dbias=FAKE + 1), dict(ws=FAKE + 8), dict(size=16)):
        assert norm_grad(lib, **bad)[0] == gcq.GC_EINVAL, bad
    assert norm_grad(lib, d=20000)[0] == gcq.GC_EUNSUPPORTED
    rc, size = norm_grad(lib, ws=None)
    assert rc == gcq.GC_OK and 0 < size < 1 << 12
    rc, size = norm_grad(lib, ws=None, rows=0)
    assert rc == gcq.GC_OK and size > 0
    assert lib.layer_norm_grad(FAKE, FAKE, None, 0, 4, 8, None, 0.0, 0, 0, None, FAKE, FAKE, FAKE, None, None, None, FAKE,
                               None, None) == gcq.GC_EINVAL


def test_binding_checks():
    d = lambda *s, **k: FakeShape(s, **k)  # noqa: E731
    ws = d(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="differ in size"):
        gcq.layer_norm(d(4, 8), d(4, 7), stream=S)
    with pytest.raises(ValueError, match="differ in size"):
        gcq.layer_norm(d(4, 8), d(4, 8), y=d(3, 8), stream=S)
    with pytest.raises(ValueError, match="one value a column"):
        gcq.layer_norm(d(4, 8), d(4, 8), bias=d(4), stream=S)
    with pytest.raises(ValueError, match="one value a row"):
        gcq.layer_norm(d(4, 8), d(4, 8), rstd=d(8), stream=S)
    with pytest.raises(ValueError, match="at least one value"):
        gcq.layer_norm(d(4, 0), d(4, 0), stream=S)
    with pytest.raises(TypeError, match="gain: expected"):
        gcq.layer_norm(d(4, 8), d(4, 8), gain=d(8, dtype=torch.bfloat16), stream=S)
    with pytest.raises(TypeError, match="h: expected"):
        gcq.layer_norm(d(4, 8, dtype=torch.bfloat16), d(4, 8), stream=S)
    with pytest.raises(gcq.GcqError, match="z without y"):
        gcq.layer_norm(d(4, 8), d(4, 8), z=d(4, 8), stream=S)
    stats = dict(mean=d(4), rstd=d(4), stream=S)
    with pytest.raises(ValueError, match="differ in size"):
        gcq.layer_norm_grad(d(4, 8), d(4, 8), d(4, 9), ws, **stats)
    with pytest.raises(ValueError, match="one value a column"):
        gcq.layer_norm_grad(d(4, 8), d(4, 8), d(4, 8), ws, dgain=d(9), **stats)
    with pytest.raises(ValueError, match="ws too small"):
        gcq.layer_norm_grad(d(4, 8), d(4, 8), d(4, 8), d(0, dtype=torch.uint8), **stats)
    with pytest.raises(gcq.GcqError, match="workspace too small"):
        gcq.layer_norm_grad(d(4, 8), d(4, 8), d(4, 8), d(16, dtype=torch.uint8), **stats)
    with pytest.raises(gcq.GcqError, match="NULL"):
        gcq.layer_norm_grad(d(4, 8), d(4, 8), d(4, 8), ws, stream=S)
