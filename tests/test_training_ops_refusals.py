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


def norm(lib, **kw):
    a = dict(x=FAKE, y=FAKE, dt=0, rows=4, d=8, post=FAKE, gate=FAKE, gates=2, pre=FAKE, s=1.0, eps=1e-6, p=0.0,
             step=None, z=FAKE, h=FAKE, rp=FAKE, rz=FAKE) | kw
    return lib.norm_residual(a["x"], a["y"], a["dt"], a["rows"], a["d"], a["post"], a["gate"], a["gates"], a["pre"],
                             a["s"], a["eps"], a["p"], 0, 0, a["step"], a["z"], a["h"], a["rp"], a["rz"], None)


def test_norm_residual_refusals(lib):
    for bad in (dict(x=None), dict(y=None), dict(z=None), dict(h=None), dict(rp=None), dict(rz=None), dict(d=0),
                dict(gates=3), dict(gates=0), dict(dt=7), dict(eps=-1.0), dict(eps=math.nan), dict(p=2.0),
                dict(x=FAKE + 2), dict(gate=FAKE + 1), dict(step=FAKE + 2), dict(dt=1, h=FAKE + 1), dict(pre=None)):
        assert norm(lib, **bad) == gcq.GC_EINVAL, bad
    assert norm(lib, d=16385) == gcq.GC_EUNSUPPORTED
    assert norm(lib, rows=0) == gcq.GC_OK


def norm_grad(lib, size=None, **kw):
    a = dict(z=FAKE, y=FAKE, dt=0, rows=4, d=8, post=FAKE, gate=FAKE, gates=2, pre=FAKE, p=0.0, step=None, rp=FAKE,
             rz=FAKE, dz=FAKE, dh=FAKE, dx=FAKE, dy=FAKE, dpost=FAKE, dgate=FAKE, dpre=FAKE, ws=FAKE) | kw
    n = ctypes.c_size_t(1 << 30 if size is None else size)
    rc = lib.norm_residual_grad(a["z"], a["y"], a["dt"], a["rows"], a["d"], a["post"], a["gate"], a["gates"], a["pre"],
                                1.0, a["p"], 0, 0, a["step"], a["rp"], a["rz"], a["dz"], a["dh"], a["dx"], a["dy"],
                                a["dpost"], a["dgate"], a["dpre"], a["ws"], ctypes.byref(n), None)
    return rc, n.value


def test_norm_residual_grad_refusals(lib):
    for bad in (dict(z=None), dict(y=None), dict(dx=None), dict(dy=None), dict(dh=None), dict(pre=None),
                dict(post=None), dict(gate=None), dict(rp=None), dict(rz=None), dict(dz=None, dh=None, pre=None, dpre=None),
                dict(d=0), dict(gates=3), dict(dt=-1), dict(p=-1.0), dict(dx=FAKE + 2), dict(dpost=FAKE + 2),
                dict(ws=FAKE + 8), dict(size=16)):
        assert norm_grad(lib, **bad)[0] == gcq.GC_EINVAL, bad
    assert norm_grad(lib, d=20000)[0] == gcq.GC_EUNSUPPORTED
    rc, size = norm_grad(lib, ws=None)
    assert rc == gcq.GC_OK and 0 < size < 1 << 16


def test_norm_residual_binding_checks():
    d = lambda *s, **k: FakeShape(s, **k)  # noqa: E731
    with pytest.raises(ValueError, match="differ in size"):
        gcq.norm_residual(d(4, 8), d(4, 8), d(4, 7), stream=S)
    with pytest.raises(ValueError, match="gain"):
        gcq.norm_residual(d(4, 8), d(4, 8), d(4, 8), post_gain=d(4), stream=S)
    with pytest.raises(ValueError, match="one value a row"):
        gcq.norm_residual(d(4, 8), d(4, 8), d(4, 8), post_gain=d(8), rstd_post=d(3), stream=S)
    with pytest.raises(ValueError, match="gate must"):
        gcq.norm_residual(d(4, 8), d(4, 8), d(4, 8), gate=d(3, 8), stream=S)
    with pytest.raises(TypeError, match="gate: expected"):
        gcq.norm_residual(d(4, 8), d(4, 8), d(4, 8), gate=d(2, 8, dtype=torch.bfloat16), stream=S)
    with pytest.raises(ValueError, match="dgate"):
        gcq.norm_residual_grad(d(4, 8), d(4, 8), d(4, 8), d(4, 8), d(64, dtype=torch.uint8), dz=d(4, 8), gate=d(2, 8),
                               dgate=d(1, 8), stream=S)


class FakeShape(FakeDev):
    """FakeDev with a shape."""

    def __init__(self, shape, dtype=torch.float32):
        super().__init__(math.prod(shape), dtype)
        self.shape = shape

    def dim(self):
        return len(self.shape)


def xent(lib, size=None, ws=FAKE, **kw):
    a = dict(h=FAKE, w=FAKE, dt=1, N=4, V=8, D=64, y=FAKE, loss=FAKE, lse=FAKE) | kw
    n = ctypes.c_size_t(1 << 30 if size is None else size)
    rc = lib.linear_xent_loss(a["h"], a["w"], a["dt"], a["N"], a["V"], a["D"], a["y"], -100, a["loss"], a["lse"], ws,
                              ctypes.byref(n), None)
    return rc, n.value


def test_linear_xent_loss_refusals(lib):
    for bad in (dict(h=None), dict(w=None), dict(y=None), dict(loss=None), dict(lse=None), dict(V=0), dict(D=0),
                dict(dt=5), dict(h=FAKE + 1), dict(w=FAKE + 2, dt=0), dict(y=FAKE + 4), dict(lse=FAKE + 2),
                dict(ws=FAKE + 4), dict(size=8)):
        assert xent(lib, **bad)[0] == gcq.GC_EINVAL, bad
    for big in (dict(N=2 ** 28 + 1), dict(V=2 ** 28 + 1), dict(D=2 ** 20 + 1), dict(N=2 ** 24, V=2 ** 24)):
        assert xent(lib, **big)[0] == gcq.GC_EUNSUPPORTED, big
    assert xent(lib, N=0)[0] == gcq.GC_OK
    rc, size = xent(lib, ws=None, N=8192, V=30522, D=768)
    assert rc == gcq.GC_OK and size < 1 << 28
    assert lib.linear_xent_loss(FAKE, FAKE, 1, 4, 8, 64, FAKE, 0, FAKE, FAKE, FAKE, None, None) == gcq.GC_EINVAL


def xent_grad(lib, size=None, ws=FAKE, **kw):
    a = dict(h=FAKE, w=FAKE, dt=1, N=4, V=8, D=64, y=FAKE, lse=FAKE, dl=FAKE, dh=FAKE, th=1, dw=FAKE, tw=0) | kw
    n = ctypes.c_size_t(1 << 40 if size is None else size)
    rc = lib.linear_xent_grad(a["h"], a["w"], a["dt"], a["N"], a["V"], a["D"], a["y"], -100, a["lse"], a["dl"], a["dh"],
                              a["th"], a["dw"], a["tw"], ws, ctypes.byref(n), None)
    return rc, n.value


def test_linear_xent_grad_refusals(lib):
    for bad in (dict(h=None), dict(w=None), dict(y=None), dict(lse=None), dict(dl=None), dict(V=0), dict(D=0),
                dict(dt=4), dict(th=2), dict(tw=2), dict(dt=0, th=1), dict(dh=FAKE + 1), dict(dw=FAKE + 2),
                dict(dl=FAKE + 2), dict(ws=FAKE + 8), dict(size=64)):
        assert xent_grad(lib, **bad)[0] == gcq.GC_EINVAL, bad
    assert xent_grad(lib, V=2 ** 28 + 1)[0] == gcq.GC_EUNSUPPORTED
    assert xent_grad(lib, dh=None, dw=None)[0] == gcq.GC_OK
    rc, size = xent_grad(lib, ws=None, N=8192, V=10 ** 6, D=1024)
    # G of one piece, not of the whole vocabulary
    assert rc == gcq.GC_OK and size < 3 * 10 ** 9 < 8192 * 10 ** 6 * 2


def test_linear_xent_binding_checks():
    d = lambda *s, **k: FakeShape(s, **k)  # noqa: E731
    y, ws = d(4, dtype=torch.int64), d(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="weight"):
        gcq.linear_xent_loss(d(4, 8), d(16, 7), y, d(4), d(4), ws, stream=S)
    with pytest.raises(ValueError, match="one value a token"):
        gcq.linear_xent_loss(d(4, 8), d(16, 8), y, d(3), d(4), ws, stream=S)
    with pytest.raises(TypeError, match="weight: expected"):
        gcq.linear_xent_loss(d(4, 8), d(16, 8, dtype=torch.bfloat16), y, d(4), d(4), ws, stream=S)
    with pytest.raises(TypeError, match="int64"):
        gcq.linear_xent_loss(d(4, 8), d(16, 8), d(4, dtype=torch.int32), d(4), d(4), ws, stream=S)
    with pytest.raises(ValueError, match="dhidden differs"):
        gcq.linear_xent_grad(d(4, 8), d(16, 8), y, d(4), d(4), d(3, 8), None, ws, stream=S)
    with pytest.raises(ValueError, match="dweight differs"):
        gcq.linear_xent_grad(d(4, 8), d(16, 8), y, d(4), d(4), None, d(15, 8), ws, stream=S)
    with pytest.raises(gcq.GcqError, match="inputs' type or fp32"):
        gcq.linear_xent_grad(d(4, 8), d(16, 8), y, d(4), d(4), d(4, 8, dtype=torch.bfloat16), None, ws, stream=S)
    with pytest.raises(gcq.GcqError, match="workspace too small"):
        gcq.linear_xent_loss(d(4, 8), d(16, 8), y, d(4), d(4), d(16, dtype=torch.uint8), stream=S)
