"""orthogonalize and muon_step refuse what they cannot do, on the host, before
anything is enqueued. No GPU is used: the addresses are never dereferenced."""
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


def pointers(*p):
    return (ctypes.c_void_p * max(len(p), 1))(*p)


def floats(*v):
    return (ctypes.c_float * len(v))(*v)


ONE = floats(1.5, -0.5, 0.0)


def orth(lib, size=None, **kw):
    a = dict(x=pointers(FAKE, FAKE), count=2, m=256, n=300, dt=0, coef=ONE, steps=1, eps=1e-7, scale=1.0,
             out=pointers(FAKE, FAKE), odt=1, ws=FAKE) | kw
    n = ctypes.c_size_t(1 << 30 if size is None else size)
    rc = lib.orthogonalize(a["x"], a["count"], a["m"], a["n"], a["dt"], a["coef"], a["steps"], a["eps"], a["scale"],
                           a["out"], a["odt"], a["ws"], ctypes.byref(n), None)
    return rc, n.value


def test_orthogonalize_refusals(lib):
    for bad in (dict(x=None), dict(out=None), dict(x=pointers(FAKE, None)), dict(out=pointers(None, FAKE)),
                dict(x=pointers(FAKE, FAKE + 2)), dict(dt=1, x=pointers(FAKE + 1, FAKE)), dict(out=pointers(FAKE, FAKE + 1)),
                dict(odt=0, out=pointers(FAKE, FAKE + 2)), dict(count=0), dict(count=-1), dict(count=65), dict(dt=3),
                dict(odt=-1), dict(coef=None), dict(steps=0), dict(steps=65), dict(steps=-3), dict(eps=-1e-9),
                dict(eps=math.nan), dict(eps=math.inf), dict(coef=floats(1.0, math.nan, 0.0)),
                dict(coef=floats(math.inf, 0.0, 0.0)), dict(ws=FAKE + 8), dict(size=1024)):
        assert orth(lib, **bad)[0] == gcq.GC_EINVAL, bad
        assert b"orthogonalize" in lib.gc_last_error()
    for big in (dict(m=2 ** 20 + 1), dict(n=2 ** 20 + 1), dict(m=2 ** 15 + 1, n=2 ** 15 + 1),
                dict(count=64, m=2 ** 15, n=2 ** 20)):
        assert orth(lib, ws=None, **big)[0] == gcq.GC_EUNSUPPORTED, big
    assert orth(lib, m=0)[0] == gcq.GC_OK
    assert orth(lib, n=0, size=0)[0] == gcq.GC_OK
    assert lib.orthogonalize(pointers(FAKE), 1, 8, 8, 0, ONE, 1, 0.0, 1.0, pointers(FAKE), 1, FAKE, None,
                             None) == gcq.GC_EINVAL


def test_workspace_sizes():
    one, two = (gcq.orthogonalize_ws_bytes(k, 4096, 4096, torch.bfloat16) for k in (1, 2))
    # two copies of X in two planes of 16 bits, A and P in one
    assert 2 * 4 * 2 ** 24 + 2 * 2 * 2 ** 24 <= one < 1.01 * (12 * 2 ** 24) and one < two <= 2 * one
    assert gcq.orthogonalize_ws_bytes(1, 4096, 4096, torch.float32) > one
    assert gcq.muon_step_ws_bytes(3, 100, 70, torch.float32) == gcq.orthogonalize_ws_bytes(3, 100, 70, torch.float32)
    assert gcq.orthogonalize_ws_bytes(1, 0, 5, torch.float32) > 0
    # what one workgroup holds needs none to speak of
    assert gcq.orthogonalize_ws_bytes(64, 64, 576, torch.bfloat16) == 256
    # sizes past 32 bits
    assert gcq.orthogonalize_ws_bytes(64, 2 ** 15, 2 ** 15, torch.bfloat16) > 64 * 8 * 2 ** 30
    with pytest.raises(gcq.GcqError, match="1 .. 64"):
        gcq.orthogonalize_ws_bytes(65, 8, 8, torch.float32)


def step(lib, size=None, **kw):
    p = pointers(FAKE)
    a = dict(g=p, count=1, m=256, n=300, m0=p, w=p, dt=0, udt=0, coef=ONE, steps=1, eps=1e-7, gs=1.0, beta=0.9, nest=1,
             lr=0.1, ls=FAKE, wd=0.0, us=1.0, m1=p, w1=p, ws=FAKE) | kw
    n = ctypes.c_size_t(1 << 30 if size is None else size)
    rc = lib.muon_step(a["g"], a["count"], a["m"], a["n"], a["m0"], a["w"], a["dt"], a["udt"], a["coef"], a["steps"],
                       a["eps"], a["gs"], a["beta"], a["nest"], a["lr"], a["ls"], a["wd"], a["us"], a["m1"], a["w1"],
                       a["ws"], ctypes.byref(n), None)
    return rc, n.value


def test_muon_step_refusals(lib):
    off = pointers(FAKE + 2)
    for bad in (dict(g=None), dict(m0=None), dict(w=None), dict(m1=None), dict(w1=None), dict(g=pointers(None)),
                dict(g=off), dict(m0=off), dict(m1=off), dict(w=off), dict(w1=off), dict(dt=1, w=pointers(FAKE + 1)),
                dict(dt=9), dict(udt=9), dict(count=0), dict(count=65), dict(coef=None), dict(steps=0), dict(eps=-1.0),
                dict(beta=-0.1), dict(beta=1.0), dict(beta=math.nan), dict(gs=math.inf), dict(lr=math.nan),
                dict(wd=math.nan), dict(us=math.inf), dict(ls=FAKE + 2), dict(ws=FAKE + 4), dict(size=512)):
        assert step(lib, **bad)[0] == gcq.GC_EINVAL, bad
        assert b"muon_step" in lib.gc_last_error()
    assert step(lib, ws=None, m=2 ** 21)[0] == gcq.GC_EUNSUPPORTED
    assert step(lib, m=0)[0] == gcq.GC_OK


def test_binding_checks():
    d = lambda *s, **k: FakeShape(s, **k)  # noqa: E731
    ws = d(1 << 24, dtype=torch.uint8)
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="number of matrices"):
        gcq.orthogonalize([], [], ws, stream=S)
    with pytest.raises(ValueError, match="number of matrices"):
        gcq.orthogonalize([d(4, 8)] * 65, [d(4, 8)] * 65, ws, stream=S)
    with pytest.raises(ValueError, match="must be matrices"):
        gcq.orthogonalize([d(4, 8, 2)], [d(4, 8, 2)], ws, stream=S)
    with pytest.raises(ValueError, match="outs differ in number"):
        gcq.orthogonalize([d(4, 8)] * 2, [d(4, 8)], ws, stream=S)
    with pytest.raises(ValueError, match="xs differ in size"):
        gcq.orthogonalize([d(4, 8), d(8, 4)], [d(4, 8)] * 2, ws, stream=S)
    with pytest.raises(TypeError, match=r"xs\[1\]: expected"):
        gcq.orthogonalize([d(4, 8), d(4, 8, dtype=bf)], [d(4, 8)] * 2, ws, stream=S)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        gcq.orthogonalize([d(4, 8)], [d(4, 8, dtype=torch.float64)], ws, stream=S)
    with pytest.raises(ValueError, match="three numbers"):
        gcq.orthogonalize([d(4, 8)], [d(4, 8)], ws, coefficients=((1.0, 2.0),), stream=S)
    with pytest.raises(gcq.GcqError, match="1 to 64 steps"):
        gcq.orthogonalize([d(4, 8)], [d(4, 8)], ws, coefficients=(), stream=S)
    with pytest.raises(gcq.GcqError, match="eps"):
        gcq.orthogonalize([d(4, 8)], [d(4, 8)], ws, eps=-1.0, stream=S)
    with pytest.raises(ValueError, match="ws too small"):
        gcq.orthogonalize([d(4, 8)], [d(4, 8)], d(0, dtype=torch.uint8), stream=S)
    with pytest.raises(gcq.GcqError, match="workspace too small"):
        gcq.orthogonalize([d(200, 300)], [d(200, 300)], d(64, dtype=torch.uint8), stream=S)
    with pytest.raises(ValueError, match="momenta differ in size"):
        gcq.muon_step([d(4, 8)], [d(4, 9)], [d(4, 8)], ws, stream=S)
    with pytest.raises(ValueError, match="new_weights differ in number"):
        gcq.muon_step([d(4, 8)], [d(4, 8)], [d(4, 8)], ws, new_weights=[], stream=S)
    with pytest.raises(TypeError, match=r"grads\[0\]: expected"):
        gcq.muon_step([d(4, 8, dtype=bf)], [d(4, 8)], [d(4, 8)], ws, stream=S)
    with pytest.raises(ValueError, match="lr_scale must hold one"):
        gcq.muon_step([d(4, 8)], [d(4, 8)], [d(4, 8)], ws, lr_scale=d(2), stream=S)
    with pytest.raises(gcq.GcqError, match="momentum must"):
        gcq.muon_step([d(4, 8)], [d(4, 8)], [d(4, 8)], ws, momentum=1.0, stream=S)
