"""orthogonalize and muon_step refuse outputs that lie in other buffers of the
call: whether what is there is read before or after it is overwritten depends on
the size of the matrices. The refusals need no GPU: the addresses are never
dereferenced."""
import ctypes

import pytest
import torch

import gradient_compression_quantize_amd as gcq_lib
from conftest import announce

SIZES = [(256, 300), (40, 90)]  # in tiles, and in one workgroup
ONE = (ctypes.c_float * 3)(1.5, -0.5, 0.0)
BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return gcq_lib.load()


def pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


def orth(lib, m, n, x, out, dt=0, odt=0):
    size = ctypes.c_size_t(1 << 40)
    return lib.orthogonalize(pointers(*x), len(x), m, n, dt, ONE, 1, 0.0, 1.0, pointers(*out), odt, BASE,
                             ctypes.byref(size), None)


def step(lib, m, n, g, m0, w, m1, w1, dt=0):
    size = ctypes.c_size_t(1 << 40)
    return lib.muon_step(pointers(*g), len(g), m, n, pointers(*m0), pointers(*w), dt, 0, ONE, 1, 0.0, 1.0, 0.9, 1, 0.1,
                         None, 0.0, 1.0, pointers(*m1), pointers(*w1), BASE, ctypes.byref(size), None)


def refused(lib, rc):
    return rc == gcq_lib.GC_EINVAL and b"overlap" in lib.gc_last_error()


@pytest.mark.parametrize("m,n", SIZES)
def test_orthogonalize(lib, m, n):
    far, b = 1 << 30, m * n * 4
    a, c, d = far, 2 * far, 3 * far
    # an out in another matrix's x, or in another out, or beside its own x
    for x, out in (((a, c), (c, a)), ((a, c), (a, a + b - 4)), ((a, c), (d, d)), ((a, c), (d, d + b - 4)),
                   ((a, c), (a, c - b + 4)), ((a,), (a + 16,)), ((a,), (a - 16,)), ((a, a), (a, d))):
        assert refused(lib, orth(lib, m, n, x, out)), (x, out)
    # one that is longer than its x, and reaches the next one
    assert refused(lib, orth(lib, m, n, (a, a + b // 2), (a, d), dt=1, odt=0))
    assert refused(lib, orth(lib, m, n, (a, a + b // 2), (a, a + b // 2), dt=0, odt=1))


@pytest.mark.parametrize("m,n", SIZES)
def test_muon_step(lib, m, n):
    far, b = 1 << 30, m * n * 4
    g, m0, w, m1, w1 = ((k * far, k * far + (1 << 28)) for k in range(1, 6))
    for bad in (dict(m1=g), dict(m1=(g[1], m1[1])), dict(m1=(g[0] + b - 4, m1[1])), dict(m1=m0[::-1]),
                dict(m1=(m0[0] + 4, m0[1])), dict(m1=(m1[0], m1[0])), dict(w1=w[::-1]), dict(w1=(w[0] - 4, w[1])),
                dict(w1=(w1[0], w1[0] + 4)), dict(w1=m1), dict(w1=g), dict(w1=m0), dict(m1=w), dict(m0=g, m1=g)):
        a = dict(g=g, m0=m0, w=w, m1=m1, w1=w1) | bad
        assert refused(lib, step(lib, m, n, **a)), bad


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
def test_what_is_allowed(gcq, m, n):
    """Outputs in their own inputs, also of another type, inputs that are the
    same, neighbours without a gap: what separate buffers give."""
    gu = pytest.importorskip("gpu_util")
    announce(f"overlaps that are allowed {m} x {n}")
    f32, bf16 = torch.float32, torch.bfloat16
    gen = torch.Generator().manual_seed(m)
    make = lambda: list(torch.randn(3, m, n, generator=gen).to(gu.DEV).unbind())  # noqa: E731
    x = make()
    for t in (f32, bf16):
        ws = torch.empty(gcq.orthogonalize_ws_bytes(3, m, n, t), dtype=torch.uint8, device=gu.DEV)
        ref = [torch.empty(m, n, dtype=t, device=gu.DEV) for _ in x]
        gcq.orthogonalize(x, ref, ws)
        own = torch.stack(x)
        outs = [v.view(-1).view(t)[:m * n].view(m, n) for v in own.unbind()]
        gcq.orthogonalize(own.unbind(), outs, ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        same = torch.empty(3, m, n, dtype=t, device=gu.DEV)
        gcq.orthogonalize([x[1]] * 3, same.unbind(), ws)
        assert all(torch.equal(v, ref[1]) for v in same)
    g, m0, w = make(), make(), make()
    ws = torch.empty(gcq.muon_step_ws_bytes(3, m, n, f32), dtype=torch.uint8, device=gu.DEV)

    def step(g, m0, w, m1, w1):
        gcq.muon_step(g, m0, w, ws, new_momenta=m1, new_weights=w1)
        gu.sync()
        return list(m1) + list(w1)
    new = lambda: torch.empty(3, m, n, device=gu.DEV).unbind()  # noqa: E731
    ref = step(g, m0, w, new(), new())
    m2, w2 = torch.stack(m0).unbind(), torch.stack(w).unbind()
    assert all(torch.equal(a, b) for a, b in zip(step(g, m2, w2, m2, w2), ref))
    of_one, ref = step([g[0]] * 3, m0, w, new(), new()), step([v.clone() for v in [g[0]] * 3], m0, w, new(), new())
    assert all(torch.equal(a, b) for a, b in zip(of_one, ref))
    from_g, ref = step(g, g, w, new(), new()), step(g, [v.clone() for v in g], w, new(), new())
    assert all(torch.equal(a, b) for a, b in zip(from_g, ref))
