"""orthogonalize and muon_step row by row and column by column, against 64 bits,
with the bounds of rounded_newton_schulz.py (drawn from the roundings of the
planes); values of any size, rank one, zero and not finite in matrices of one
workgroup and of tiles."""
import pytest
import torch

import plain_ops as po
from conftest import announce
from rounded_newton_schulz import allowed, lines
from test_rounded_newton_schulz import exact

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
QUINTIC = ((3.4445, -4.7750, 2.0315),) * 5
MIXED = QUINTIC[:2] + ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375))
EPS = 1e-7


def update(m, n, seed):
    g = torch.Generator().manual_seed(seed)
    strong = (torch.randn(m, 8, generator=g) * 2.0 ** -torch.arange(8)) @ torch.randn(8, n, generator=g)
    return 1e-3 * (0.5 * torch.randn(m, n, generator=g) + strong)


def reference(x, series=QUINTIC, eps=EPS):
    return exact(x, series, eps) if x.shape[0] <= x.shape[1] else exact(x.t(), series, eps).t()


def check(got, x, both, series=QUINTIC, eps=EPS, ref=None, bounds=None):
    ref = reference(x, series, eps) if ref is None else ref
    matrix, line = allowed(x, ref, series, both, eps) if bounds is None else bounds
    half = 1.01 * po.HALF_STEP[got.dtype]
    off = got.cpu().double() - ref
    assert float(off.norm() / ref.norm()) <= matrix + half, (float(off.norm() / ref.norm()), matrix)
    worst = float((lines(off) / lines(ref)).max())
    assert worst <= line + half, (worst, line)


def orthogonalize(gcq, xs, out_dtype, series=QUINTIC, eps=EPS):
    outs = [torch.full(x.shape, float("nan"), dtype=out_dtype, device=gu.DEV) for x in xs]
    size = gcq.orthogonalize_ws_bytes(len(xs), *xs[0].shape, out_dtype)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.orthogonalize([x.to(gu.DEV) for x in xs], outs, ws, coefficients=series, eps=eps)
    gu.sync()
    return outs


def unrounded(gcq, xs, update_dtype, series=QUINTIC, eps=EPS):
    """X as muon_step computes it for updates of this type, in fp32: a step of -1
    from weights of zero, along the gradients themselves."""
    g = [x.to(gu.DEV) for x in xs]
    m0, w = ([torch.zeros_like(v) for v in g] for _ in range(2))
    size = gcq.muon_step_ws_bytes(len(xs), *xs[0].shape, update_dtype)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step(g, m0, w, ws, coefficients=series, eps=eps, momentum=0.0, lr=-1.0, update_dtype=update_dtype)
    gu.sync()
    return w


# one workgroup: each of its kinds, wide and tall; tiles of 64, 128 and 256, ragged
SHAPES = [(17, 20), (20, 33), (31, 1000), (1000, 31), (64, 576), (576, 64), (50, 250), (250, 50), (128, 256), (200, 100),
          (129, 257), (300, 290), (70, 90), (520, 1500), (1500, 520), (700, 640), (130, 3000),
          # thin ones past one workgroup, whose smaller side is mostly padding
          (16, 16384), (16384, 16), (20, 5001), (5001, 20)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("series", [QUINTIC, MIXED], ids=["quintic", "mixed"])
def test_products_of_one_plane(gcq, shape, series):
    announce(f"orthogonalize lines of {shape}, one plane, {len(series)} steps")
    x = update(*shape, seed=sum(shape))
    ref = reference(x, series)
    bounds = allowed(x, ref, series, False, EPS)
    check(unrounded(gcq, [x], BF16, series)[0], x, False, ref=ref, bounds=bounds)
    check(orthogonalize(gcq, [x], BF16, series)[0], x, False, ref=ref, bounds=bounds)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("series", [QUINTIC, MIXED], ids=["quintic", "mixed"])
def test_products_of_both_planes(gcq, shape, series):
    announce(f"orthogonalize lines of {shape}, both planes, {len(series)} steps")
    x = update(*shape, seed=sum(shape) + 1)
    ref = reference(x, series)
    bounds = allowed(x, ref, series, True, EPS)
    check(unrounded(gcq, [x], F32, series)[0], x, True, ref=ref, bounds=bounds)
    check(orthogonalize(gcq, [x], F32, series)[0], x, True, ref=ref, bounds=bounds)


@pytest.mark.parametrize("count,m,n", [(3, 1, 70001), (2, 70001, 1), (5, 3, 2000), (64, 2, 1500)])
@pytest.mark.parametrize("t", [F32, BF16], ids=str)
def test_vectors_and_a_few_rows(gcq, count, m, n, t):
    """Of one row the singular value is 1 and stays beside it: what the steps make of
    1, times x / |x|. Matrices of a call do not meet in each other's padding."""
    announce(f"orthogonalize {count} of {m} x {n} {t}")
    xs = [update(m, n, seed=k) for k in range(count)]
    xs[count // 2][0, 0] = float("nan")
    for k, (got, x) in enumerate(zip(orthogonalize(gcq, xs, t), xs)):
        if k == count // 2:
            assert bool(got.isnan().all())
            continue
        ref = reference(x)
        # the few roundings of A and P, which all values share (2^-11 or 2^-22 of P up
        # to 4.8 each, grown by at most 3.4445 in each of the other steps)
        most = (2.0 ** -22 if t == F32 else 2.0 ** -11) * 4.8 * 6 * 3.4445 ** 4
        off = float((got.cpu().double() - ref).norm() / ref.norm())
        assert off <= most + po.HALF_STEP[t], (off, most)


@pytest.mark.parametrize("shape", [(16, 1000, 1100), (16, 1100, 1000), (40, 700, 513), (64, 300, 290)], ids=str)
@pytest.mark.parametrize("both", [False, True])
def test_larger_tiles(gcq, shape, both):
    announce(f"orthogonalize lines of {shape}, both planes={both}")
    count, m, n = shape
    x = update(m, n, seed=m)
    ref = reference(x)
    matrix, line = allowed(x, ref, QUINTIC, both, EPS)
    # the same matrix with its rows in another order, so that no two are alike
    order = [torch.randperm(m, generator=torch.Generator().manual_seed(k)) for k in range(count)]
    for got, o in zip(unrounded(gcq, [x[o].contiguous() for o in order], F32 if both else BF16), order):
        check(got, x, both, ref=ref[o], bounds=(matrix, line))


# (matrices in one workgroup of one plane and two, in tiles of either)
KINDS = [(40, 90, F32), (300, 30, F32), (128, 200, BF16), (500, 60, BF16), (70, 90, F32), (300, 290, BF16)]


@pytest.mark.parametrize("m,n,t", KINDS, ids=str)
@pytest.mark.parametrize("size", [1e30, 1e18, 1e-30, 3e-39], ids=str)
def test_any_magnitude(gcq, m, n, t, size):
    """A factor of a power of two changes no bit of the result, as long as all
    values stay normal; below that, what is left of them is what counts."""
    announce(f"orthogonalize {m} x {n} {t} near {size}")
    x = update(m, n, seed=5) * 1e3 * size
    check(orthogonalize(gcq, [x], t, eps=0.0)[0], x, t != BF16, eps=0.0)
    if size > 1e-38:
        times = 2.0 ** (20 if size < 1 else -20)
        a, b = orthogonalize(gcq, [x], t, eps=0.0), orthogonalize(gcq, [x * times], t, eps=0.0)
        assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("m,n,t", KINDS, ids=str)
def test_rank_one_and_zero(gcq, m, n, t):
    announce(f"orthogonalize rank one and zero {m} x {n} {t}")
    g = torch.Generator().manual_seed(6)
    # (values away from zero: each of a row and column of it is a line of its own)
    u, v = (torch.randn(k, generator=g).sign() * (0.5 + torch.rand(k, generator=g)) for k in (m, n))
    x, zero = torch.outer(u, v), torch.zeros(m, n)
    got = orthogonalize(gcq, [x, zero, x], t)
    # one singular value, of 1: what the steps make of it, along u v'
    s = 1.0
    for a, b, c in QUINTIC:
        s = a * s + b * s ** 3 + c * s ** 5
    way = torch.outer(u.double() / u.double().norm(), v.double() / v.double().norm())
    ref = reference(x)
    # (x is rounded, by at most 2^-24 of its norm, and what lies beside one direction
    # grows by 3.4445 in each of the five steps: 485 times)
    assert float((ref - s * way).norm()) < 3.4445 ** 5 * po.F32
    check(got[0], x, t != BF16, ref=ref)
    assert bool((got[1] == 0).all()) and torch.equal(got[0], got[2])
    # without eps nothing says where zero goes
    got = orthogonalize(gcq, [x, zero], t, eps=0.0)
    assert bool(got[1].isnan().all()) and bool(got[0].isfinite().all())


@pytest.mark.parametrize("m,n,t", KINDS, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite_stays_in_its_matrix(gcq, m, n, t, bad):
    announce(f"orthogonalize {m} x {n} {t} with {bad}")
    xs = [update(m, n, seed=k) for k in range(3)]
    ref = orthogonalize(gcq, xs, t)
    for where in ((17, 3), (0, 0), (m - 1, n - 1)):
        held = xs[1][where].clone()
        xs[1][where] = bad
        got = orthogonalize(gcq, xs, t)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
        assert bool(got[1].isnan().all())
        for series in (QUINTIC[:1], ((1.5, -0.5, 0.0),), ((1.0, 0.0, 0.0),)):
            assert bool(orthogonalize(gcq, xs, t, series)[1].isnan().all()), series
        xs[1][where] = held
