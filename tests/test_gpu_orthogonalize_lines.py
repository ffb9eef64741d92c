"""orthogonalize and muon_step row by row and column by column, against 64 bits,
with the bounds of rounded_newton_schulz.py (drawn from the roundings of the
planes)."""
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
          (129, 257), (300, 290), (70, 90), (520, 1500), (1500, 520), (700, 640), (130, 3000)]


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
