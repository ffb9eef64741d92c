"""linear_xent_loss and linear_xent_grad against the formulas in 64 bits.

Tolerances. A logit is a sum of D products in fp32 sums: at most (D + 2) fp32
half steps of the terms' magnitudes. bf16 and fp16 factors are exact; an fp32
one is two fp16 planes, the second scaled by 2^11: each rounding leaves 2^-11,
so 2^-22 of the value is left of each factor and the left-out pair of second
planes is 2^-22 of the term, 3 * 2^-22 together. lse and loss follow, plus the
sums' own steps. A gradient is a sum of products whose factor G is off by the
logit's error and exp's steps times p, plus the rounding of G: 2^-8 (bf16 all
through), 2^-11 (any other gradient of 16 bits) or 2^-22 (fp32); the other
factor is exact, or two planes for fp32 inputs (3 * 2^-22 of a term with G's
own); then the fp32 sums, and one rounding to the gradient's type. Values far
below the largest of a matrix: planes of G stop at 2^-24-11 of their units,
2^-49 where the largest is 2^14 or more, one plane at 2^-24 of them, 2^-38;
inputs scaled the same way, of two planes at 2^-49, of bf16 at 2^-38."""
import math

import pytest
import torch

import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

TYPES = [torch.float32, torch.bfloat16, torch.float16]
IGNORE = -100


def inputs(N, V, D, t, seed=0, ignore=0.2, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, D, generator=g).to(t)
    w = (torch.randn(V, D, generator=g) * scale / math.sqrt(D)).to(t)
    y = torch.randint(0, V, (N,), generator=g)
    y[torch.rand(N, generator=g) < ignore] = IGNORE
    d = torch.randn(N, generator=g)
    return h, w, y, d


def logits64(h, w):
    """Logits, and for each row a bound of their error."""
    l = h.double() @ w.double().t()
    D = h.shape[1]
    mag = h.double().abs() @ w.double().abs().t()
    each = (D + 2) * po.F32 + (3.1 * 2.0 ** -22 if h.dtype == torch.float32 else 0.0)
    floor = 2.0 ** -36 * D * float(h.abs().max()) * float(w.abs().max())
    return l, mag.max(dim=1).values * each + floor


def plain_loss(h, w, y):
    l, e = logits64(h, w)
    lse = torch.logsumexp(l, dim=1)
    has = y != IGNORE
    at = torch.where(has, y, 0)
    loss = torch.where(has, lse - l.gather(1, at[:, None])[:, 0], 0.0)
    return loss, lse, e


def run_loss(gcq, h, w, y, ignore=IGNORE, stream=None):
    N, (V, D) = h.shape[0], w.shape
    dev = [x.to(gu.DEV) for x in (h, w, y)]
    loss, lse = (torch.full((N,), float("nan"), device=gu.DEV) for _ in range(2))
    ws = torch.full((max(1, gcq.linear_xent_loss_ws_bytes(N, V, D, h.dtype)),), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.linear_xent_loss(*dev, loss, lse, ws, ignore_index=ignore, stream=stream)
    gu.sync()
    return loss.cpu(), lse.cpu()


def check_loss(loss, lse, ref, ref_lse, e):
    # sums of up to 2^28 exponentials in fp32 pieces, a logarithm, one sum
    steps = 64 * po.F32
    allowed = e + steps * (1 + ref_lse.abs())
    assert bool(((lse.double() - ref_lse).abs() <= allowed).all())
    assert bool(((loss.double() - ref).abs() <= 2 * allowed + steps * ref.abs()).all())


SIZES = [(1, 1, 1), (1, 1000, 64), (2, 257, 65), (31, 64, 8), (33, 63, 128), (64, 300, 72), (257, 1000, 200),
         (300, 513, 768), (5, 30522, 768), (1000, 70, 1001)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_loss(gcq, size, t):
    announce(f"linear_xent_loss {size} {t}")
    h, w, y, _ = inputs(*size, t, seed=sum(size))
    ref, ref_lse, e = plain_loss(h, w, y)
    check_loss(*run_loss(gcq, h, w, y), ref, ref_lse, e)


def plain_grad(h, w, y, lse, d, out, other):
    """Gradients in 64 bits, and bounds of their errors before the outputs'
    own rounding."""
    l, e = logits64(h, w)
    has = (y != IGNORE)
    p = torch.exp(l - lse.double()[:, None])
    g = p.clone()
    rows = has.nonzero()[:, 0]
    g[rows, y[rows]] -= 1.0
    g *= torch.where(has, d.double(), 0.0)[:, None]
    ad = torch.where(has, d.double().abs(), 0.0)[:, None]
    # G: the logit's error and exp's own steps times p, one step of p - 1, the
    # planes' rounding of the whole
    top = float(ad.max())
    if out == torch.float32:
        rounding = g.abs() * 2.0 ** -22 + top * 2.0 ** -36
    elif h.dtype == out == other == torch.bfloat16:
        rounding = g.abs() * 2.0 ** -8
    else:
        rounding = g.abs() * 2.0 ** -11 + top * 2.0 ** -38
    eg = ad * p * (e[:, None] + 16 * po.F32) + rounding + ad * 2 * po.F32
    drop = 3.1 * 2.0 ** -22 if h.dtype == torch.float32 else 0.0

    def product(a, ea, b, k):
        # k terms summed in fp32, operands in planes
        mag = a.abs() @ b.abs()
        floor = 2.0 ** -38 * float(b.abs().max()) * a.abs().sum(1, keepdim=True)
        return a @ b, ea @ b.abs() + mag * ((k + 2) * po.F32 + drop) + floor
    hz = torch.where(has[:, None], h.double(), 0.0)
    return product(g, eg, w.double(), w.shape[0]) + product(g.t(), eg.t(), hz, h.shape[0])


def run_grad(gcq, h, w, y, lse, d, th, tw, skip=()):
    N, (V, D) = h.shape[0], w.shape
    dev = [x.to(gu.DEV) for x in (h, w, y, lse, d)]
    dh = None if "h" in skip else torch.full((N, D), float("nan"), dtype=th, device=gu.DEV)
    dw = None if "w" in skip else torch.full((V, D), float("nan"), dtype=tw, device=gu.DEV)
    ws = torch.full((max(1, gcq.linear_xent_grad_ws_bytes(N, V, D, h.dtype, th, tw)),), 255, dtype=torch.uint8,
                    device=gu.DEV)
    gcq.linear_xent_grad(*dev, dh, dw, ws)
    gu.sync()
    return None if dh is None else dh.cpu(), None if dw is None else dw.cpu()


def check_grad(got, ref, err):
    t = got.dtype
    allowed = err + ref.abs() * 1.01 * po.HALF_STEP[t] + po.TINY[t]
    off = (got.double() - ref).abs()
    assert bool((off <= allowed).all()), float((off / allowed).max())


CASES = [(t, th, tw) for t in TYPES for th in {t, torch.float32} for tw in {t, torch.float32}]


@pytest.mark.parametrize("types", CASES, ids=lambda c: "-".join(str(t)[6:] for t in c))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_grad(gcq, size, types):
    t, th, tw = types
    announce(f"linear_xent_grad {size} {types}")
    h, w, y, d = inputs(*size, t, seed=sum(size) + 1)
    lse = plain_loss(h, w, y)[1].float()
    dh, dw = run_grad(gcq, h, w, y, lse, d, th, tw)
    rh, eh, _, _ = plain_grad(h, w, y, lse, d, th, tw)
    _, _, rw, ew = plain_grad(h, w, y, lse, d, tw, th)
    check_grad(dh, rh, eh)
    check_grad(dw, rw, ew)


def test_grad_alone_of_each(gcq):
    announce("linear_xent_grad of one operand")
    h, w, y, d = inputs(70, 500, 96, torch.bfloat16)
    lse = plain_loss(h, w, y)[1].float()
    # a gradient left out counts as one of the inputs' type
    for tw in (torch.bfloat16, torch.float32):
        both = run_grad(gcq, h, w, y, lse, d, torch.bfloat16, tw)
        if tw == torch.bfloat16:
            dh, none = run_grad(gcq, h, w, y, lse, d, torch.bfloat16, tw, skip="w")
            assert none is None and torch.equal(dh, both[0])
        none, dw = run_grad(gcq, h, w, y, lse, d, torch.bfloat16, tw, skip="h")
        assert none is None and torch.equal(dw, both[1])
