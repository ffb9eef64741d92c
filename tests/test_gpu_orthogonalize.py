"""orthogonalize and muon_step against the formulas in 64 bits.

Tolerance. A step's factors are rounded by u = 2^-11 (a bf16 result) or 2^-22 at
most, and a sum of K fp32 terms by some 2^-24 sqrt(K) / 2 of the root of its
terms' squares, all independently: an error of mean square u^2 / 3 a value. With
U, S the singular vectors and values of X and p_i the eigenvalues of P, the error
of a step is dP X + P dX: in the singular basis s_j dP_ij + p_i dX_ij. The steps
that follow multiply it by the divided differences of what they make of the
singular values (D_ij = (f_i - f_j) / (s_i - s_j) for the symmetric part, (f_i +
f_j) / (s_i + s_j) for the other, f_i / s_i beside a square). The root of the sum
of squares of all that, four times over, and the output's rounding, is allowed
(relative to the result, as Frobenius norms)."""
import math

import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
F = po.F32
QUINTIC = ((3.4445, -4.7750, 2.0315),) * 5
CUBIC = ((1.5, -0.5, 0.0),) * 4
MIXED = ((3.4445, -4.7750, 2.0315),) * 2 + ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375))
EPS = 1e-7


def update(m, n, seed=0, strong=True):
    """A few strong directions over many weak ones, as gradients of weights have."""
    g = torch.Generator().manual_seed(seed)
    x = 0.5 * torch.randn(m, n, generator=g)
    k = min(8, m, n)
    if strong:
        x = x + (torch.randn(m, k, generator=g) * 2.0 ** -torch.arange(k)) @ torch.randn(k, n, generator=g)
    return 1e-3 * x


def plain(x, series, eps=EPS):
    x = x.double()
    x = x / (x.square().sum().sqrt() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in series:
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.t() if tall else x


def allowed(x, series, both, eps=EPS):
    """What may be off, relative to the result (Frobenius norms)."""
    x = x.double()
    x = x / (x.square().sum().sqrt() + eps)
    x = x if x.shape[0] <= x.shape[1] else x.t()
    r, c = x.shape
    u2 = (2.0 ** (-22 if both else -11)) ** 2 / 3
    total = 0.0
    mean = lambda v: float(v.square().mean())  # noqa: E731
    for k, (a, b, c2) in enumerate(series):
        sums = lambda K: F * F * K / 4  # noqa: E731
        A = x @ x.t()
        ms_x, ms_a = mean(x), mean(A)
        P = b * A + c2 * (A @ A)
        spread = lambda v: float((v.square() @ v.square().t()).mean())  # noqa: E731
        v_a = (2 * u2 + sums(c)) * spread(x) + (u2 if not both else 4 * F * F) * ms_a
        v_p = (b * b + 4 * c2 * c2 * r * ms_a) * v_a + c2 * c2 * (2 * u2 + sums(r)) * spread(A) + u2 * mean(P)
        s = torch.linalg.svdvals(x)
        p = b * s ** 2 + c2 * s ** 4
        nxt = a * s + p * s
        f = nxt.clone()
        for a2, b2, c3 in series[k + 1:]:
            f = a2 * f + b2 * f ** 3 + c3 * f ** 5
        # divided differences of what the later steps make of this one's result
        d, dd = nxt[:, None] - nxt[None, :], f[:, None] - f[None, :]
        near = d.abs() < 1e-9 * nxt.abs().max()
        slope = torch.ones_like(nxt)
        v = nxt.clone()
        for a2, b2, c3 in series[k + 1:]:
            slope = slope * (a2 + 3 * b2 * v ** 2 + 5 * c3 * v ** 4)
            v = a2 * v + b2 * v ** 3 + c3 * v ** 5
        sym = torch.where(near, slope[:, None].expand(r, r), dd / torch.where(near, torch.ones_like(d), d))
        both_sum = nxt[:, None] + nxt[None, :]
        anti = (f[:, None] + f[None, :]) / torch.where(both_sum.abs() < 1e-300, torch.ones_like(d), both_sum)
        D2 = torch.maximum(sym.square(), anti.square())
        beside = (f / torch.where(nxt.abs() < 1e-300, torch.ones_like(nxt), nxt)).square()
        # sums of the third product, and the carried X to 2^-22
        v_out = sums(r) * float((P.square() @ x.square()).mean()) + 2.0 ** -44 * mean(a * x + P @ x)
        e2 = (D2 * (s[None, :] ** 2 * v_p + p[:, None] ** 2 * u2 * ms_x + v_out)).sum()
        e2 = e2 + (c - r) * (beside * (p ** 2 * u2 * ms_x + v_out)).sum()
        total += math.sqrt(float(e2))
        x = a * x + P @ x
    return 4 * total / max(float(x.norm()), 1e-300)


def check(got, x, series, scale=1.0, eps=EPS):
    ref = scale * plain(x, series, eps)
    t = got.dtype
    off = float((got.cpu().double() - ref).norm() / max(float(ref.norm()), 1e-300))
    most = allowed(x, series, t != BF16, eps) + 1.01 * po.HALF_STEP[t]
    if t == F16:  # values below its normal range
        most += po.TINY[t] * math.sqrt(ref.numel()) / max(float(ref.norm()), 1e-300)
    assert off <= most, (off, most)


def run(gcq, xs, out_dtype, series=QUINTIC, place=lambda v: v, **kw):
    xd = [place(x.to(gu.DEV)) for x in xs]
    outs = [place(torch.full(x.shape, float("nan"), dtype=out_dtype, device=gu.DEV)) for x in xs]
    m, n = xs[0].shape
    # whatever the workspace holds
    ws = torch.full((gcq.orthogonalize_ws_bytes(len(xs), m, n, out_dtype),), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.orthogonalize(xd, outs, ws, coefficients=series, eps=EPS, **kw)
    gu.sync()
    return outs


SHAPES = [(1, 1, 1), (2, 1, 7), (1, 5, 1), (3, 3, 5), (1, 64, 64), (1, 64, 576), (2, 65, 63), (1, 100, 300),
          (2, 128, 128), (3, 129, 257), (1, 300, 100), (2, 513, 40), (1, 10, 1000), (1, 700, 640), (5, 257, 700),
          # what one workgroup holds: each of its kinds, at its edges
          (64, 17, 20), (3, 32, 256), (2, 33, 31), (1, 1024, 32), (2, 24, 1000), (1, 64, 256), (7, 257, 64), (1, 50, 1024),
          (2, 128, 256), (1, 200, 70), (1, 65, 129), (1, 31, 1025), (1, 129, 129)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16), (BF16, F32)], ids=str)
def test_against_64_bits(gcq, shape, types):
    announce(f"orthogonalize {shape} {types}")
    count, m, n = shape
    xs = [update(m, n, seed=m + n + k, strong=k != 1).to(types[0]) for k in range(count)]
    for got, x in zip(run(gcq, xs, types[1]), xs):
        check(got, x, QUINTIC)


@pytest.mark.parametrize("series", [QUINTIC[:1], QUINTIC[:2], CUBIC, MIXED, ((0.5, 0.0, 0.0),) * 3,
                                    ((1.0, 0.0, -0.25),) * 2], ids=len)
@pytest.mark.parametrize("shape", [(40, 90), (200, 130)], ids=str)
@pytest.mark.parametrize("t", [F32, BF16], ids=str)
def test_series(gcq, series, shape, t):
    announce(f"orthogonalize series {len(series)} {shape} {t}")
    x = update(*shape, seed=3).to(t)
    check(run(gcq, [x], t, series, scale=0.75)[0], x, series, scale=0.75)


# (larger tiles, ragged edges of theirs, more rounds than one of the chip)
@pytest.mark.parametrize("shape", [(16, 1000, 1100), (16, 1100, 1000), (40, 700, 513), (12, 520, 1500), (64, 300, 290),
                                   (1, 300, 20000), (1, 20000, 300), (2, 130, 9000), (1, 16384, 256), (1, 520, 5003),
                                   (1, 1500, 2600)], ids=str)
@pytest.mark.parametrize("t", [F32, BF16], ids=str)
def test_many_tiles(gcq, shape, t):
    announce(f"orthogonalize {shape} {t}")
    count, m, n = shape
    x = update(m, n, seed=m).to(t)
    ref = plain(x, QUINTIC)
    most = allowed(x, QUINTIC, t != BF16) + 1.01 * po.HALF_STEP[t]
    # the same matrix with its rows in another order, so that no two are alike
    order = [torch.randperm(m, generator=torch.Generator().manual_seed(k)) for k in range(count)]
    for got, o in zip(run(gcq, [x[o].contiguous() for o in order], t), order):
        off = float((got.cpu().double() - ref[o]).norm() / ref.norm())
        assert off <= most, (off, most)


def off16(v):
    """The same values one element past a 16-byte boundary."""
    buf = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)
    out = buf[1:].view(v.shape)
    out.copy_(v)
    return out


@pytest.mark.parametrize("t", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("shape", [(33, 64), (7, 101), (150, 130)], ids=str)
def test_views_off_16_bytes(gcq, shape, t):
    announce(f"orthogonalize views {shape} {t}")
    x = update(*shape, seed=4).to(t)
    check(run(gcq, [x], t, place=off16)[0], x, QUINTIC)


def test_in_place_and_nothing_else(gcq):
    announce("orthogonalize in place")
    for m, n in ((50, 70), (131, 67), (64, 192)):
        xs = [update(m, n, seed=k) for k in range(3)]
        ref = run(gcq, xs, F32)
        flat = torch.full((3 * (m * n + 3) + 5,), 7.0, device=gu.DEV)
        views = [flat[k * (m * n + 3) + 1:][:m * n].view(m, n) for k in range(3)]
        for v, x in zip(views, xs):
            v.copy_(x)
        size = gcq.orthogonalize_ws_bytes(3, m, n, F32)
        ws = torch.full((size + 256,), 9, dtype=torch.uint8, device=gu.DEV)
        gcq.orthogonalize(views, views, ws[:size], eps=EPS)
        assert all(torch.equal(a, b) for a, b in zip(views, ref))
        assert bool((ws[size:] == 9).all())
        for v in views:
            v.fill_(7.0)
        assert bool((flat == 7.0).all())


@pytest.mark.parametrize("size", [1e30, 3e-39, 1e-30], ids=str)
def test_any_magnitude(gcq, size):
    """The norm neither overflows nor vanishes."""
    announce(f"orthogonalize values near {size}")
    x = update(70, 90, seed=5) * 1e3 * size
    got = torch.empty(70, 90, device=gu.DEV)
    ws = torch.empty(gcq.orthogonalize_ws_bytes(1, 70, 90, F32), dtype=torch.uint8, device=gu.DEV)
    gcq.orthogonalize([x.to(gu.DEV)], [got], ws, eps=0.0)
    check(got, x, QUINTIC, eps=0.0)


def test_rank_one_and_zero(gcq):
    announce("orthogonalize rank one and zero")
    g = torch.Generator().manual_seed(6)
    x = torch.outer(torch.randn(300, generator=g), torch.randn(200, generator=g))
    zero = torch.zeros(300, 200)
    got = run(gcq, [x, zero, x], BF16)
    check(got[0], x, QUINTIC)
    assert bool((got[1] == 0).all()) and torch.equal(got[0], got[2])
    got = run(gcq, [zero, x], F32)
    check(got[1], x, QUINTIC)
    assert bool((got[0] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite_stays_in_its_matrix(gcq, bad):
    announce(f"orthogonalize {bad}")
    xs = [update(100, 130, seed=k) for k in range(3)]
    ref = run(gcq, xs, F32)
    xs[1][17, 3] = bad
    got = run(gcq, xs, F32)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
    assert bool(got[1].isnan().all())


def test_empty(gcq):
    announce("orthogonalize empty")
    for m, n in ((0, 5), (5, 0)):
        e = torch.empty(m, n, device=gu.DEV)
        gcq.orthogonalize([e], [e], torch.empty(256, dtype=torch.uint8, device=gu.DEV))


def test_repeats_streams_and_graphs(gcq):
    """The same call gives the same bits: eager, on another stream, and from
    two graphs with workspaces of their own, replayed in turn."""
    announce("orthogonalize graphs")
    sides = [(96, 300), (700, 512)]
    calls = []
    for k, (m, n) in enumerate(sides):
        x = update(m, n, seed=k).to(gu.DEV)
        out = torch.empty(m, n, dtype=BF16, device=gu.DEV)
        ws = torch.empty(gcq.orthogonalize_ws_bytes(1, m, n, BF16), dtype=torch.uint8, device=gu.DEV)
        calls.append((x, out, ws))
    go = lambda c: gcq.orthogonalize([c[0]], [c[1]], c[2])  # noqa: E731
    eager = []
    s = torch.cuda.Stream()
    for c in calls:
        go(c)
        gu.sync()
        eager.append(c[1].clone())
        with torch.cuda.stream(s):
            c[1].zero_()
            go(c)
        s.synchronize()
        assert torch.equal(c[1], eager[-1])
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for g, c in zip(graphs, calls):
        with torch.cuda.graph(g):
            go(c)
    for turn in range(3):
        for c in calls:
            c[0].mul_(2.0)
            c[1].fill_(float("nan"))
        for g in graphs:
            g.replay()
        gu.sync()
        for c in calls:
            replayed = c[1].clone()
            go(c)
            gu.sync()
            assert torch.equal(c[1], replayed)


def test_two_calls_at_once(gcq):
    """On two streams, with workspaces of their own: what each gives alone. The
    same matrix may be read twice."""
    announce("orthogonalize two at once")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (m, n), (m2, n2) in (((600, 1500), (513, 700)), ((64, 500), (700, 600)), ((64, 200), (120, 250))):
        calls = []
        for k, (a, b) in enumerate(((m, n), (m2, n2))):
            x = update(a, b, seed=k).to(gu.DEV)
            outs = [torch.empty(a, b, dtype=BF16, device=gu.DEV) for _ in range(2)]
            ws = torch.empty(gcq.orthogonalize_ws_bytes(2, a, b, BF16), dtype=torch.uint8, device=gu.DEV)
            gcq.orthogonalize([x, x], outs, ws)
            gu.sync()
            assert torch.equal(outs[0], outs[1])
            calls.append((x, outs, ws, outs[0].clone()))
        for _ in range(4):
            for k, (x, outs, ws, _) in enumerate(calls):
                with torch.cuda.stream(s[k]):
                    for o in outs:
                        o.fill_(float("nan"))
                    gcq.orthogonalize([x, x], outs, ws)
        gu.sync()
        for x, outs, ws, alone in calls:
            assert torch.equal(outs[0], alone) and torch.equal(outs[1], alone)


@pytest.mark.parametrize("tall", [True, False], ids=["tall", "wide"])
def test_past_32_bit_offsets(gcq, tall):
    """2^20 x 2100 and 2100 x 2^20: more than 2^31 values, 2^32 bytes, 2^32 values of
    the planes. One step, row (column) by row: with |X| = 1 and u = 2^-11 a factor's
    rounding is at most u, so that |dA| <= 2 u + 2^-24 sqrt(K) + u |A|, |dP| <= |b| |dA|
    + |c| (2 |A| |dA| + 2 u |A|^2) + u |P|, and a row is off by |x| (|dP| + u |P|) and its
    rounding (2^-22 of what is carried is far less)."""
    announce(f"orthogonalize past 32 bits {tall}")
    c, r, at_once = 1 << 20, 2100, 1 << 16
    a, b, c2 = QUINTIC[0]
    g = torch.Generator(device=gu.DEV).manual_seed(5)
    right = torch.randn(4, r, generator=g, device=gu.DEV)
    shape = (c, r) if tall else (r, c)
    x = torch.empty(shape, dtype=BF16, device=gu.DEV)

    def part(t, k):
        """Rows (of the wide one: columns) k on."""
        return t[k:k + at_once] if tall else t[:, k:k + at_once].t()
    squares = 0.0
    A = torch.zeros(r, r, dtype=torch.float64, device=gu.DEV)
    for k in range(0, c, at_once):
        rows = torch.randn(at_once, 4, generator=g, device=gu.DEV) @ right
        part(x, k).copy_(0.1 * torch.randn(at_once, r, generator=g, device=gu.DEV) + rows)
        v = part(x, k).double().contiguous()
        A += v.t().contiguous() @ v
        squares += float(v.square().sum())
    out = torch.full(shape, float("nan"), dtype=BF16, device=gu.DEV)
    ws = torch.empty(gcq.orthogonalize_ws_bytes(1, *shape, BF16), dtype=torch.uint8, device=gu.DEV)
    gcq.orthogonalize([x], [out], ws, coefficients=((a, b, c2),), eps=EPS)
    gu.sync()
    norm = math.sqrt(squares) + EPS
    A /= norm ** 2
    P = b * A + c2 * (A @ A)
    u, nA, nP = 2.0 ** -11, float(A.norm()), float(P.norm())
    dA = 2 * u + 2.0 ** -24 * math.sqrt(c) + u * nA
    dP = abs(b) * dA + abs(c2) * (2 * nA * dA + 2 * u * nA ** 2) + u * nP
    for k in range(0, c, at_once):
        v = part(x, k).double().contiguous() / norm
        ref = a * v + v @ P
        off = (part(out, k).double() - ref).norm(dim=1)
        most = v.norm(dim=1) * (dP + u * nP) + 1.01 * po.HALF_STEP[BF16] * ref.norm(dim=1)
        assert bool((off <= most).all()), (k, float((off / most).max()))


# ---- the optimiser step ---------------------------------------------------------

def step_case(count, m, n, t, seed=0):
    g = torch.Generator().manual_seed(seed)
    grads = [8 * update(m, n, seed=seed + k) for k in range(count)]
    momenta = [update(m, n, seed=seed + 100 + k) for k in range(count)]
    weights = [(torch.randn(m, n, generator=g) / math.sqrt(n)).to(t) for _ in range(count)]
    return grads, momenta, weights


KW = dict(momentum=0.95, grad_scale=0.125, lr=0.05, weight_decay=0.1, update_scale=1.5)


def check_step(case, got_m, got_w, nesterov=True, update_dtype=None, lr_scale=1.0, series=QUINTIC, kw=KW):
    beta, lr = kw["momentum"], kw["lr"] * lr_scale
    for g, m0, w, m1, w1 in zip(*case, got_m, got_w):
        g64 = g.double() * kw["grad_scale"]
        m64 = g64 + beta * (m0.double() - g64)
        # g, m - g and the fma round once each, beta and 1 / scale are fp32
        em = 4 * F * (g64.abs() + m0.double().abs())
        assert bool(((m1.cpu().double() - m64).abs() <= em).all())
        u = g64 + beta * (m64 - g64) if nesterov else m64
        x = plain(u, series)
        ref = (1 - lr * kw["weight_decay"]) * w.double() - lr * kw["update_scale"] * x
        both = (update_dtype or w.dtype) != BF16
        # (u is off by a few F too, which grows with the small singular values
        # as the first step's error does)
        ex = (allowed(u, series, both) + 400 * F) * float(x.norm()) * abs(lr * kw["update_scale"])
        ew = 1.01 * po.HALF_STEP[w.dtype] * float(ref.norm()) + 4 * F * float(w.double().norm())
        off = float((w1.cpu().double() - ref).norm())
        assert off <= ex + ew, (off, ex, ew)


@pytest.mark.parametrize("t", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 30, 50), (1, 131, 64), (3, 256, 300), (1, 600, 257)], ids=str)
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(gcq, shape, t, nesterov):
    announce(f"muon_step {shape} {t} nesterov={nesterov}")
    count, m, n = shape
    case = step_case(count, m, n, t, seed=m)
    g, m0, w = ([v.to(gu.DEV) for v in vs] for vs in case)
    m1, w1 = [torch.full_like(v, float("nan")) for v in m0], [torch.full_like(v, float("nan")) for v in w]
    ws = torch.full((gcq.muon_step_ws_bytes(count, m, n, t),), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step(g, m0, w, ws, nesterov=nesterov, new_momenta=m1, new_weights=w1, **KW)
    gu.sync()
    check_step(case, m1, w1, nesterov)
    for dev, cpu in zip((g, m0, w), case):
        assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, cpu))
    # in place
    gcq.muon_step(g, m0, w, ws, nesterov=nesterov, **KW)
    assert all(torch.equal(a, b) for a, b in zip(m0 + w, m1 + w1))


@pytest.mark.parametrize("t,u", [(F32, BF16), (BF16, F32), (F16, BF16)], ids=str)
def test_step_update_dtype(gcq, t, u):
    announce(f"muon_step weights {t} update {u}")
    case = step_case(2, 200, 90, t, seed=9)
    g, m0, w = ([v.to(gu.DEV) for v in vs] for vs in case)
    ws = torch.empty(gcq.muon_step_ws_bytes(2, 200, 90, u), dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step(g, m0, w, ws, update_dtype=u, **KW)
    check_step(case, m0, w, update_dtype=u)


def test_step_of_flat_bucket_views(gcq):
    """Gradients, momenta and weights as views into flat buckets, at any offset
    of an element; what lies between them is left."""
    announce("muon_step flat buckets")
    m, n, gap = 37, 53, 3
    for t in (F32, BF16):
        case = step_case(3, m, n, t, seed=20)
        flat, views = [], []
        for vs in case:
            b = torch.full((3 * (m * n + gap) + 1,), 5.0, dtype=vs[0].dtype, device=gu.DEV)
            v = [b[1 + k * (m * n + gap):][:m * n].view(m, n) for k in range(3)]
            for dst, src in zip(v, vs):
                dst.copy_(src)
            flat.append(b)
            views.append(v)
        ws = torch.empty(gcq.muon_step_ws_bytes(3, m, n, t), dtype=torch.uint8, device=gu.DEV)
        gcq.muon_step(*views, ws, **KW)
        gu.sync()
        check_step(case, views[1], views[2])
        for b, v in zip(flat, views):
            for k in v:
                k.fill_(5.0)
            assert bool((b == 5.0).all())


def test_step_without_a_gradient_and_with_nan(gcq):
    announce("muon_step zero and nan")
    case = step_case(3, 60, 80, F32, seed=30)
    case[0][0].zero_(), case[1][0].zero_()
    case[0][1][3, 4] = float("nan")
    g, m0, w = ([v.to(gu.DEV) for v in vs] for vs in case)
    ws = torch.empty(gcq.muon_step_ws_bytes(3, 60, 80, F32), dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step(g, m0, w, ws, **KW)
    # no direction: decay alone
    keep = float(np.float32(1) - np.float32(KW["lr"]) * np.float32(KW["weight_decay"]))
    assert float((w[0].cpu().double() - case[2][0].double() * keep).abs().max()) < 4 * F
    assert bool((m0[0] == 0).all())
    assert bool(w[1].isnan().all()) and int(m0[1].isnan().sum()) == 1
    check_step([[v[2]] for v in case], m0[2:], w[2:])


@pytest.mark.parametrize("shape", [(40, 90), (300, 257)], ids=str)
def test_step_of_no_length(gcq, shape):
    """A rate of zero leaves the weights bit for bit and moves the momenta."""
    announce(f"step of no length {shape}")
    m, n = shape
    grads, momenta, weights = step_case(2, m, n, BF16)
    gd, md, wd = ([v.to(gu.DEV) for v in t] for t in (grads, momenta, weights))
    ws = torch.empty(gcq.muon_step_ws_bytes(2, m, n, BF16), dtype=torch.uint8, device=gu.DEV)
    for kw in (dict(lr=0.0, weight_decay=0.1), dict(lr=0.1, update_scale=0.0)):
        gcq.muon_step(gd, md, wd, ws, momentum=0.5, **kw)
    gu.sync()
    for k in range(2):
        assert torch.equal(wd[k].cpu(), weights[k])
        # a step rounds a difference, halved, and a sum: 2^-24 of the larger value each
        ref = 0.25 * momenta[k].double() + 0.75 * grads[k].double()
        size = torch.maximum(momenta[k].abs(), grads[k].abs()).double()
        assert bool(((md[k].cpu().double() - ref).abs() <= 3 * F * size).all())


def test_step_in_a_graph_follows_its_rate(gcq):
    announce("muon_step graph")
    case = step_case(2, 128, 200, BF16, seed=40)
    g, m0, w = ([v.to(gu.DEV) for v in vs] for vs in case)
    m1, w1 = [torch.empty_like(v) for v in m0], [torch.empty_like(v) for v in w]
    rate = torch.ones(1, device=gu.DEV)
    ws = torch.empty(gcq.muon_step_ws_bytes(2, 128, 200, BF16), dtype=torch.uint8, device=gu.DEV)

    def go():
        gcq.muon_step(g, m0, w, ws, lr_scale=rate, new_momenta=m1, new_weights=w1, **KW)
    go()
    gu.sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for r in (1.0, 0.5, 0.0):
        rate.fill_(r)
        go()
        gu.sync()
        eager = [v.clone() for v in m1 + w1]
        for v in m1 + w1:
            v.fill_(float("nan"))
        graph.replay()
        gu.sync()
        assert all(torch.equal(a, b) for a, b in zip(m1 + w1, eager))
        check_step(case, m1, w1, lr_scale=r)
    assert all(torch.equal(a, b) for a, b in zip(w1, w))


def test_step_from_compressed_gradients(gcq):
    """The chain of a data-parallel step: layer norm's and a weight's gradients
    of W workers, compressed and summed where the operators wrote them, and the
    optimiser step on the sum."""
    announce("muon_step from compressed gradients")
    W, rows, d, out_d, thr = 3, 64, 96, 80, 0.05
    g = torch.Generator().manual_seed(50)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gain, bias, weight = 1 + 0.1 * n(d), 0.1 * n(d), n(out_d, d) / math.sqrt(d)
    dev = lambda v: v.to(gu.DEV)  # noqa: E731
    blocks, words = [], gcq.gc_compressed_2bit_words(out_d * d)
    for w in range(W):
        x, y, dout = dev(n(rows, d)), dev(n(rows, d)), dev(n(rows, out_d) / rows)
        z, h, dx, dy = (torch.empty_like(x) for _ in range(4))
        mean, rstd = torch.empty(rows, device=gu.DEV), torch.empty(rows, device=gu.DEV)
        dgain, dbias = torch.empty(d, device=gu.DEV), torch.empty(d, device=gu.DEV)
        ws = torch.empty(gcq.layer_norm_grad_ws_bytes(rows, d), dtype=torch.uint8, device=gu.DEV)
        kw = dict(gain=dev(gain), p=0.1, seed=3, worker=w, mean=mean, rstd=rstd)
        gcq.layer_norm(x, h, y=y, z=z, bias=dev(bias), **kw)
        dweight = (dout.t() @ h).contiguous()
        gcq.layer_norm_grad(z, (dout @ dev(weight)).contiguous(), dx, ws, dy=dy, dgain=dgain, dbias=dbias, **kw)
        block = torch.empty(words, dtype=torch.int32, device=gu.DEV)
        gcq.compress_2bit(dweight, torch.zeros_like(dweight), -thr, thr, block)
        blocks.append(block)
        small = torch.empty(gcq.gc_compressed_2bit_words(d), dtype=torch.int32, device=gu.DEV)
        gcq.compress_2bit(dgain, torch.zeros_like(dgain), -thr, thr, small)
        ref = oracle.quantize_2bit(gu.host(dgain), np.zeros(d, np.float32), -thr, thr)
        np.testing.assert_array_equal(gu.host(small, np.uint32), ref)
    total = torch.empty(out_d, d, device=gu.DEV)
    gcq.decompress_2bit_sum(blocks, out_d * d, total)
    summed = oracle.dequantize_2bit_sum([gu.host(b, np.uint32) for b in blocks], out_d * d)
    momentum = update(out_d, d, seed=51)
    m0, w0 = dev(momentum), dev(weight)
    ws = torch.empty(gcq.muon_step_ws_bytes(1, out_d, d, F32), dtype=torch.uint8, device=gu.DEV)
    kw = KW | dict(grad_scale=1.0 / W)
    gcq.muon_step([total], [m0], [w0], ws, **kw)
    gu.sync()
    np.testing.assert_array_equal(gu.host(total).reshape(-1), summed)
    check_step(([torch.from_numpy(summed).view(out_d, d)], [momentum], [weight]), [m0], [w0], kw=kw)
