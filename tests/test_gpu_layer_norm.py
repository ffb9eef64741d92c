"""layer_norm and layer_norm_grad against the formulas in 64 bits.

Tolerances (F = 2^-24): a sum over a row is at most 64 fp32 additions deep, so
it is off by 64 F of its terms' magnitudes (SUM). The variance is off by 72 F of
itself (the sum, and three steps a term twice) and, where the means that the
deviations are taken from are off by m each, by 2 sigma (2 m) + (2 m)^2. Each
product or sum adds its F; each output rounds once to its type. Sums over rows
are at most `rows` + 16 additions deep."""
import pytest
import torch

import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

TYPES = [torch.float32, torch.bfloat16, torch.float16]
F = po.F32
SUM = 64 * F
EPS = 1e-5


def case(rows, d, t, seed=0, sub=True, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(n(rows, d) + mean).to(t), y=(n(rows, d) * 0.7).to(t) if sub else None, gain=1 + 0.1 * n(d),
                bias=0.2 * n(d), dz=n(rows, d).to(t), dh=n(rows, d).to(t))


def factor(c, p, seed, worker):
    rows, d = c["x"].shape
    return po.factor(rows * d, p, seed, worker).reshape(rows, d) if p else torch.ones(rows, d, dtype=torch.float64)


def one(v, other=1.0):
    return other if v is None else v.double()


def plain(c, p, seed, worker, eps=EPS):
    """(value, allowed error before the output's rounding) of z, h, mean, rstd."""
    z, ez = c["x"].double(), 0.0
    if c["y"] is not None:
        b = factor(c, p, seed, worker) * c["y"].double()
        z = z + b
        ez = (2 * b.abs() + z.abs()) * F
    ez = ez + torch.zeros_like(z)
    mean = z.mean(1, keepdim=True)
    em = SUM * z.abs().mean(1, keepdim=True) + ez.mean(1, keepdim=True)
    dev = z - mean
    var = dev.square().mean(1, keepdim=True)
    m = 2 * em + ez.square().mean(1, keepdim=True).sqrt()
    ev = 72 * F * var + 2 * var.sqrt() * m + m.square()
    rstd = (var + eps).rsqrt()
    # 1 / sqrt: the slope is half of the relative error as long as that is
    # small, and never more than it here
    er = ev / (var + eps) + 4 * F
    h = dev * rstd * one(c["gain"]) + one(c["bias"], 0.0)
    scaled = (rstd * one(c["gain"])).abs()
    eh = (ez + em + dev.abs() * F) * scaled + dev.abs() * scaled * (er + 2 * F) + h.abs() * F
    return (z, ez), (h, eh), (mean.squeeze(1), em.squeeze(1)), (rstd.squeeze(1), (rstd * er).squeeze(1))


def check(got, ref, err, live=None):
    t = got.dtype
    assert got.shape == ref.shape
    allowed = 1.01 * err + ref.abs() * 1.01 * po.HALF_STEP[t] + po.TINY[t]
    off = (got.cpu().double() - ref).abs()
    ok = off <= allowed
    assert bool((ok if live is None else ok[live]).all()), float((off / allowed).nan_to_num(0.0).max())


def on(v):
    return None if v is None else v.to(gu.DEV)


def forward(gcq, c, p=0.0, seed=11, worker=3, place=lambda v: v, keep_z=True, stats=True, **kw):
    x, y = place(on(c["x"])), None if c["y"] is None else place(on(c["y"]))
    h = place(torch.full_like(x, float("nan")))
    z = place(torch.full_like(x, float("nan"))) if y is not None and keep_z else None
    mean, rstd = (torch.full((x.shape[0],), float("nan"), device=gu.DEV) if stats else None for _ in range(2))
    gcq.layer_norm(x, h, y=y, z=z, gain=on(c["gain"]), bias=on(c["bias"]), eps=EPS, p=p, seed=seed, worker=worker,
                   mean=mean, rstd=rstd, **kw)
    gu.sync()
    return z, h, mean, rstd


def compare(got, ref, live=None):
    for g, r in zip(got, ref):
        if g is not None:
            check(g, *r, live=live)


SHAPES = [(1, 1), (3, 5), (2, 64), (9, 100), (5, 257), (33, 768), (6, 1001), (700, 513), (37, 2048), (5, 4096),
          (3, 4104), (4, 8192), (2, 9001), (3, 16384), (5000, 72)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("p", [None, 0.0, 0.3])
def test_forward(gcq, shape, t, p):
    announce(f"layer_norm {shape} {t} p={p}")
    c = case(*shape, t, seed=sum(shape), sub=p is not None)
    compare(forward(gcq, c, p or 0.0), plain(c, p or 0.0, 11, 3))


def plain_grad(c, z, mean, rstd, p, seed, worker):
    """(value, allowed error) of dx, dy, dgain, dbias."""
    z, mu, r = z.cpu().double(), mean.cpu().double()[:, None], rstd.cpu().double()[:, None]
    dz = torch.zeros_like(z) if c["dz"] is None else c["dz"].double()
    dh = c["dh"].double()
    zn, g = (z - mu) * r, dh * one(c["gain"])
    c0, c1 = g.mean(1, keepdim=True), (g * zn).mean(1, keepdim=True)
    inner = g - c0 - zn * c1
    dx = dz + r * inner
    e = r * ((g.abs() + c0.abs() + (zn * c1).abs()) * 6 * F + SUM * g.abs().mean(1, keepdim=True)
             + zn.abs() * 2 * SUM * (g * zn).abs().mean(1, keepdim=True)) + (dx.abs() + dz.abs()) * F
    f = factor(c | {"x": z}, p, seed, worker)
    dy = dx * f
    deep = (z.shape[0] + 16) * F
    return ((dx, e), (dy, e * f + dy.abs() * 2 * F), ((dh * zn).sum(0), deep * (dh * zn).abs().sum(0)),
            (dh.sum(0), deep * dh.abs().sum(0)))


def backward(gcq, c, z, mean, rstd, p=0.0, seed=11, worker=3, place=lambda v: v, dy=True, ws=None):
    rows, d = z.shape
    dx = place(torch.full((rows, d), float("nan"), dtype=z.dtype, device=gu.DEV))
    dyt = place(torch.full_like(dx, float("nan"))) if dy else None
    dgain, dbias = (torch.full((d,), float("nan"), device=gu.DEV) for _ in range(2))
    if ws is None:
        ws = torch.empty(gcq.layer_norm_grad_ws_bytes(rows, d), dtype=torch.uint8, device=gu.DEV)
    gcq.layer_norm_grad(z, place(on(c["dh"])), dx, ws, dz=None if c["dz"] is None else place(on(c["dz"])), dy=dyt,
                        gain=on(c["gain"]), p=p, seed=seed, worker=worker, mean=mean, rstd=rstd, dgain=dgain,
                        dbias=dbias)
    gu.sync()
    return dx, dyt, dgain, dbias


def both(gcq, c, p=0.0, place=lambda v: v, dy=True):
    z, _, mean, rstd = forward(gcq, c, p, place=place)
    z = place(on(c["x"])) if z is None else z
    return backward(gcq, c, z, mean, rstd, p, place=place, dy=dy), plain_grad(c, z, mean, rstd, p, 11, 3)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("p", [None, 0.0, 0.3])
def test_backward(gcq, shape, t, p):
    announce(f"layer_norm_grad {shape} {t} p={p}")
    c = case(*shape, t, seed=sum(shape) + 1, sub=p is not None)
    if p is None:
        c["dz"] = None
    compare(*both(gcq, c, p or 0.0, dy=p is not None))


@pytest.mark.parametrize("shape", [(33, 768), (7, 1001), (5, 4096), (3, 8200)], ids=str)
def test_what_is_optional(gcq, shape):
    """Without gain, bias, z, the statistics, dz, dy, dgain or dbias the rest
    comes out the same, bit for bit where nothing it depends on is missing."""
    announce(f"layer_norm options {shape}")
    c = case(*shape, torch.bfloat16, seed=2)
    full = forward(gcq, c, 0.3)
    assert torch.equal(full[1], forward(gcq, c, 0.3, keep_z=False)[1])
    assert torch.equal(full[1], forward(gcq, c, 0.3, stats=False)[1])
    for missing in (("gain",), ("bias",), ("gain", "bias")):
        m = c | dict.fromkeys(missing)
        compare(forward(gcq, m, 0.3), plain(m, 0.3, 11, 3))
        compare(*both(gcq, m, 0.3))
    z, _, mean, rstd = full
    ref = backward(gcq, c, z, mean, rstd, 0.3)
    no_dy = backward(gcq, c, z, mean, rstd, 0.3, dy=False)
    assert all(torch.equal(a, b) for a, b in zip(ref[:1] + ref[2:], no_dy[:1] + no_dy[2:]))
    compare(*both(gcq, c | {"dz": None}, 0.3))
    dx = torch.empty_like(z)
    ws = torch.empty(gcq.layer_norm_grad_ws_bytes(*shape), dtype=torch.uint8, device=gu.DEV)
    args = dict(dz=on(c["dz"]), gain=on(c["gain"]), mean=mean, rstd=rstd)
    gcq.layer_norm_grad(z, on(c["dh"]), dx, ws, **args)
    assert torch.equal(dx, ref[0])
    dbias = torch.empty(shape[1], device=gu.DEV)
    gcq.layer_norm_grad(z, on(c["dh"]), dx, ws, dbias=dbias, **args)
    assert torch.equal(dbias, ref[3])


def off16(v):
    """The same values two bytes (fp32: four) past a 16-byte boundary."""
    buf = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)
    out = buf[1:].view(v.shape)
    out.copy_(v)
    return out


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(5, 64), (9, 768), (4, 1000), (3, 4096), (2, 12288)], ids=str)
def test_views_off_16_bytes(gcq, shape, t):
    announce(f"layer_norm views {shape} {t}")
    c = case(*shape, t, seed=4)
    compare(forward(gcq, c, 0.3, place=off16), plain(c, 0.3, 11, 3))
    compare(*both(gcq, c, 0.3, place=off16))


@pytest.mark.parametrize("d", [96, 2048, 10000])
def test_outputs_in_the_inputs_buffers(gcq, d):
    announce(f"layer_norm in place {d}")
    c = case(21, d, torch.bfloat16, seed=5)
    z, h, mean, rstd = forward(gcq, c, 0.3)
    x, y = on(c["x"]), on(c["y"])
    gcq.layer_norm(x, y, y=y, z=x, gain=on(c["gain"]), bias=on(c["bias"]), eps=EPS, p=0.3, seed=11, worker=3)
    assert torch.equal(x, z) and torch.equal(y, h)
    ref = backward(gcq, c, z, mean, rstd, 0.3)
    for into in (("dh", "dz"), ("z", "dh"), ("dz", "z")):
        b = dict(z=z.clone(), dh=on(c["dh"]), dz=on(c["dz"]))
        ws = torch.empty(gcq.layer_norm_grad_ws_bytes(21, d), dtype=torch.uint8, device=gu.DEV)
        gcq.layer_norm_grad(b["z"], b["dh"], b[into[0]], ws, dz=b["dz"], dy=b[into[1]], gain=on(c["gain"]), p=0.3,
                            seed=11, worker=3, mean=mean, rstd=rstd)
        assert torch.equal(b[into[0]], ref[0]) and torch.equal(b[into[1]], ref[1]), into


@pytest.mark.parametrize("t,mean", [(torch.float32, 1000.0), (torch.float32, -30000.0), (torch.float16, 500.0)], ids=str)
@pytest.mark.parametrize("d", [768, 5000, 16384])
def test_mean_far_larger_than_the_deviations(gcq, d, t, mean):
    """The squares are taken of the deviations: mean(z^2) - mean^2 would be off
    by F mean^2, more than the variance itself."""
    announce(f"layer_norm mean {mean} {t} {d}")
    c = case(6, d, t, seed=6, sub=False, mean=mean)
    got, ref = forward(gcq, c), plain(c, 0.0, 11, 3)
    compare(got, ref)
    # what the worst case allows is loose here; the deviations' own roundings
    # are not: each value is off by 2^-24 of the mean, at random
    off = (got[1].cpu().double() - ref[1][0]).norm() / ref[1][0].norm()
    assert float(off) < po.HALF_STEP[t] + 8 * F * abs(mean)


def test_rows_that_are_constant_or_not_finite(gcq):
    announce("layer_norm rows")
    c = case(8, 768, torch.float32, seed=7)
    c["x"][1], c["y"][1] = 3.25, 0.0
    c["x"][3, 5] = float("inf")
    c["x"][5, 700] = float("nan")
    z, h, mean, rstd = forward(gcq, c)
    live = torch.tensor([0, 1, 2, 4, 6, 7])
    compare((z, h, mean, rstd), plain(c, 0.0, 11, 3), live=live)
    assert torch.equal(h[1].cpu(), c["bias"])  # no deviation at all
    assert bool(h[3].isnan().all()) and bool(h[5].isnan().all())
    # a dropped value takes no part, whatever it holds
    c = case(8, 768, torch.float32, seed=8)
    gone = factor(c, 0.5, 11, 3) == 0
    a = forward(gcq, c, 0.5)
    c["y"][gone] = float("nan")
    b = forward(gcq, c, 0.5)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_no_rows(gcq):
    announce("layer_norm no rows")
    c = case(0, 64, torch.bfloat16)
    z, h, mean, rstd = forward(gcq, c)
    assert h.numel() == 0
    _, _, dgain, dbias = backward(gcq, c, z, mean, rstd)
    assert bool((dgain == 0).all()) and bool((dbias == 0).all())


@pytest.mark.parametrize("d", [64, 1001, 6000])
def test_everything_dropped(gcq, d):
    """p = 1: y does not count, whatever it holds, and gets no gradient."""
    announce(f"layer_norm p = 1, {d}")
    c = case(9, d, torch.bfloat16, seed=12)
    y = torch.full_like(c["x"], float("nan"))
    z, h, alone = (torch.empty(9, d, dtype=torch.bfloat16, device=gu.DEV) for _ in range(3))
    mean, rstd = (torch.empty(9, device=gu.DEV) for _ in range(2))
    kw = dict(gain=on(c["gain"]), bias=on(c["bias"]), eps=EPS)
    gcq.layer_norm(on(c["x"]), h, y=on(y), z=z, p=1.0, mean=mean, rstd=rstd, **kw)
    gcq.layer_norm(on(c["x"]), alone, **kw)
    dx, dy = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
    gcq.layer_norm_grad(z, on(c["dh"]), dx, torch.empty(gcq.layer_norm_grad_ws_bytes(9, d), dtype=torch.uint8, device=gu.DEV),
                        dy=dy, gain=kw["gain"], p=1.0, mean=mean, rstd=rstd)
    assert torch.equal(z.cpu(), c["x"]) and torch.equal(h, alone)
    assert bool((dy == 0).all()) and bool(torch.isfinite(dx.float()).all())


def test_rows_behind_the_last_are_left(gcq):
    announce("layer_norm padded")
    for d in (64, 1001, 6000):
        c = case(5, d, torch.float16, seed=9)
        z, h, mean, rstd = (torch.full((8, d) if k < 2 else (8,), 7.0, dtype=torch.float16 if k < 2 else torch.float32,
                                       device=gu.DEV) for k in range(4))
        gcq.layer_norm(on(c["x"]), h[:5], y=on(c["y"]), z=z[:5], gain=on(c["gain"]), bias=on(c["bias"]), eps=EPS,
                       mean=mean[:5], rstd=rstd[:5])
        compare((z[:5], h[:5], mean[:5], rstd[:5]), plain(c, 0.0, 0, 0))
        dx, dy = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
        sums = torch.full((2, d + 8), 7.0, device=gu.DEV)
        size = gcq.layer_norm_grad_ws_bytes(5, d)
        ws = torch.full((size + 64,), 7, dtype=torch.uint8, device=gu.DEV)
        gcq.layer_norm_grad(z[:5], on(c["dh"]), dx[:5], ws[:size], dz=on(c["dz"]), dy=dy[:5], gain=on(c["gain"]),
                            mean=mean[:5], rstd=rstd[:5], dgain=sums[0, :d], dbias=sums[1, :d])
        for v in (z[5:], h[5:], mean[5:], rstd[5:], dx[5:], dy[5:], sums[:, d:], ws[size:]):
            assert bool((v == 7).all())


def test_gradient_against_differences(gcq):
    """Along a direction, the gradients predict what the 64-bit function does."""
    announce("layer_norm_grad differences")
    c = case(40, 330, torch.float32, seed=10)
    got, _ = both(gcq, c, 0.3)
    g = torch.Generator().manual_seed(1)
    way = {k: torch.randn(c[k].shape, generator=g, dtype=torch.float64) for k in ("x", "y", "gain", "bias")}

    def value(s):
        (z, _), (h, _), _, _ = plain({k: v.double() + s * way[k] if k in way else v for k, v in c.items()}, 0.3, 11, 3)
        return float((z * c["dz"].double()).sum() + (h * c["dh"].double()).sum())
    s = 1e-4
    rise = (value(s) - value(-s)) / (2 * s)
    said = sum(float((v.cpu().double() * way[k]).sum()) for v, k in zip(got, ("x", "y", "gain", "bias")))
    # the third derivative's s^2, and fp32 gradients of 40 x 330 random terms
    assert abs(rise - said) < 1e-5 * abs(rise) + 1e-4, (rise, said)


def test_step_counter_streams_and_graphs(gcq):
    """A captured call draws a new mask as the counter moves; a replay gives
    what the eager call gives, also on a stream of its own."""
    announce("layer_norm graph")
    c = case(64, 1024, torch.bfloat16, seed=12)
    x, y, dh, gain, bias = (on(c[k]) for k in ("x", "y", "dh", "gain", "bias"))
    step = torch.zeros(1, dtype=torch.int64, device=gu.DEV)
    z, h, dx, dy = (torch.empty_like(x) for _ in range(4))
    mean, rstd = torch.empty(64, device=gu.DEV), torch.empty(64, device=gu.DEV)
    dgain, dbias = torch.empty(1024, device=gu.DEV), torch.empty(1024, device=gu.DEV)
    ws = torch.empty(gcq.layer_norm_grad_ws_bytes(64, 1024), dtype=torch.uint8, device=gu.DEV)

    def go():
        kw = dict(gain=gain, p=0.3, seed=5, worker=2, step=step, mean=mean, rstd=rstd)
        gcq.layer_norm(x, h, y=y, z=z, bias=bias, **kw)
        gcq.layer_norm_grad(z, dh, dx, ws, dy=dy, dgain=dgain, dbias=dbias, **kw)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    seen = []
    for k in range(3):
        step.fill_(k)
        go()
        gu.sync()
        eager = [v.clone() for v in (z, h, dx, dy, dgain, dbias, mean, rstd)]
        for v in (z, h, dx, dy, dgain, dbias, mean, rstd):
            v.fill_(float("nan"))
        graph.replay()
        gu.sync()
        assert all(torch.equal(a, b) for a, b in zip(eager, (z, h, dx, dy, dgain, dbias, mean, rstd)))
        seen.append(eager[0])
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    compare((seen[2],), plain(c, 0.3, 7, 2)[:1])


def test_sums_repeat_bit_for_bit(gcq):
    announce("layer_norm_grad repeats")
    c = case(3000, 1001, torch.float32, seed=13)
    a, _ = both(gcq, c, 0.3)
    b, _ = both(gcq, c, 0.3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_many_values(gcq):
    """More than 2^32 bytes and 2^31 values of one activation."""
    announce("layer_norm past 2^31 values")
    rows, d = 2 ** 18 + 3, 8192
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=gu.DEV).normal_()
    h = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=gu.DEV), torch.empty(rows, device=gu.DEV)
    gcq.layer_norm(x, h, eps=EPS, mean=mean, rstd=rstd)
    at = torch.tensor([0, 2 ** 17, 2 ** 18 - 1, 2 ** 18, rows - 1], device=gu.DEV)
    c = dict(x=x[at].cpu(), y=None, gain=None, bias=None, dz=None)
    compare((None, h[at], mean[at], rstd[at]), plain(c, 0.0, 0, 0))
    dx = torch.empty_like(x)
    dbias = torch.empty(d, device=gu.DEV)
    ws = torch.empty(gcq.layer_norm_grad_ws_bytes(rows, d), dtype=torch.uint8, device=gu.DEV)
    gcq.layer_norm_grad(x, h, dx, ws, mean=mean, rstd=rstd, dbias=dbias)
    gu.sync()
    c["dh"] = h[at].cpu()
    compare((dx[at],), plain_grad(c, x[at], mean[at], rstd[at], 0.0, 0, 0)[:1])
