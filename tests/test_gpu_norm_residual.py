"""norm_residual and norm_residual_grad against the formulas in 64 bits.

Tolerances (F = 2^-24): a sum over a row is at most 64 fp32 additions deep, so
it is off by 64 F of its terms' magnitudes; a root mean square's factor by
half of that and a few steps (40 F); each product or sum adds its F; each
output rounds once to its type. Sums over rows are at most `rows` additions
deep."""
import pytest
import torch

import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

TYPES = [torch.float32, torch.bfloat16, torch.float16]
F = po.F32
SUM, RSTD = 64 * F, 40 * F
EPS = 1e-6


def case(rows, d, gates, t, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=n(rows, d).to(t), y=(n(rows, d) * 0.7).to(t), post=1 + 0.1 * n(d), pre=1 + 0.1 * n(d),
                gate=0.5 + 0.5 * n(gates, d), dz=n(rows, d).to(t), dh=n(rows, d).to(t))


def spread(gate, rows):
    return 1.0 if gate is None else gate.double().repeat_interleave(rows // gate.shape[0], dim=0)


def one(v):
    return 1.0 if v is None else v.double()


def plain(c, s, p, seed, worker):
    """(value, allowed error before the output's rounding) of z, h, rstd_post, rstd_pre."""
    x, y = c["x"].double(), c["y"].double()
    rows, d = y.shape
    f = po.factor(rows * d, p, seed, worker).reshape(rows, d) if p else torch.ones(rows, d, dtype=torch.float64)
    rp = (y.square().mean(1) + EPS).rsqrt() if c["post"] is not None else torch.ones(rows, dtype=torch.float64)
    b = spread(c["gate"], rows) * f * (y * rp[:, None] * one(c["post"]))
    z = s * x + b
    ez = (s * x).abs() * F + b.abs() * (RSTD + 8 * F) + z.abs() * F
    rz = (z.square().mean(1) + EPS).rsqrt()
    erz = rz * ((z.abs() * ez).mean(1) * rz.square() + RSTD)
    h = z * rz[:, None] * one(c["pre"])
    eh = (rz[:, None] * one(c["pre"])).abs() * ez + h.abs() * (erz / rz)[:, None] + h.abs() * 3 * F
    return (z, ez), (h, eh), (rp, rp * RSTD), (rz, erz)


def check(got, ref, err):
    t = got.dtype
    assert got.shape == ref.shape
    allowed = 1.01 * err + ref.abs() * 1.01 * po.HALF_STEP[t] + po.TINY[t]
    off = (got.cpu().double() - ref).abs()
    assert bool((off <= allowed).all()), float((off / allowed).max())


def to(c, *names):
    return {k: None if c[k] is None else c[k].to(gu.DEV) for k in names}


def forward(gcq, c, s, p, seed, worker, place=lambda v: v):
    rows, d = c["y"].shape
    v = to(c, "x", "y", "post", "pre", "gate")
    x, y = place(v["x"]), place(v["y"])
    z, h = (place(torch.full_like(v["y"], float("nan"))) for _ in range(2))
    rp, rz = (torch.full((rows,), float("nan"), device=gu.DEV) for _ in range(2))
    gcq.norm_residual(x, y, z, h=h if c["pre"] is not None else None, post_gain=v["post"], gate=v["gate"],
                      pre_gain=v["pre"], residual_scale=s, eps=EPS, p=p, seed=seed, worker=worker, rstd_post=rp,
                      rstd_pre=rz)
    gu.sync()
    return z, h, rp, rz


def compare_forward(c, got, s, p, seed, worker):
    z, h, rp, rz = plain(c, s, p, seed, worker)
    check(got[0], *z)
    if c["post"] is not None:
        check(got[2], *rp)
    if c["pre"] is not None:
        check(got[1], *h)
        check(got[3], *rz)


SHAPES = [(1, 1, 1), (3, 5, 1), (2, 64, 2), (9, 100, 3), (5, 257, 5), (33, 768, 1), (6, 1001, 2), (700, 513, 350),
          (37, 2048, 1), (5, 4096, 1), (3, 4104, 3), (4, 8192, 2), (2, 9001, 1), (3, 16384, 1), (5000, 72, 1)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_forward(gcq, shape, t, p):
    announce(f"norm_residual {shape} {t} p={p}")
    c = case(*shape, t, seed=sum(shape))
    compare_forward(c, forward(gcq, c, 0.5, p, 11, 3), 0.5, p, 11, 3)


def plain_grad(c, z, rp, rz, s, p, seed, worker):
    """(value, allowed error) of dx, dy, dpost, dgate, dpre."""
    z, y = z.cpu().double(), c["y"].double()
    rows, d = y.shape
    zero = torch.zeros(rows, d, dtype=torch.float64)
    dz = zero if c["dz"] is None else c["dz"].double()
    f = po.factor(rows * d, p, seed, worker).reshape(rows, d) if p else torch.ones(rows, d, dtype=torch.float64)
    gate, post, pre = spread(c["gate"], rows), one(c["post"]), one(c["pre"])
    if c["pre"] is None:
        dh, r = zero, torch.zeros(rows, 1, dtype=torch.float64)
    else:
        dh, r = c["dh"].double(), rz.cpu().double()[:, None]
    a = rp.cpu().double()[:, None] if c["post"] is not None else torch.ones(rows, 1, dtype=torch.float64)
    zn, yn, g = z * r, y * a, dh * pre
    c1 = (g * zn).mean(1, keepdim=True)
    ec1 = (g * zn).abs().mean(1, keepdim=True) * SUM
    e = dz + r * g
    ee = (dz.abs() + (r * g).abs()) * 4 * F
    t = e - zn * r * c1
    et = ee + (zn * r).abs() * ec1 + (zn * r * c1).abs() * 4 * F
    q = gate * f * post * yn
    du = t * gate * f * post
    if c["post"] is not None:
        c2 = (t * q).mean(1, keepdim=True)
        ec2 = ((q * e).abs().mean(1, keepdim=True) + (r * c1 * q * zn).abs().mean(1, keepdim=True)) * (SUM + 8 * F) \
            + r * ec1 * (q * zn).abs().mean(1, keepdim=True) + (q.abs() * ee).mean(1, keepdim=True)
    else:
        c2, ec2 = torch.zeros(rows, 1, dtype=torch.float64), torch.zeros(rows, 1, dtype=torch.float64)
    dy = a * (du - yn * c2)
    edy = a * ((gate * f * post).abs() * et + du.abs() * 7 * F + yn.abs() * ec2 + (yn * c2).abs() * 4 * F)
    deep = (rows + 70) * F

    def over(v, ev, groups):
        v, ev = v.reshape(groups, -1, d), ev.reshape(groups, -1, d)
        return v.sum(1), ev.sum(1) + v.abs().sum(1) * deep
    wy, ewy = t * f * yn, (f * yn).abs() * et + (t * f * yn).abs() * 5 * F
    gates = 1 if c["gate"] is None else c["gate"].shape[0]
    dpost = over(wy * gate, ewy * (gate if isinstance(gate, float) else gate.abs()) + (wy * gate).abs() * 2 * F, 1)
    dgate = over(wy * post, ewy * (post if isinstance(post, float) else post.abs()) + (wy * post).abs() * 2 * F, gates)
    dpre = over(dh * zn, (dh * zn).abs() * 3 * F, 1)
    return ((s * t, abs(s) * et + (s * t).abs() * F), (dy, edy), (dpost[0][0], dpost[1][0]), dgate,
            (dpre[0][0], dpre[1][0]))


def backward(gcq, c, z, rp, rz, s, p, seed, worker, place=lambda v: v, step=None):
    rows, d = c["y"].shape
    v = to(c, "y", "post", "pre", "gate", "dz", "dh")
    gates = 1 if c["gate"] is None else c["gate"].shape[0]
    dx, dy = (place(torch.full_like(v["y"], float("nan"))) for _ in range(2))
    grads = {k: None if v[k] is None else torch.full_like(v[k], float("nan")) for k in ("post", "gate", "pre")}
    ws = torch.full((gcq.norm_residual_grad_ws_bytes(rows, d, gates),), 255, dtype=torch.uint8, device=gu.DEV)
    place_or = lambda k: None if v[k] is None else place(v[k])  # noqa: E731
    gcq.norm_residual_grad(place(z), place(v["y"]), dx, dy, ws, dz=place_or("dz"), dh=place_or("dh"),
                           post_gain=v["post"], gate=v["gate"], pre_gain=v["pre"], residual_scale=s, p=p, seed=seed,
                           worker=worker, rstd_post=rp, rstd_pre=rz, dpost_gain=grads["post"], dgate=grads["gate"],
                           dpre_gain=grads["pre"], step=step)
    gu.sync()
    return dx, dy, grads["post"], grads["gate"], grads["pre"]


def compare_grad(c, got, *args):
    for g, (ref, err) in zip(got, plain_grad(c, *args)):
        if g is not None:
            check(g, ref, err)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_grad(gcq, shape, t, p):
    announce(f"norm_residual_grad {shape} {t} p={p}")
    c = case(*shape, t, seed=sum(shape) + 1)
    z, _, rp, rz = forward(gcq, c, 0.5, p, 11, 3)
    compare_grad(c, backward(gcq, c, z, rp, rz, 0.5, p, 11, 3), z, rp, rz, 0.5, p, 11, 3)


@pytest.mark.parametrize("absent", [("post",), ("gate",), ("pre", "dh"), ("dz",), ("post", "gate"),
                                    ("post", "pre", "dh"), ("gate", "pre", "dh"), ("post", "gate", "pre", "dh"),
                                    ("post", "gate", "dz")], ids="-".join)
def test_without_some_of_it(gcq, absent):
    announce(f"norm_residual without {absent}")
    for t, (rows, d) in ((torch.bfloat16, (40, 300)), (torch.float32, (7, 1024)), (torch.float32, (4, 3000))):
        c = case(rows, d, 1, t) | dict.fromkeys(absent)
        for p in (0.0, 0.2):
            got = forward(gcq, c, 1.0, p, 5, 1)
            compare_forward(c, got, 1.0, p, 5, 1)
            z, _, rp, rz = got
            compare_grad(c, backward(gcq, c, z, rp, rz, 1.0, p, 5, 1), z, rp, rz, 1.0, p, 5, 1)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("d", [768, 1001])
def test_alignment_does_not_change_the_result(gcq, t, d):
    announce(f"norm_residual misaligned {t} d={d}")
    rows = 20
    c = case(rows, d, 4, t)
    guards = []

    def off(v):
        buf = torch.full((v.numel() + 64,), 7.0, dtype=v.dtype, device=gu.DEV)
        view = buf[1:1 + v.numel()].view(v.shape)
        view.copy_(v)
        guards.append((buf, v.numel()))
        return view
    a, b = forward(gcq, c, 0.5, 0.1, 2, 2), forward(gcq, c, 0.5, 0.1, 2, 2, place=off)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    a, b = backward(gcq, c, *a[::2], a[3], 0.5, 0.1, 2, 2), backward(gcq, c, *a[::2], a[3], 0.5, 0.1, 2, 2, place=off)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    for buf, n in guards:
        assert float(buf[0]) == 7.0 and bool((buf[1 + n:] == 7.0).all())


def test_in_place(gcq):
    announce("norm_residual over its inputs")
    c = case(50, 776, 5, torch.bfloat16)
    z, h, rp, rz = forward(gcq, c, 0.5, 0.1, 2, 2)
    v = to(c, "x", "y", "post", "pre", "gate", "dz", "dh")
    x, y = v["x"].clone(), v["y"].clone()
    kw = dict(post_gain=v["post"], gate=v["gate"], pre_gain=v["pre"], residual_scale=0.5, p=0.1, seed=2, worker=2)
    gcq.norm_residual(x, y, x, h=y, eps=EPS, rstd_post=rp, rstd_pre=rz, **kw)
    assert torch.equal(x, z) and torch.equal(y, h)
    dx, dy = backward(gcq, c, z, rp, rz, 0.5, 0.1, 2, 2)[:2]
    ws = torch.empty(gcq.norm_residual_grad_ws_bytes(50, 776, 5), dtype=torch.uint8, device=gu.DEV)
    gcq.norm_residual_grad(z, v["y"], v["dz"], v["dh"], ws, dz=v["dz"], dh=v["dh"], rstd_post=rp, rstd_pre=rz, **kw)
    gu.sync()
    assert torch.equal(v["dz"], dx) and torch.equal(v["dh"], dy)


def test_no_rows(gcq):
    announce("norm_residual of no rows")
    e = torch.empty(0, 8, device=gu.DEV)
    one_, per = torch.ones(8, device=gu.DEV), torch.empty(0, device=gu.DEV)
    gcq.norm_residual(e, e, e.clone(), h=e.clone(), post_gain=one_, pre_gain=one_, rstd_post=per, rstd_pre=per)
    gate = torch.ones(3, 8, device=gu.DEV)
    grads = [torch.full_like(v, 9.0) for v in (one_, gate, one_)]
    ws = torch.empty(max(1, gcq.norm_residual_grad_ws_bytes(0, 8, 3)), dtype=torch.uint8, device=gu.DEV)
    gcq.norm_residual_grad(e, e, e.clone(), e.clone(), ws, dz=e, dh=e, post_gain=one_, gate=gate, pre_gain=one_,
                           rstd_post=per, rstd_pre=per, dpost_gain=grads[0], dgate=grads[1], dpre_gain=grads[2])
    gu.sync()
    assert all(bool((g == 0).all()) for g in grads)


def test_gradient_against_differences(gcq):
    """(f(v + e) - f(v - e)) / 2e of the kernels' own forward pass, fp32."""
    announce("norm_residual differences")
    rows, d = 4, 96
    c = case(rows, d, 2, torch.float32, seed=4)
    s, p, seed, worker = 0.7, 0.25, 9, 1
    z, _, rp, rz = forward(gcq, c, s, p, seed, worker)
    dx, dy, dpost, dgate, dpre = backward(gcq, c, z, rp, rz, s, p, seed, worker)

    def value(k, i, e):
        m = dict(c)
        m[k] = c[k].clone()
        m[k].view(-1)[i] += e
        got = forward(gcq, m, s, p, seed, worker)
        return float((got[0].cpu().double() * c["dz"].double()).sum()
                     + (got[1].cpu().double() * c["dh"].double()).sum())
    # the loss sums 768 terms of size about 1 that each carry some F of error:
    # 768 * 8 F / (2 e) of noise at most, and e^2 / 6 times a third derivative
    # that stays below 100 here
    e = 2.0 ** -7
    allowed = 768 * 8 * F / (2 * e) + 100 * e * e / 6
    for k, got in (("x", dx), ("y", dy), ("post", dpost), ("gate", dgate), ("pre", dpre)):
        for i in (0, 17, c[k].numel() - 1):
            diff = (value(k, i, e) - value(k, i, -e)) / (2 * e)
            assert abs(diff - float(got.view(-1)[i])) <= allowed, (k, i)


def test_same_mask_as_dropout(gcq):
    announce("norm_residual's mask is dropout's")
    rows, d = 7, 130
    y = torch.ones(rows, d, device=gu.DEV)
    out, z = torch.empty_like(y), torch.empty_like(y)
    gcq.dropout(y, 0.3, 77, 5, out)
    gcq.norm_residual(torch.zeros_like(y), y, z, p=0.3, seed=77, worker=5)
    gu.sync()
    assert torch.equal(out, z)


def test_graph_replays(gcq):
    announce("norm_residual and its gradient in a HIP graph")
    rows, d, gates = 300, 520, 3
    c = case(rows, d, gates, torch.bfloat16)
    v = to(c, "x", "y", "post", "pre", "gate", "dz", "dh")
    step = torch.zeros(1, dtype=torch.int64, device=gu.DEV)
    z, h, dx, dy = (torch.empty_like(v["x"]) for _ in range(4))
    rp, rz = (torch.empty(rows, device=gu.DEV) for _ in range(2))
    grads = [torch.empty_like(v[k]) for k in ("post", "gate", "pre")]
    ws = torch.empty(gcq.norm_residual_grad_ws_bytes(rows, d, gates), dtype=torch.uint8, device=gu.DEV)
    kw = dict(post_gain=v["post"], gate=v["gate"], pre_gain=v["pre"], residual_scale=0.5, p=0.1, seed=3, worker=1,
              step=step, rstd_post=rp, rstd_pre=rz)

    def body():
        gcq.norm_residual(v["x"], v["y"], z, h=h, eps=EPS, **kw)
        gcq.norm_residual_grad(z, v["y"], dx, dy, ws, dz=v["dz"], dh=v["dh"], dpost_gain=grads[0], dgate=grads[1],
                               dpre_gain=grads[2], **kw)
        step.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    gu.sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for k in range(1, 4):
        c2 = case(rows, d, gates, torch.bfloat16, seed=k)
        for name in ("x", "y", "dz", "dh"):
            v[name].copy_(c2[name])
        c2 |= {n: c[n] for n in ("post", "pre", "gate")}
        for out in (z, h, dx, dy, rp, rz, *grads):
            out.fill_(float("nan"))
        ws.fill_(255)
        gu.sync()
        graph.replay()
        gu.sync()
        compare_forward(c2, (z, h, rp, rz), 0.5, 0.1, 3 + k, 1)
        compare_grad(c2, (dx, dy, *grads), z, rp, rz, 0.5, 0.1, 3 + k, 1)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_grad_without_norms_of_specials(gcq, t, p):
    """Without gains z is linear in y: its gradient does not depend on what y
    holds, infinities and NaN included. (dgate does, where they are kept.)"""
    announce(f"norm_residual_grad of infinities in y {t} p={p}")
    rows, d = 12, 136
    c = case(rows, d, 3, t) | dict.fromkeys(("post", "pre", "dh"))
    want = backward(gcq, c, c["y"].to(gu.DEV), None, None, 0.5, p, 8, 2)
    bad = dict(c, y=c["y"].clone())
    for k, v in enumerate((float("inf"), -float("inf"), float("nan"))):
        bad["y"][k::4, k::5] = v
    got = backward(gcq, bad, c["y"].to(gu.DEV), None, None, 0.5, p, 8, 2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    f = po.factor(rows * d, p, 8, 2).reshape(rows, d) if p else torch.ones(rows, d)
    reached = ((bad["y"] != c["y"]) & (f != 0)).reshape(3, -1, d).any(1)
    assert bool(torch.isfinite(got[3].cpu())[~reached].all()) and not bool(torch.isfinite(got[3].cpu())[reached].any())


# more gates than strips of rows: a workgroup has several, the last one fewer
# (teams of one wave twice, teams of a workgroup)
MANY_GATES = [(1545, 72, 515), (3081, 513, 1027), (771, 2056, 257)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", MANY_GATES, ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_grad_of_several_gates_a_strip(gcq, shape, t, p):
    announce(f"norm_residual_grad {shape} {t} p={p}")
    c = case(*shape, t, seed=sum(shape))
    z, _, rp, rz = forward(gcq, c, 0.5, p, 11, 3)
    got = backward(gcq, c, z, rp, rz, 0.5, p, 11, 3)
    compare_grad(c, got, z, rp, rz, 0.5, p, 11, 3)
    # dgate left out, and each gain's gradient: the rest stays the same
    rows, d, gates = shape
    v = to(c, "y", "post", "pre", "gate", "dz", "dh")
    ws = torch.full((gcq.norm_residual_grad_ws_bytes(rows, d, gates),), 255, dtype=torch.uint8, device=gu.DEV)
    for names in ({"post", "pre"}, {"gate"}, {"pre"}, set()):
        out = {k: torch.full_like(v[k], float("nan")) if k in names else None for k in ("post", "gate", "pre")}
        dx, dy = torch.empty_like(v["y"]), torch.empty_like(v["y"])
        gcq.norm_residual_grad(z, v["y"], dx, dy, ws, dz=v["dz"], dh=v["dh"], post_gain=v["post"], gate=v["gate"],
                               pre_gain=v["pre"], residual_scale=0.5, p=p, seed=11, worker=3, rstd_post=rp,
                               rstd_pre=rz, dpost_gain=out["post"], dgate=out["gate"], dpre_gain=out["pre"])
        gu.sync()
        assert torch.equal(dx, got[0]) and torch.equal(dy, got[1])
        for k, full in zip(("post", "gate", "pre"), got[2:]):
            assert out[k] is None or torch.equal(out[k], full)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(600, 4096, 3), (1100, 2100, 11), (300, 8192, 3), (150, 16384, 3), (150, 9001, 5)],
                         ids=str)
def test_several_rows_of_a_wide_team(gcq, shape, t):
    """More rows than teams of several waves: each takes rows in turn, the next
    one's loads under this one's sums, over a gate's end too."""
    announce(f"norm_residual {shape} {t}")
    c = case(*shape, t, seed=sum(shape))
    got = forward(gcq, c, 0.5, 0.1, 11, 3)
    compare_forward(c, got, 0.5, 0.1, 11, 3)
    z, _, rp, rz = got
    compare_grad(c, backward(gcq, c, z, rp, rz, 0.5, 0.1, 11, 3), z, rp, rz, 0.5, 0.1, 11, 3)


@pytest.mark.slow
def test_offsets_past_32_bits(gcq):
    """2^32 values and more: rows on both sides of that index, in place."""
    rows, d, gates, t, p, seed, worker = 1_048_583, 4096, 1, torch.bfloat16, 0.3, 5, 2
    free, _ = torch.cuda.mem_get_info()
    if free < 50 << 30:
        pytest.skip("needs 50 GiB of device memory")
    announce(f"norm_residual {rows} x {d}")
    g = torch.Generator(device=gu.DEV).manual_seed(1)
    big = [torch.empty(rows, d, dtype=t, device=gu.DEV).normal_(generator=g) for _ in range(4)]
    x, y, dz, dh = big
    at = torch.tensor([0, 3, 524_287, 1_048_575, 1_048_576, rows - 1])
    post, pre, gate = (1 + 0.1 * torch.randn(d, generator=g, device=gu.DEV) for _ in range(3))
    c = dict(x=x[at].cpu(), y=y[at].cpu(), dz=dz[at].cpu(), dh=dh[at].cpu(), post=post.cpu(), pre=pre.cpu(),
             gate=gate[None].cpu())
    rp, rz = torch.empty(rows, device=gu.DEV), torch.empty(rows, device=gu.DEV)
    h = torch.empty_like(y)
    kw = dict(post_gain=post, gate=gate, pre_gain=pre, residual_scale=0.5, p=p, seed=seed, worker=worker,
              rstd_post=rp, rstd_pre=rz)
    gcq.norm_residual(x, y, x, h=h, eps=EPS, **kw)  # z over x
    z = x
    got = [v[at].cpu() for v in (z, h, rp, rz)]
    ws = torch.empty(gcq.norm_residual_grad_ws_bytes(rows, d, gates), dtype=torch.uint8, device=gu.DEV)
    gcq.norm_residual_grad(z, y, dz, dh, ws, dz=dz, dh=dh, **kw)  # dx over dz, dy over dh
    gu.sync()
    grads = [v[at].cpu() for v in (dz, dh)]
    for k, row in enumerate(at.tolist()):
        one_row = {n: v if n in ("post", "pre", "gate") else v[k:k + 1] for n, v in c.items()}
        # the row's own part of the mask: 1 row at offset row * d
        f = po.factor(d, p, seed, worker, row * d).reshape(1, d)
        with pytest.MonkeyPatch.context() as m:
            m.setattr(po, "factor", lambda *a, **kw: f)
            for v, (ref, err) in zip(got, plain(one_row, 0.5, p, seed, worker)):
                check(v[k:k + 1], ref, err)
            ref = plain_grad(one_row, got[0][k:k + 1], got[2][k:k + 1], got[3][k:k + 1], 0.5, p, seed, worker)
            check(grads[0][k:k + 1], *ref[0])
            check(grads[1][k:k + 1], *ref[1])
    del big, x, y, z, dz, dh, h
    torch.cuda.empty_cache()
