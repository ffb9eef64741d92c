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


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_a_last_round_of_small_tiles(gcq, t):
    """258 tiles of 256 x 256: the vocabulary's end goes as smaller ones, with
    targets on both sides of the border and in the last row."""
    N, V, D = 300, 33_000, 72
    announce(f"linear_xent {N} x {V} x {D} {t}")
    h, w, y, d = inputs(N, V, D, t, seed=6)
    y[:6] = torch.tensor([0, 128 * 256 - 1, 128 * 256, 128 * 256 + 127, 128 * 256 + 128, V - 1])
    ref, ref_lse, e = plain_loss(h, w, y)
    check_loss(*run_loss(gcq, h, w, y), ref, ref_lse, e)
    lse = ref_lse.float()
    dh, dw = run_grad(gcq, h, w, y, lse, d, t, torch.float32)
    rh, eh, _, _ = plain_grad(h, w, y, lse, d, t, torch.float32)
    _, _, rw, ew = plain_grad(h, w, y, lse, d, torch.float32, t)
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


def test_no_tokens_and_no_targets(gcq):
    announce("linear_xent of no tokens, and of none with a target")
    w = torch.randn(40, 24, device=gu.DEV)
    e = torch.empty(0, 24, device=gu.DEV)
    per, none = torch.empty(0, device=gu.DEV), torch.empty(0, dtype=torch.int64, device=gu.DEV)
    ws = torch.empty(gcq.linear_xent_grad_ws_bytes(0, 40, 24, w.dtype), dtype=torch.uint8, device=gu.DEV)
    dw = torch.full_like(w, 5.0)
    gcq.linear_xent_loss(e, w, none, per, per.clone(), ws)
    gcq.linear_xent_grad(e, w, none, per, per, e.clone(), dw, ws)
    gu.sync()
    assert bool((dw == 0).all())
    with pytest.raises(ValueError, match="ws too small"):
        gcq.linear_xent_grad(e, w, none, per, per, e.clone(), dw, torch.empty(0, dtype=torch.uint8, device=gu.DEV))
    for t in TYPES:
        h, w, y, d = inputs(37, 130, 65, t)
        y[:] = IGNORE
        loss, lse = run_loss(gcq, h, w, y)
        assert bool((loss == 0).all())
        dh, dw = run_grad(gcq, h, w, y, lse, d, torch.float32, t)
        assert bool((dh == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_rows_without_a_target_reach_nothing(gcq, t):
    """NaN, infinities and huge values in the hidden states, lse and dloss of
    padded rows; targets outside the vocabulary; an ignore_index inside it."""
    announce(f"linear_xent padded rows {t}")
    h, w, y, d = inputs(300, 513, 130, t, ignore=0.0)
    pad = torch.arange(300) % 3 == 1
    out = torch.arange(300) % 7 == 2
    clean_y = torch.where(pad | out, IGNORE, y)
    lse = plain_loss(h, w, y)[1].float()
    want_loss = run_loss(gcq, h, w, clean_y)[0]
    want = run_grad(gcq, h, w, clean_y, lse, d, t, torch.float32)
    bad_h, bad_y, bad_lse, bad_d = h.clone(), y.clone(), lse.clone(), d.clone()
    big = torch.finfo(t).max
    for k, v in enumerate((float("nan"), float("inf"), -float("inf"), big)):
        rows = (pad | out).nonzero()[k::4, 0]
        bad_h[rows] = v
        bad_lse[rows] = v
        bad_d[rows] = v
    bad_y[pad] = IGNORE
    bad_y[out] = torch.tensor([513, -1, 2 ** 40, -2 ** 62, 514])[torch.arange(int(out.sum())) % 5]
    bad_y[pad & out] = IGNORE
    loss, _ = run_loss(gcq, bad_h, w, bad_y)
    off = out & ~pad
    assert bool(torch.isnan(loss[off]).all()) and torch.equal(loss[~off], want_loss[~off])
    got = run_grad(gcq, bad_h, w, bad_y, bad_lse, bad_d, t, torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # an ignore_index that is a row of the vocabulary
    y7 = torch.where(pad, 7, torch.where(y == 7, 8, y))
    loss7, _ = run_loss(gcq, h, w, y7, ignore=7)
    ref, ref_lse, e = plain_loss(h, w, torch.where(pad, IGNORE, y7))
    assert bool((loss7[pad] == 0).all())
    assert bool(((loss7.double() - ref).abs() <= 2 * e + 200 * po.F32 * (1 + ref_lse.abs()))[~pad].all())


def test_confident_and_extreme_logits(gcq):
    """Targets of probability near 1 and logits of some hundreds: the sums of
    exponentials neither overflow nor vanish."""
    announce("linear_xent extreme logits")
    for t in TYPES:
        h, w, y, d = inputs(64, 400, 128, t, ignore=0.0, scale=40.0)
        ref, ref_lse, e = plain_loss(h, w, y)
        assert float(ref_lse.max()) > 80
        check_loss(*run_loss(gcq, h, w, y), ref, ref_lse, e)
        y = (h.double() @ w.double().t()).argmax(dim=1)
        ref, ref_lse, e = plain_loss(h, w, y)
        loss, lse = run_loss(gcq, h, w, y)
        check_loss(loss, lse, ref, ref_lse, e)
        dh, dw = run_grad(gcq, h, w, y, ref_lse.float(), d, t, torch.float32)
        # e^x of the logit's error, which reaches some 1e-3 here, grows faster than it
        rh, eh, _, _ = plain_grad(h, w, y, ref_lse.float(), d, t, torch.float32)
        _, _, rw, ew = plain_grad(h, w, y, ref_lse.float(), d, torch.float32, t)
        check_grad(dh, rh, 1.01 * eh)
        check_grad(dw, rw, 1.01 * ew)


def test_scale_of_the_inputs_does_not_matter(gcq):
    """fp32 inputs scaled by powers of two far outside fp16's range give the
    same loss bit for bit where the logits are the same."""
    announce("linear_xent fp32 scales")
    h, w, y, d = inputs(50, 300, 96, torch.float32)
    want = run_loss(gcq, h, w, y)
    lse = want[1]
    dh, dw = run_grad(gcq, h, w, y, lse, d, torch.float32, torch.float32)
    for k in (-100, -40, 40, 100):
        a, b = torch.ldexp(h, torch.tensor(k)), torch.ldexp(w, torch.tensor(-k))
        got = run_loss(gcq, a, b, y)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), k
        gh, gw = run_grad(gcq, a, b, y, lse, d, torch.float32, torch.float32)
        assert torch.equal(torch.ldexp(gh, torch.tensor(k)), dh), k
        if k < 100:  # (2^100 dh's own values stay finite, and above the subnormal)
            assert torch.equal(torch.ldexp(gw, torch.tensor(-k)), dw), k
    gh, gw = run_grad(gcq, h, w, y, lse, torch.ldexp(d, torch.tensor(-60)), torch.float32, torch.float32)
    assert torch.equal(torch.ldexp(gh, torch.tensor(60)), dh) and torch.equal(torch.ldexp(gw, torch.tensor(60)), dw)


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_flat_bucket_views_and_guards(gcq, t):
    """Inputs and outputs one element into their allocation, as views of a
    flat bucket are: the same bits, and nothing written beside them."""
    announce(f"linear_xent misaligned {t}")
    N, V, D = 70, 301, 128
    h, w, y, d = inputs(N, V, D, t)
    lse = plain_loss(h, w, y)[1].float()
    want = run_grad(gcq, h, w, y, lse, d, t, torch.float32)
    want_loss = run_loss(gcq, h, w, y)
    guards = []

    def off(v, dtype=None):
        buf = torch.full((v.numel() + 40,), 7, dtype=v.dtype if dtype is None else dtype, device=gu.DEV)
        view = buf[1:1 + v.numel()].view(v.shape)
        view.copy_(v)
        guards.append(buf)
        return view
    dev = [off(x) for x in (h, w, y, lse, d)]
    dh, dw = off(torch.zeros(N, D), t), off(torch.zeros(V, D), torch.float32)
    loss, lse2 = off(torch.zeros(N)), off(torch.zeros(N))
    size = gcq.linear_xent_grad_ws_bytes(N, V, D, t, t, torch.float32)
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.linear_xent_grad(*dev, dh, dw, ws[:size])
    size2 = gcq.linear_xent_loss_ws_bytes(N, V, D, t)
    ws2 = torch.full((size2 + 256,), 255, dtype=torch.uint8, device=gu.DEV)
    gcq.linear_xent_loss(dev[0], dev[1], dev[2], loss, lse2, ws2[:size2])
    gu.sync()
    assert torch.equal(dh.cpu(), want[0]) and torch.equal(dw.cpu(), want[1])
    assert torch.equal(loss.cpu(), want_loss[0]) and torch.equal(lse2.cpu(), want_loss[1])
    assert bool((ws[size:] == 255).all()) and bool((ws2[size2:] == 255).all())
    for buf in guards:
        assert float(buf[0]) == 7 and bool((buf[-39:] == 7).all())


@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32)], ids=str)
def test_several_pieces_and_splits(gcq, types):
    """More tokens x vocabulary than one piece of G holds, a last piece that
    ends inside a tile, and products split over k: against float64 on the
    device, sampled rows in full."""
    t, tw = types
    N, V, D = 4100, 70_003, 72
    announce(f"linear_xent_grad in pieces {types}")
    g = torch.Generator(device=gu.DEV).manual_seed(3)
    h = torch.randn(N, D, generator=g, device=gu.DEV).to(t)
    w = (torch.randn(V, D, generator=g, device=gu.DEV) * 2 / D ** 0.5).to(t)
    y = torch.randint(0, V, (N,), generator=g, device=gu.DEV)
    y[::9] = IGNORE
    d = torch.randn(N, generator=g, device=gu.DEV)
    size = gcq.linear_xent_grad_ws_bytes(N, V, D, t, t, tw)
    # G, of 2 bytes a plane, is never whole
    assert size < 2 * (2 if tw == torch.float32 else 1) * N * V
    loss, lse = torch.empty(N, device=gu.DEV), torch.empty(N, device=gu.DEV)
    gcq.linear_xent_loss(h, w, y, loss, lse,
                         torch.empty(gcq.linear_xent_loss_ws_bytes(N, V, D, t), dtype=torch.uint8, device=gu.DEV))
    dh, dw = torch.empty_like(h), torch.empty(V, D, dtype=tw, device=gu.DEV)
    gcq.linear_xent_grad(h, w, y, lse, d, dh, dw, torch.empty(size, dtype=torch.uint8, device=gu.DEV))
    gu.sync()
    rows = torch.cat([torch.arange(0, N, 311), torch.tensor([N - 1])])
    ref, ref_lse, e = plain_loss(h[rows].cpu(), w.cpu(), y[rows].cpu())
    check_loss(loss[rows].cpu(), lse[rows].cpu(), ref, ref_lse, e)
    rh, eh, _, _ = plain_grad(h[rows].cpu(), w.cpu(), y[rows].cpu(), lse[rows].cpu(), d[rows].cpu(), t, tw)
    check_grad(dh[rows].cpu(), rh, eh + 2.0 ** -36 * float(d.abs().max()) * w.double().abs().sum(0).cpu())
    # rows of the vocabulary on both sides of every piece's and tile's end, and targets
    vocab = torch.unique(torch.cat([torch.arange(0, V, 1021), torch.arange(15_800, V, 256)[::8] + 255, y[y >= 0][:50].cpu(),
                                    torch.tensor([V - 1])]).clamp(max=V - 1))
    l64 = h.double() @ w[vocab.to(gu.DEV)].double().t()
    has = y != IGNORE
    gm = torch.exp(l64 - lse.double()[:, None]) - (y[:, None] == vocab.to(gu.DEV)[None, :]).double()
    gm = torch.where(has[:, None], gm * d.double()[:, None], 0.0)
    ref = gm.t().contiguous() @ torch.where(has[:, None], h.double(), 0.0)
    # per term: the logit's error (D + 2 steps of its magnitude), exp's steps, G's rounding
    rel = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}[tw if tw == torch.float32 else t]
    el = ((D + 2) * po.F32 + 3.1 * 2.0 ** -22) * (h.double().abs() @ w[vocab.to(gu.DEV)].double().abs().t()).max() + 16 * po.F32
    mag = gm.abs().t().contiguous() @ h.double().abs()
    err = mag * (rel + el + (N + 2) * po.F32 + 3.1 * 2.0 ** -22)
    check_grad(dw[vocab.to(gu.DEV)].cpu(), ref.cpu(), err.cpu())


def test_gradient_against_differences(gcq):
    """(f(v + e) - f(v - e)) / 2e of the kernels' own loss, fp32."""
    announce("linear_xent differences")
    h, w, y, d = inputs(6, 40, 32, torch.float32, seed=8)
    lse = run_loss(gcq, h, w, y)[1]
    dh, dw = run_grad(gcq, h, w, y, lse, d, torch.float32, torch.float32)

    def value(k, i, e):
        a, b = h.clone(), w.clone()
        (a if k == "h" else b).view(-1)[i] += e
        return float((run_loss(gcq, a, b, y)[0].double() * d.double()).sum())
    # noise: 6 losses off by at most 300 F each, times |d| < 4, over 2 e; and
    # e^2 / 6 times a third derivative below 4 * 6 * 4^3
    e = 2.0 ** -6
    allowed = 6 * 4 * 300 * po.F32 / (2 * e) + e * e / 6 * 1536
    for k, got in (("h", dh), ("w", dw)):
        for i in (0, 33, 77, got.numel() - 1):
            diff = (value(k, i, e) - value(k, i, -e)) / (2 * e)
            assert abs(diff - float(got.view(-1)[i])) <= allowed, (k, i)


def test_graph_replays_and_streams(gcq):
    """Loss and gradient captured once and replayed on new inputs, and the
    same calls on two streams at once, each with its own workspace."""
    announce("linear_xent in a HIP graph, and on two streams")
    N, V, D = 200, 700, 136
    for t, tw in ((torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)):
        sets = []
        for k in range(2):
            h, w, y, d = [x.to(gu.DEV) for x in inputs(N, V, D, t, seed=k)]
            sets.append(dict(h=h, w=w, y=y, d=d, loss=torch.empty(N, device=gu.DEV), lse=torch.empty(N, device=gu.DEV),
                             dh=torch.empty_like(h), dw=torch.empty(V, D, dtype=tw, device=gu.DEV),
                             ws=torch.empty(max(gcq.linear_xent_loss_ws_bytes(N, V, D, t),
                                                gcq.linear_xent_grad_ws_bytes(N, V, D, t, t, tw)), dtype=torch.uint8,
                                            device=gu.DEV)))

        def body(s, stream=None):
            gcq.linear_xent_loss(s["h"], s["w"], s["y"], s["loss"], s["lse"], s["ws"], stream=stream)
            gcq.linear_xent_grad(s["h"], s["w"], s["y"], s["lse"], s["d"], s["dh"], s["dw"], s["ws"], stream=stream)
        s = sets[0]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            body(s)
        torch.cuda.current_stream().wait_stream(side)
        gu.sync()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body(s)
        for k in range(3):
            new = inputs(N, V, D, t, seed=10 + k)
            for name, v in zip("hwyd", new):
                s[name].copy_(v)
            for name in ("loss", "lse", "dh", "dw"):
                s[name].fill_(float("nan"))
            s["ws"].fill_(255)
            gu.sync()
            graph.replay()
            gu.sync()
            loss, lse = run_loss(gcq, *new[:3])
            dh, dw = run_grad(gcq, *new[:3], lse, new[3], t, tw)
            assert torch.equal(s["loss"].cpu(), loss) and torch.equal(s["lse"].cpu(), lse)
            assert torch.equal(s["dh"].cpu(), dh) and torch.equal(s["dw"].cpu(), dw)
        want = []
        for s in sets:
            body(s)
            gu.sync()
            want.append([s[k].clone() for k in ("loss", "lse", "dh", "dw")])
        streams = [torch.cuda.Stream() for _ in sets]
        gu.sync()
        for _ in range(5):
            for s, st in zip(sets, streams):
                body(s, stream=st)
        gu.sync()
        for s, ref in zip(sets, want):
            for k, r in zip(("loss", "lse", "dh", "dw"), ref):
                assert torch.equal(s[k], r)


@pytest.mark.slow
def test_offsets_past_32_bits(gcq):
    """A weight matrix of 4.6 GB: byte offsets of its rows, and of its
    gradient's, pass 2^32. Against float64 on the device, in pieces."""
    N, V, D = 130, 1_100_003, 2112
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    announce(f"linear_xent V={V} D={D}")
    g = torch.Generator(device=gu.DEV).manual_seed(1)
    w = (torch.empty(V, D, dtype=torch.bfloat16, device=gu.DEV).normal_(generator=g)).mul_(2.0 / D ** 0.5)
    h = torch.randn(N, D, generator=g, device=gu.DEV).to(torch.bfloat16)
    y = torch.randint(V - 70_000, V, (N,), generator=g, device=gu.DEV)
    y[3] = IGNORE
    y[4], y[5] = 0, V - 1
    d = torch.randn(N, generator=g, device=gu.DEV)
    loss, lse = torch.empty(N, device=gu.DEV), torch.empty(N, device=gu.DEV)
    gcq.linear_xent_loss(h, w, y, loss, lse,
                         torch.empty(gcq.linear_xent_loss_ws_bytes(N, V, D, w.dtype), dtype=torch.uint8, device=gu.DEV))
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    gcq.linear_xent_grad(h, w, y, lse, d, dh, dw,
                         torch.empty(gcq.linear_xent_grad_ws_bytes(N, V, D, w.dtype), dtype=torch.uint8, device=gu.DEV))
    gu.sync()
    h64 = h.double()
    sums = torch.zeros(N, dtype=torch.float64, device=gu.DEV)
    target = torch.zeros(N, dtype=torch.float64, device=gu.DEV)
    rh = torch.zeros(N, D, dtype=torch.float64, device=gu.DEV)
    has = y != IGNORE
    dl = torch.where(has, d.double(), 0.0)
    e = (D + 2) * po.F32 * (h64.abs().sum(1).max() * 2.0 / D ** 0.5 * 6)  # |w| stays below 6 deviations
    for lo in range(0, V, 50_000):
        wp = w[lo:lo + 50_000].double()
        l = h64 @ wp.t()
        sums += torch.exp(l).sum(1)
        at = torch.where(has & (y >= lo) & (y < lo + wp.shape[0]), y - lo, -1)
        rows = (at >= 0).nonzero()[:, 0]
        target[rows] = l[rows, at[rows]]
        gm = torch.exp(l - lse.double()[:, None])
        gm[rows, at[rows]] -= 1.0
        gm *= dl[:, None]
        rh += gm @ wp
        ref = gm.t() @ torch.where(has[:, None], h64, 0.0)
        mag = gm.abs().t() @ h64.abs()
        got = dw[lo:lo + 50_000].double()
        assert bool(((got - ref).abs() <= mag * (2.0 ** -8 + e + 300 * po.F32) + ref.abs() * 1.01 * 2.0 ** -8).all()), lo
        # every term of dhidden is off by at most G's rounding and the logit's error
        # and the fp32 sums, 16 products deep at a time, by their steps
        errh = gm.abs() @ wp.abs() * (2.0 ** -8 + e + (V / 16 + 300) * po.F32)
        eh = errh if lo == 0 else eh + errh
    ref_lse = sums.log()
    assert bool(((lse.double() - ref_lse).abs() <= e + 64 * po.F32 * (1 + ref_lse)).all())
    ref = torch.where(has, ref_lse - target, 0.0)
    assert bool(((loss.double() - ref).abs() <= 2 * e + 200 * po.F32 * (1 + ref_lse)).all())
    assert bool(((dh.double() - rh).abs() <= eh + rh.abs() * 1.01 * 2.0 ** -8).all())
    del w, dw
    torch.cuda.empty_cache()


def leading(t, base, N=12, V=400):
    """Logits that are exact in every type: base plus sixteenths, one of each
    row some 10 to 15 above the others. Returns inputs, logits, leaders."""
    g = torch.Generator().manual_seed(17)
    x = torch.randint(0, 32, (V, N), generator=g).double() / 16
    lead = torch.randint(0, V, (N,), generator=g)
    x[lead, torch.arange(N)] = torch.randint(192, 256, (N,), generator=g).double() / 16
    w = torch.cat([torch.full((V, 1), float(base), dtype=torch.float64), x], dim=1).to(t)
    h = torch.cat([torch.ones(N, 1), torch.eye(N)], dim=1).to(t)
    l = h.double() @ w.double().t()
    assert torch.equal(l.float().double(), l) and torch.equal(w.double()[:, 1:], x)
    return h, w, l, lead


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("base", [0, 960, -960, 32768])
def test_loss_of_a_leading_target(gcq, t, base):
    """log(sum) with a sum near 1 is the loss of a confident token, whatever
    the size of its lse. The sum of at most 16 + 3 + 7 rounded additions, the
    leader's exponential and factors (6 steps), log's own steps and those of
    the small terms (some 25 of at most 0.02): 40 F."""
    announce(f"linear_xent_loss of leading targets {t} {base}")
    h, w, l, lead = leading(t, base)
    y = lead.clone()
    y[::4] = (y[::4] + 1) % w.shape[0]  # and some that do not lead
    loss, lse = run_loss(gcq, h, w, y)
    top = l.max(dim=1, keepdim=True).values
    ref = (top - l.gather(1, y[:, None]))[:, 0] + (l - top).exp().sum(1).log()
    assert float(ref[1::4].max()) < 0.02
    assert bool(((loss.double() - ref).abs() <= 40 * po.F32 + 4 * po.F32 * ref.abs()).all())
    ref_lse = torch.logsumexp(l, dim=1)
    assert bool(((lse.double() - ref_lse).abs() <= 40 * po.F32 + 1.01 * po.F32 * ref_lse.abs()).all())
    assert bool((loss >= 0).all())


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("base", [2.0 ** 34, -2.0 ** 34, 2.0 ** 62, -2.0 ** 62, 2.0 ** 126])
def test_logits_of_any_size(gcq, t, base):
    """Logits far beyond those whose exponential's argument still has bits of
    its own: one leads by 2^-6 of the others' size, so that its probability is 1."""
    announce(f"linear_xent_loss of logits of {base} {t}")
    N, V, D = 5, 300, 8
    h, w = torch.ones(N, D).to(t), torch.full((V, D), base / D).to(t)
    lead = torch.tensor([0, 17, 128, 255, 299])
    for n in range(N):
        h[n] = 0
        h[n, n] = D
    w[lead, torch.arange(N)] += base / D / 64 if base > 0 else -base / D / 64
    l = h.double() @ w.double().t()
    loss, lse = run_loss(gcq, h, w, lead)
    assert torch.equal(lse.double(), l.max(dim=1).values) and bool((loss == 0).all())
    loss, lse = run_loss(gcq, h, w, (lead + 1) % V)
    assert torch.equal(loss.double(), (l.max(dim=1).values - base))


@pytest.mark.parametrize("types", CASES, ids=lambda c: "-".join(str(t)[6:] for t in c))
@pytest.mark.parametrize("base", [0, 960, 32768])
def test_grad_of_a_leading_target(gcq, types, base):
    """p - 1 of a confident token, whatever the size of its lse. Each token has
    a channel of its own, h = 1 in it: dweight is G there. p is off by the
    exponential's argument (|l - lse| < 24: two half steps of it), 2 steps of
    exp and one of the difference: 60 F of p for l far below, 8 F of p at the
    target, where |l - lse| < 1; then G's rounding and the output's."""
    t, th, tw = types
    announce(f"linear_xent_grad of leading targets {types} {base}")
    h, w, l, lead = leading(t, base)
    N, V = h.shape[0], w.shape[0]
    lse = torch.logsumexp(l, dim=1).float()
    d = torch.ones(N)
    dh, dw = run_grad(gcq, h, w, lead, lse, d, th, tw)
    p = (l - lse.double()[:, None]).exp()
    assert float(p.gather(1, lead[:, None]).min()) > 0.5
    g = p.clone()
    g[torch.arange(N), lead] -= 1.0
    rounding = 2.0 ** -22 if tw == torch.float32 else po.HALF_STEP[t] if th == t == tw else 2.0 ** -11
    off = (dw.double()[:, 1:].t() - g).abs()
    # (a p of 1e-7 is subnormal in fp16, a multiple of 2^-24: off by half of that)
    allowed = 60 * po.F32 * p + g.abs() * (1.01 * rounding + 1.01 * po.HALF_STEP[tw]) + 2.0 ** -38 + po.TINY[tw]
    allowed[torch.arange(N), lead] += 8 * po.F32
    assert bool((off <= allowed).all()), float((off / allowed).max())


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_lse_of_rows_without_a_target(gcq, t):
    """Padded rows some times larger than the others have an lse like any
    other row, and no row's size costs another one bits."""
    announce(f"linear_xent_loss lse of padded rows {t}")
    N, V, D = 80, 300, 96
    h, w, y, _ = inputs(N, V, D, t, seed=12, ignore=0.0)
    y[::3] = IGNORE
    want = run_loss(gcq, h, w, y)
    for k in (2, 4, 7):
        big = h.clone()
        big[::3] = torch.ldexp(h[::3].float(), torch.tensor(k)).to(t)
        loss, lse = run_loss(gcq, big, w, y)
        rest = torch.arange(N) % 3 != 0
        assert torch.equal(loss[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])
        for n in range(0, N, 3):  # each with the bounds of its own size
            ref, ref_lse, e = plain_loss(big[n:n + 1], w, y[n:n + 1])
            check_loss(loss[n:n + 1], lse[n:n + 1], ref, ref_lse, e)
    # of a token with a target too, however large
    if t != torch.float16:
        big = h.clone()
        big[1] = torch.ldexp(h[1].float(), torch.tensor(60)).to(t)
        loss, lse = run_loss(gcq, big, w, y)
        rest = torch.arange(N) != 1
        assert torch.equal(loss[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])
        ref, ref_lse, e = plain_loss(big[1:2], w, y[1:2])
        check_loss(loss[1:2], lse[1:2], ref, ref_lse, e)


@pytest.mark.parametrize("types", CASES, ids=lambda c: "-".join(str(t)[6:] for t in c))
def test_range_of_small_probabilities(gcq, types):
    """Probabilities down to e^-60, next to |dloss| up to 1. Each token has a
    channel of its own with h = 1: dweight is G there. G in bf16 has no floor.
    Two planes of fp16, the largest |dloss| of them at 2^14 or more, are off by
    half of 2^-24 times 2^-11 at least, 2^-50 of it, one by 2^-39, which
    no fp16 output can tell from 0."""
    t, th, tw = types
    announce(f"linear_xent_grad of small probabilities {types}")
    N, V = 6, 250
    g = torch.Generator().manual_seed(2)
    x = -torch.randint(0, 241, (V, N), generator=g).double() / 4
    x[0] = 0
    h, w = torch.eye(N).to(t), x.to(t)
    y, d = torch.zeros(N, dtype=torch.int64), torch.tensor([1.0, -1.0, 0.5, 2.0 ** -6, 2.0 ** -10, -2.0 ** -12])
    l = h.double() @ w.double().t()
    lse = torch.logsumexp(l, dim=1).float()
    dh, dw = run_grad(gcq, h, w, y, lse, d, th, tw)
    p = (l - lse.double()[:, None]).exp()
    gm = p.clone()
    gm[:, 0] -= 1.0
    gm *= d.double()[:, None]
    wide = torch.float32 in (th, tw)
    if t == torch.bfloat16 and not wide:
        rounding, floor = po.HALF_STEP[t], 0.0
    elif tw == torch.float32 or t == torch.bfloat16:
        rounding, floor = 2.0 ** -22, 2.0 ** -50
    else:
        rounding, floor = 2.0 ** -11, 2.0 ** -39
    # |l - lse| < 64: its difference, and two half steps of the argument; exp
    ep = d.double().abs()[:, None] * (p * 200 * po.F32)
    ep[:, 0] += 4 * po.F32 * d.double().abs()
    off = (dw.double().t() - gm).abs()
    allowed = ep + gm.abs() * 1.01 * (rounding + po.HALF_STEP[tw]) + 1.01 * floor + po.TINY[tw]
    assert bool((off <= allowed).all()), float((off / allowed).max())


@pytest.mark.parametrize("types", [c for c in CASES if c[0] != torch.float16],
                         ids=lambda c: "-".join(str(t)[6:] for t in c))
@pytest.mark.parametrize("base", [2.0 ** 34, -2.0 ** 62])
def test_grad_of_logits_of_any_size(gcq, types, base):
    """One logit leads by far more than an exponential holds: p is 1 there and 0
    elsewhere, and every product of the gradient is exact."""
    t, th, tw = types
    announce(f"linear_xent_grad of logits of {base} {types}")
    N, V, D = 5, 300, 8
    h, w = (torch.eye(N, D) * D).to(t), torch.full((V, D), base / D).to(t)
    lead = torch.tensor([0, 17, 128, 255, 299])
    w[lead, torch.arange(N)] += abs(base) / D / 64
    y = lead.clone()
    y[::2] = (y[::2] + 3) % V
    d = torch.tensor([1.0, -0.5, 2.0, 0.25, 1.0])
    lse = (h.double() @ w.double().t()).max(dim=1).values.float()
    dh, dw = run_grad(gcq, h, w, y, lse, d, th, tw)
    g = torch.zeros(N, V, dtype=torch.float64)
    g[torch.arange(N), lead] += d.double()
    g[torch.arange(N), y] -= d.double()
    assert torch.equal(dw.double(), g.t() @ h.double())
    ref = g @ w.double()
    assert bool(((dh.double() - ref).abs() <= ref.abs() * po.HALF_STEP[th] + abs(base) * 2.0 ** -21).all())
