"""The operators together, as a data-parallel step uses them: W workers run
the end of a block (norms, dropout, gate, residual) and the vocabulary's loss,
go back through both, and compress the gradients where the operators wrote
them; the reducer sums the blocks. Against the same step in 64 bits and the
oracle's compression of the very gradients that the kernels produced."""
import math

import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32], ids=str)
def test_step_of_w_workers(gcq, t):
    W, rows, V, D, thr, p, seed = 3, 96, 517, 192, 0.002, 0.1, 21
    announce(f"training step with compression {t}")
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    post, pre, gate = 1 + 0.1 * n(D), 1 + 0.1 * n(D), 0.5 + 0.2 * n(1, D)
    weight = (n(V, D) * 2 / math.sqrt(D)).to(t)
    P = [v.to(gu.DEV) for v in (post, pre, gate, weight)]
    sizes = [V * D, D, D, D]
    blocks, exact = [], []
    for w in range(W):
        x, y = n(rows, D).to(t), n(rows, D).to(t)
        target = torch.randint(0, V, (rows,), generator=g)
        target[::5] = -100
        dev = lambda v: v.to(gu.DEV)  # noqa: E731
        xd, yd, td = dev(x), dev(y), dev(target)
        z, h, dh, dx, dy = (torch.empty_like(xd) for _ in range(5))
        rp, rz, loss, lse = (torch.empty(rows, device=gu.DEV) for _ in range(4))
        dloss = torch.full((rows,), 1.0 / rows, device=gu.DEV)
        # one flat bucket of fp32 gradients, as the compressor's plan holds it
        bucket = torch.full((sum(sizes),), float("nan"), device=gu.DEV)
        grads = list(bucket.split(sizes))
        residuals = [torch.zeros(k, device=gu.DEV) for k in sizes]
        plan = gcq.Plan2bitMulti(grads, residuals)
        compr = torch.empty(plan.compressed_words, dtype=torch.int32, device=gu.DEV)
        kw = dict(post_gain=P[0], gate=P[2], pre_gain=P[1], residual_scale=0.5, p=p, seed=seed, worker=w, rstd_post=rp,
                  rstd_pre=rz)
        size = max(gcq.linear_xent_loss_ws_bytes(rows, V, D, t),
                   gcq.linear_xent_grad_ws_bytes(rows, V, D, t, t, torch.float32),
                   gcq.norm_residual_grad_ws_bytes(rows, D))
        ws = torch.empty(size, dtype=torch.uint8, device=gu.DEV)  # shared: the calls are in order
        gcq.norm_residual(xd, yd, z, h=h, **kw)
        gcq.linear_xent_loss(h, P[3], td, loss, lse, ws)
        gcq.linear_xent_grad(h, P[3], td, lse, dloss, dh, grads[0].view(V, D), ws)
        gcq.norm_residual_grad(z, yd, dx, dy, ws, dh=dh, dpost_gain=grads[1], dpre_gain=grads[2],
                               dgate=grads[3].view(1, D), **kw)
        plan.compress(-thr, thr, compr)
        gu.sync()
        # the compressed words are the oracle's of these gradients
        words = gu.host(compr, np.uint32)
        for k, off in enumerate(plan.block_offsets()):
            gk = gu.host(grads[k])
            assert np.isfinite(gk).all()
            ref = oracle.quantize_2bit(gk, np.zeros(sizes[k], np.float32), -thr, thr)
            np.testing.assert_array_equal(words[off:off + ref.size], ref)
        blocks.append((compr, plan.block_offsets()))

        # the whole step in 64 bits, by autograd
        leaf = [v.double().requires_grad_() for v in (weight, post, pre, gate)]
        f = po.factor(rows * D, p, seed, w).reshape(rows, D)
        y64 = y.double()
        u = y64 * (y64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * leaf[1]
        z64 = 0.5 * x.double() + leaf[3] * (u * f)
        h64 = z64 * (z64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * leaf[2]
        l64 = torch.nn.functional.cross_entropy(h64 @ leaf[0].t(), target, ignore_index=-100, reduction="sum") / rows
        l64.backward()
        # roundings of z, h and dh to t reach every gradient: four half steps
        # of its norm, ten times over for what they meet on the way
        for got, ref in zip(grads, leaf):
            off = (got.cpu().double() - ref.grad.reshape(-1)).norm() / ref.grad.norm()
            assert float(off) < 40 * max(po.HALF_STEP[t], 2.0 ** -20), (t, float(off))
        assert abs(float(loss.cpu().double().sum()) / rows - float(l64.detach())) < 40 * po.HALF_STEP[t]
        exact.append([gu.host(v) for v in grads])
        plan.destroy()

    # the reducer's sum of the vocabulary gradient
    out = torch.empty(V * D, device=gu.DEV)
    words = gcq.gc_compressed_2bit_words(V * D)
    gcq.decompress_2bit_sum([c[o[0]:o[0] + words] for c, o in blocks], V * D, out)
    gu.sync()
    ref = oracle.dequantize_2bit_sum([gu.host(c, np.uint32)[o[0]:o[0] + words] for c, o in blocks], V * D)
    np.testing.assert_array_equal(gu.host(out), ref)
