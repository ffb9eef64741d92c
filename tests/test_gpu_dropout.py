"""dropout and dropout_backward against the formula in 64 bits: the mask of
every value exactly, the values within their roundings."""
import numpy as np
import pytest
import torch

import oracle
import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def values(n, t, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).to(t)


def check(out, x, f, r, t):
    """x * fl(1/(1-p)): two fp32 roundings; the residual's sum: one; the
    output's own type: one more."""
    out, x = out.cpu().double(), x.cpu().double()
    prod = x * f
    expect = prod if r is None else prod + r.cpu().double()
    allowed = prod.abs() * 2.5 * po.F32 + expect.abs() * (1.01 * po.HALF_STEP[t] + 1.5 * po.F32) + po.TINY[t]
    assert bool(((out - expect).abs() <= allowed).all())
    assert bool((out[f == 0] == (0.0 if r is None else r.cpu().double()[f == 0])).all())


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n", [1, 3, 4, 5, 7, 8, 1023, 4096, 4097, 70_001])
def test_dropout_and_its_gradient(gcq, t, n):
    announce(f"dropout n={n} {t}")
    for p, seed, worker, offset in ((0.1, 7, 0, 0), (0.5, 2 ** 63 + 11, 3, 8), (0.3, 5, 2 ** 32 - 1, 2 ** 34 + 3)):
        x, r = values(n, t, n).to(gu.DEV), values(n, t, n + 1).to(gu.DEV)
        f = po.factor(n, p, seed, worker, offset)
        out = torch.full_like(x, float("nan"))
        gcq.dropout(x, p, seed, worker, out, offset=offset)
        check(out, x, f, None, t)
        gcq.dropout(x, p, seed, worker, out, residual=r, offset=offset)
        check(out, x, f, r, t)
        dx = torch.full_like(x, float("nan"))
        gcq.dropout_backward(r, p, seed, worker, dx, offset=offset)
        check(dx, r, f, None, t)
        # in place, over the values and over the residual
        y = x.clone()
        gcq.dropout(y, p, seed, worker, y, offset=offset)
        z = r.clone()
        gcq.dropout(x, p, seed, worker, z, residual=z, offset=offset)
        gu.sync()
        check(y, x, f, None, t)
        assert torch.equal(z, out)


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_alignment_does_not_change_the_result(gcq, t):
    n = 20_003
    announce(f"dropout misaligned {t}")
    x = values(n + 16, t).to(gu.DEV)
    for start in (0, 1, 4, 8):
        a = x[start:start + n]
        out = torch.empty(n + 3, dtype=t, device=gu.DEV)[3 if start == 1 else 0:][:n]
        guard = torch.empty(n, dtype=t, device=gu.DEV)
        gcq.dropout(a, 0.2, 9, 1, out)
        gcq.dropout(a.clone(), 0.2, 9, 1, guard)
        gu.sync()
        assert torch.equal(out, guard)


@pytest.mark.parametrize("offset", [0, 2])
def test_nothing_outside_the_output_is_written(gcq, offset):
    for t in TYPES:
        for n in (1, 9, 4099):
            announce(f"dropout guard {t} n={n}")
            buf = torch.full((n + 64,), 3.0, dtype=t, device=gu.DEV)
            gcq.dropout(values(n, t).to(gu.DEV), 0.5, 1, 1, buf[32:32 + n], offset=offset)
            gu.sync()
            assert bool((buf[:32] == 3.0).all()) and bool((buf[32 + n:] == 3.0).all())


def test_edges_of_p_and_dropped_specials(gcq):
    n = 4103
    announce("dropout p = 0, p = 1, NaN and infinities where dropped")
    x = values(n, torch.float32).to(gu.DEV)
    out = torch.empty_like(x)
    gcq.dropout(x, 0.0, 1, 0, out)
    assert torch.equal(out, x)
    gcq.dropout(x, 1.0, 1, 0, out)
    assert bool((out == 0).all())
    f = po.factor(n, 0.5, 1, 0)
    bad = torch.where(f.to(gu.DEV) == 0, torch.tensor(float("nan"), device=gu.DEV), x)
    bad[(f == 0).nonzero()[::2, 0].to(gu.DEV)] = float("inf")
    gcq.dropout(bad, 0.5, 1, 0, out)
    gu.sync()
    check(out, x, f, None, torch.float32)
    # the smallest probability that can drop anything: only a zero draw falls below it
    gcq.dropout(x, 2.0 ** -24, 1, 0, out)
    gu.sync()
    check(out, x, po.factor(n, 2.0 ** -24, 1, 0), None, torch.float32)


def test_mask_words_are_the_oracles_philox(gcq):
    slots = [0, 1, 2 ** 31, 2 ** 32 + 5]
    for worker, purpose in ((0, 0), (5, 2)):
        got = po.philox(np.array(slots, np.uint64), 0x123456789ABCDEF0, worker, purpose)
        for s, row in zip(slots, got):
            ref = oracle.philox4x32_10((s & 0xFFFFFFFF, s >> 32, worker, purpose), (0x9ABCDEF0, 0x12345678))
            assert list(row) == list(ref)


def test_workers_and_seeds_draw_apart(gcq):
    n = 1 << 20
    announce("dropout keep rates and pairs of workers")
    x = torch.ones(n, device=gu.DEV)
    outs = []
    for seed, worker in ((1, 0), (1, 1), (2, 0)):
        out = torch.empty_like(x)
        gcq.dropout(x, 0.25, seed, worker, out)
        outs.append(out != 0)
    gu.sync()
    # 6 standard deviations of a binomial share
    six = 6 * (0.25 * 0.75 / n) ** 0.5
    for k in outs:
        assert abs(float(k.double().mean()) - 0.75) < six
    for a, b in ((0, 1), (0, 2), (1, 2)):
        both = float((outs[a] & outs[b]).double().mean())
        assert abs(both - 0.75 ** 2) < 6 * (0.75 ** 2 * (1 - 0.75 ** 2) / n) ** 0.5


def test_step_counter_in_a_graph(gcq):
    """A captured forward and backward, replayed: the device counter moves the
    mask, and both use the same one."""
    n = 10_001
    announce("dropout in a HIP graph with a device step")
    x, g = values(n, torch.bfloat16).to(gu.DEV), values(n, torch.bfloat16, 1).to(gu.DEV)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    step = torch.zeros(1, dtype=torch.int64, device=gu.DEV)

    def body():
        gcq.dropout(x, 0.4, 2 ** 64 - 2, 6, out, step=step)
        gcq.dropout_backward(g, 0.4, 2 ** 64 - 2, 6, dx, step=step)
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
    for t in range(1, 5):
        out.fill_(7.0)
        dx.fill_(7.0)
        graph.replay()
        gu.sync()
        f = po.factor(n, 0.4, (2 ** 64 - 2 + t) % 2 ** 64, 6)
        check(out, x, f, None, torch.bfloat16)
        check(dx, g, f, None, torch.bfloat16)


def test_grid_strides_over_many_tiles(gcq):
    """More values than one launch's workgroups take (2^20 tiles of 2048
    fp32 values at most): the striding form, checked by the mask's own
    repetition and at both ends."""
    n = (1 << 31) + 4097
    free, _ = torch.cuda.mem_get_info()
    if free < 4 * n * 2 + (4 << 30):
        pytest.skip("needs 20 GiB of device memory")
    announce(f"dropout n={n}")
    x = torch.ones(n, dtype=torch.float32, device=gu.DEV)
    gcq.dropout(x, 0.5, 3, 2, x)
    gu.sync()
    for lo in (0, (1 << 31) - 2048, n - 4000):
        f = po.factor(4000, 0.5, 3, 2, lo)
        assert torch.equal(x[lo:lo + 4000].cpu().double(), f)
    del x
    torch.cuda.empty_cache()


def test_the_last_indices(gcq):
    """offset + n = 2^64, and not one value more."""
    announce("dropout up to index 2^64 - 1")
    for n in (1, 4, 9, 8192, 8195):
        x = values(n, torch.float32, n).to(gu.DEV)
        out = torch.full_like(x, float("nan"))
        gcq.dropout(x, 0.5, 4, 1, out, offset=2 ** 64 - n)
        check(out, x, po.factor(n, 0.5, 4, 1, 2 ** 64 - n), None, torch.float32)
        gcq.dropout_backward(x, 0.5, 4, 1, out, offset=2 ** 64 - n)
        check(out, x, po.factor(n, 0.5, 4, 1, 2 ** 64 - n), None, torch.float32)
        if n > 1:
            with pytest.raises(gcq.GcqError, match="exceeds 2"):
                gcq.dropout(x, 0.5, 4, 1, out, offset=2 ** 64 - n + 1)
