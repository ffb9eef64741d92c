"""muon_step's momentum and what it orthogonalises, value by value, where
gradients are far larger (or smaller) than the momenta that they move: a running
mean at a momentum of 0.95 is a sixth of gradients that are noise.

With w the smaller of beta and 1 - beta, a mix of two values p and q is p + w (q
- p), p the one with the larger weight: the difference, w and the sum round once
each (F = 2^-24 of |q - p|, of w, of the result), and a relative F each of what
went into p and q."""
import pytest
import torch

import plain_ops as po
from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

F = po.F32
SCALE = 0.3  # of the gradients: not a power of two
SHAPES = [(40, 90), (200, 70), (300, 257), (130, 520)]  # in one workgroup, and in tiles; wide and tall


def mix(g, eg, m, em, beta):
    """(value, what it may be off by) of (1 - beta) g + beta m, of g and m that
    may be off by eg and em."""
    p, q, w = (m, g, 1.0 - beta) if beta >= 0.5 else (g, m, beta)
    v = p + w * (q - p)
    return v, 1.01 * ((1.0 - beta) * eg + beta * em + F * (2 * w * (q - p).abs() + v.abs()))


def case(m, n, ratio, seed=0):
    g = torch.Generator().manual_seed(seed)
    return ratio / SCALE * torch.randn(m, n, generator=g), torch.randn(m, n, generator=g)


def exact(grad, m0, beta, nesterov):
    """(value, error) of the new momentum and of u."""
    # (the scale is an fp32 argument)
    g = float(torch.tensor(SCALE, dtype=torch.float32)) * grad.double()
    m1 = mix(g, F * g.abs(), m0.double(), 0.0, beta)
    return m1, mix(g, F * g.abs(), *m1, beta) if nesterov else m1


@pytest.mark.parametrize("beta", [0.0, 0.3, 0.5, 0.9, 0.95, 0.999, 1.0 - 2.0 ** -30])
@pytest.mark.parametrize("ratio", [0.03, 1.0, 6.0, 30.0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_and_direction(gcq, shape, ratio, beta, nesterov):
    """One step of X <- X writes u / |u| as the update of weights of zero: its
    scale is fp32's, and X is held to 2^-22."""
    announce(f"muon_step momentum {shape} ratio {ratio} beta {beta} nesterov={nesterov}")
    grad, m0 = case(*shape, ratio, seed=shape[0])
    (m64, em), (u64, eu) = exact(grad, m0, beta, nesterov)
    g, m = grad.to(gu.DEV), m0.to(gu.DEV)
    m1, w1 = torch.full_like(m, float("nan")), torch.full_like(m, float("nan"))
    ws = torch.empty(gcq.muon_step_ws_bytes(1, *shape, torch.float32), dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step([g], [m], [torch.zeros_like(m)], ws, coefficients=((1.0, 0.0, 0.0),), eps=0.0, momentum=beta,
                  nesterov=nesterov, grad_scale=SCALE, lr=-1.0, new_momenta=[m1], new_weights=[w1])
    gu.sync()
    off = (m1.cpu().double() - m64).abs()
    assert bool((off <= em).all()), float((off / em).max())
    # |u| is a norm of 64 bits of values that may be off, at most by |eu| (Frobenius);
    # the factor, its product, the scale of the result: 4 F
    norm = float(u64.norm())
    x = u64 / norm
    ex = eu / norm + x.abs() * (float(eu.norm()) / norm + 4 * F + 2.0 ** -22)
    off = (w1.cpu().double() - x).abs()
    # (what lies 2^-25 below 2^-14, the smallest that a second plane holds, is lost)
    assert bool((off <= ex + 2.0 ** -39).all()), float((off / ex).max())


@pytest.mark.parametrize("shape", SHAPES[::2], ids=str)
def test_no_momentum_is_the_gradient(gcq, shape):
    """With a momentum of zero, what the momenta held (not a NaN) does not count."""
    announce(f"muon_step without momentum {shape}")
    grad, m0 = case(*shape, 1e-6)
    g, m, w = grad.to(gu.DEV), m0.to(gu.DEV), torch.zeros(shape, device=gu.DEV)
    ws = torch.empty(gcq.muon_step_ws_bytes(1, *shape, torch.float32), dtype=torch.uint8, device=gu.DEV)
    gcq.muon_step([g], [m], [w], ws, momentum=0.0, grad_scale=1.0)
    gu.sync()
    assert torch.equal(m, g)
