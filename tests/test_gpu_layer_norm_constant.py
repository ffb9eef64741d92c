"""Rows of one value have no deviations: h is the bias, mean the value, whatever
their size, their length and eps. (The sum over a row and its quotient round;
what that leaves, divided by an eps of 1e-12, was of the size of the gain.)"""
import pytest
import torch

from conftest import announce

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")

VALUES = [3.25, 100.0, -7.5, 0.1, 1000.3, -31.7, 1e6, 3e-5]


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("d", [1, 5, 257, 768, 1000, 1001, 2040, 4104, 6000, 9001, 12288, 16384])
@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_rows_of_one_value(gcq, d, t, eps):
    announce(f"layer_norm rows of one value {d} {t} {eps}")
    g = torch.Generator().manual_seed(d)
    bias, gain = torch.randn(d, generator=g).to(gu.DEV), torch.randn(d, generator=g).to(gu.DEV)
    values = torch.tensor([v for v in VALUES if t != torch.float16 or abs(v) < 6e4]).to(t)
    x = values[:, None].repeat(1, d).to(gu.DEV)
    h = torch.full_like(x, float("nan"))
    mean = torch.full((len(values),), float("nan"), device=gu.DEV)
    gcq.layer_norm(x, h, gain=gain, bias=bias, eps=eps, mean=mean)
    gu.sync()
    assert torch.equal(mean.cpu(), values.float())
    assert torch.equal(h, bias.to(t).expand_as(h)), float((h - bias).abs().max())
    # the same as a sum: x + y of rows that cancel
    y = (torch.randn(len(values), d, generator=g) * 0.5).to(t).to(gu.DEV)
    z = torch.full_like(x, float("nan"))
    gcq.layer_norm(-y, h, y=y, z=z, gain=gain, bias=bias, eps=eps, mean=mean)
    gu.sync()
    assert bool((z == 0).all()) and bool((mean == 0).all())
    assert torch.equal(h, bias.to(t).expand_as(h))


@pytest.mark.parametrize("d", [64, 768, 4104, 12288])
def test_squares_past_fp32(gcq, d):
    """Deviations of 1e25 have an infinite variance in fp32, and rstd is 0."""
    announce(f"layer_norm squares past fp32 {d}")
    g = torch.Generator().manual_seed(d)
    x, bias = (torch.randn(4, d, generator=g) * 1e25).to(gu.DEV), torch.randn(d, generator=g).to(gu.DEV)
    x[1] = torch.randn(d, generator=g).to(gu.DEV)
    h, rstd = torch.full_like(x, float("nan")), torch.full((4,), float("nan"), device=gu.DEV)
    gcq.layer_norm(x, h, bias=bias, rstd=rstd)
    gu.sync()
    rows = torch.tensor([0, 2, 3], device=gu.DEV)
    assert bool((rstd[rows] == 0).all()) and torch.equal(h[rows], bias.expand(3, d))
    assert bool(h[1].isfinite().all()) and float(rstd[1]) > 0.5


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("d", [5, 100, 768, 1001, 2048, 4096, 6000, 8200, 12288, 16384])
def test_mean_of_sums_that_are_exact(gcq, d, t):
    """Small whole numbers have exact sums, however large their deviations are next
    to the mean: 1 / d and its product round, and nothing else."""
    announce(f"layer_norm mean of whole numbers {d} {t}")
    g = torch.Generator().manual_seed(d)
    x = torch.randint(-100, 101, (300, d), generator=g)
    mean = torch.full((300,), float("nan"), device=gu.DEV)
    x_dev = x.to(t).to(gu.DEV)
    gcq.layer_norm(x_dev, torch.empty_like(x_dev), mean=mean)
    gu.sync()
    ref = x.double().sum(1) / d
    off = (mean.cpu().double() - ref).abs()
    assert bool((off <= 2.01 * 2.0 ** -24 * ref.abs()).all()), float((off / ref.abs()).nan_to_num(0.0).max())
