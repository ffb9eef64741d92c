"""What the bounds of rounded_newton_schulz.py tell apart, without a GPU."""
import pytest
import torch

from rounded_newton_schulz import allowed, lines, rounded

QUINTIC = ((3.4445, -4.7750, 2.0315),) * 5
EPS = 1e-7


def exact(x, series, eps=EPS):
    x = x.double()
    x = x / (x.square().sum().sqrt() + eps)
    for a, b, c in series:
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x


@pytest.mark.parametrize("shape", [(17, 20), (64, 576), (100, 300), (128, 256), (290, 300)], ids=str)
@pytest.mark.parametrize("strong", [True, False])
def test_diagonals_in_the_planes_and_lost_lines_are_seen(shape, strong):
    g = torch.Generator().manual_seed(sum(shape))
    x = 0.5 * torch.randn(*shape, generator=g)
    if strong:
        x = x + (torch.randn(shape[0], 8, generator=g) * 2.0 ** -torch.arange(8)) @ torch.randn(8, shape[1], generator=g)
    ref = exact(x, QUINTIC)
    matrix, line = allowed(x, ref, QUINTIC, False, EPS)
    assert matrix < 1e-2 and line < 1e-2
    # another draw passes, the diagonals of A and P rounded with the rest do not
    off = rounded(x, QUINTIC, False, EPS, noise=torch.Generator().manual_seed(99)) - ref
    assert float(off.norm() / ref.norm()) <= matrix and float((lines(off) / lines(ref)).max()) <= line
    off = rounded(x, QUINTIC, False, EPS, diagonals_apart=False) - ref
    assert float(off.norm() / ref.norm()) > matrix
    # nor does a column of zeros
    off = torch.zeros_like(ref)
    off[:, -1] = ref[:, -1]
    assert float((lines(off) / lines(ref)).max()) > line


def test_both_planes_are_a_thousand_times_nearer():
    x = torch.randn(64, 200, generator=torch.Generator().manual_seed(1))
    ref = exact(x, QUINTIC)
    one, both = (allowed(x, ref, QUINTIC, b, EPS)[0] for b in (False, True))
    assert both < one / 100
