"""orthogonalize()'s iteration in 64 bits with its roundings where the kernels
have them: the factors of the products as fp16 planes (one, or two that add up),
the diagonals of A and P apart. What fp32 sums add is left out, or drawn: a sum of K
terms is off by some 2^-24 sqrt(K) / 2 of the root of its terms' squares."""
import math

import torch

X_EXP, A_EXP, P_EXP = 14, 12, 10  # powers of two that X, A and P are held times


def planes(v, exponent, both):
    """[first plane, second (zeros unless `both`)], in units of v."""
    s = v * 2.0 ** exponent
    p0 = s.half().double()
    p1 = (s - p0).half().double() if both else torch.zeros_like(p0)
    return p0 * 2.0 ** -exponent, p1 * 2.0 ** -exponent


def product(a, b, noise):
    """a b of planes, without that of two second ones."""
    p = a[0] @ b[0] + a[0] @ b[1] + a[1] @ b[0]
    if noise is not None:
        size = (a[0].square() @ b[0].square()).sqrt() * (2.0 ** -25 * math.sqrt(a[0].shape[1]))
        p = p + size * torch.randn(p.shape, generator=noise, dtype=p.dtype)
    return p


def rounded(x, series, both, eps, diagonals_apart=True, noise=None):
    """noise: a generator that draws the errors of fp32 sums."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x / (x.square().sum().sqrt() + eps)
    x = x.t() if tall else x
    for a, b, c in series:
        held = planes(x, X_EXP, True)  # what is carried
        f = (held[0], held[1] if both else torch.zeros_like(x))
        A = product(f, (f[0].t(), f[1].t()), noise)
        if noise is not None:  # (symmetric in the kernels)
            A = torch.tril(A) + torch.tril(A, -1).t()
        d = A.diagonal().clone() if diagonals_apart else torch.zeros(A.shape[0], dtype=A.dtype)
        if diagonals_apart:
            A.fill_diagonal_(0.0)
        A = planes(A, A_EXP, both)
        square = product(A, A, noise)
        if noise is not None:
            square = torch.tril(square) + torch.tril(square, -1).t()
        P = (b + c * (d[:, None] + d[None, :])) * (A[0] + A[1]) + c * square
        p = torch.zeros_like(d)
        if diagonals_apart:
            p = (b + c * d) * d + c * square.diagonal()
            P.fill_diagonal_(0.0)
        x = (a + p)[:, None] * (held[0] + held[1]) + product(planes(P, P_EXP, both), f, noise)
    return x.t() if tall else x


def lines(v):
    """Norms of the rows and of the columns."""
    return torch.cat([v.norm(dim=1), v.norm(dim=0)])


def allowed(x, ref, series, both, eps):
    """(matrix, lines): how far a result may be off `ref`, which is exact, relative
    to its norm and to those of its rows and columns. After the first step the
    roundings of two computations with different fp32 sums have little in common:
    the errors of a kernel are one more draw of what five draws here show. The
    matrix's is a sum over thousands of roundings, 1.3 times the largest draw's; a
    line's is one over its 17 values or more, and of hundreds of lines the
    largest is taken, 1.5 times. Where both planes are multiplied the sums, whose
    order the drawn size leaves open, are most of it: twice that."""
    draws = [rounded(x, series, both, eps, noise=None if k == 0 else torch.Generator().manual_seed(k)) - ref
             for k in range(5)]
    matrix = max(float(e.norm()) for e in draws) / float(ref.norm())
    line = max(float((lines(e) / lines(ref)).max()) for e in draws)
    more = 2.0 if both else 1.0
    return 1.3 * more * matrix, 1.5 * more * line
