"""Plain 64-bit form of the orthogonalised update, and bounds on what its fp16 terms may add.

A step is X -> f(X), f(s) = a s + b s^3 + c s^5 on the singular values.  An error D made in step k reaches the result
through the derivative of the remaining steps' f, whose norm (Frobenius to Frobenius) is the largest divided difference
|f(s) - f(t)| / |s - t| and |f(s) + f(t)| / (s + t) over pairs of X's singular values, 0 among them where X is not
square.  Summed over the steps that is the first-order bound; twice it is allowed for what is of second order.
"""
import math

import torch

from tests._train_ref import U

COEF = (3.4445, -4.7750, 2.0315)
H16, H22 = 2.0 ** -11, 2.0 ** -22  # half steps of one fp16 term and of two


def coefs(coef, steps):
    """fp32 values, as the calls take them."""
    c = coef if coef is not None and hasattr(coef[0], "__len__") else [coef or COEF] * steps
    return [[float(torch.tensor(v, dtype=torch.float32)) for v in t] for t in c]


def newton64(u, steps=5, coef=None, eps=1e-7):
    """o of one matrix u [R, K]."""
    x = u.detach().cpu().double()
    n = x.norm() + eps
    x = x / n if n > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in coefs(coef, steps):
        g = x @ x.t()
        x = a * x + (b * g + c * g @ g) @ x
    return x.t().contiguous() if tall else x


def _gain(s, f, square):
    """Largest divided difference of values f at points s, all >= 0."""
    if not square:
        s, f = torch.cat([s, s.new_zeros(1)]), torch.cat([f, f.new_zeros(1)])
    ds, df = s[:, None] - s[None, :], f[:, None] - f[None, :]
    ss, sf = s[:, None] + s[None, :], f[:, None] + f[None, :]
    near = 1e-6 * s.max()
    a = (df.abs() / ds.abs().clamp(min=near)).where(ds.abs() > near, torch.zeros_like(ds)).max()
    b = (sf.abs() / ss.clamp(min=near)).where(ss > near, torch.zeros_like(ss)).max()
    return float(max(a, b))


def newton_bound(u, o_dtype, steps=5, coef=None, eps=1e-7):
    """Bound of |o - newton64(u)|_F, before o's own rounding.

    One step in fp16 terms.  h is X to H (11 bits in one term, 22 in two), so A = h h^T is off by 2 |X|_2 H |X|_F, by A's own
    rounding H |A|_F, and by its sums' roundings, whose number is at most K and which are as often up as down:
    2 sqrt(K) u |A|_F.  Through P = b A + c A^2 an error D becomes at most max |b + c (l + l')| D over eigenvalues of A (the
    divided difference of a quadratic), and P's rounding adds H |P|_F, its sums 2 sqrt(m) u |c| |A^2|_F.  Then
    X' = a X + P h: (error of P) |X|_2 + |P|_2 H |X|_F + 2 sqrt(m) u |P X|_F, and what X' is held to, H22 |X'|_F + u-sized
    roundings of the sum.  The first X is off by H22 and a few u."""
    H = H16 if o_dtype == torch.bfloat16 else H22
    x = u.detach().cpu().double()
    x = x / (x.norm() + eps)
    x = x.t() if x.shape[0] > x.shape[1] else x
    m, n = x.shape
    s = torch.linalg.svdvals(x)
    cs = coefs(coef, steps)
    path = [s]
    for a, b, c in cs:
        t = path[-1]
        path.append(a * t + b * t ** 3 + c * t ** 5)
    assert all((t >= 0).all() for t in path), "the gain is counted for values that stay above zero"
    total = (H22 + 4 * U) * _gain(path[0], path[-1], m == n)
    for k, (a, b, c) in enumerate(cs):
        s = path[k]
        l = s ** 2
        p = b * l + c * l ** 2
        F = lambda v: float((v ** 2).sum().sqrt())  # noqa: E731
        top, low = float(l.max()), float(l.min())
        dA = 2 * float(s.max()) * H * F(s) + H * F(l) + 2 * math.sqrt(n) * U * F(l)
        slope = max(abs(b + 2 * c * top), abs(b + 2 * c * low))
        dP = slope * dA + H * F(p) + 2 * math.sqrt(m) * U * abs(c) * F(l ** 2) + 4 * U * (abs(b) * F(l) + F(p))
        dX = dP * float(s.max()) + float(p.abs().max()) * H * F(s) + 2 * math.sqrt(m) * U * F(p * s)
        dX += H22 * F(path[k + 1]) + 4 * U * abs(a) * F(s)
        total += dX * _gain(path[k + 1], path[-1], m == n)
    # below fp16's normal range the terms are off by up to 2^-25 of 2^-13, counted for every value of X in every step
    return 2 * total + steps * 2.0 ** -38 * math.sqrt(m * n) * _gain(path[0], path[-1], m == n)


def scalar_bound(d, norm, o_dtype, steps=5, coef=None):
    """(o, bound) of matrices with one value d in each row and column: each step acts on every value by itself, and A
    and P are diagonal.  With h = x (1 + H): A = x^2 (1 + 3 H) (two of h, one of its own), p = b A + c A^2 in fp32 and never rounded
    below it, x' = a x + p h; 4 u for the roundings of the sums, H22 for what x' is held to."""
    H = H16 if o_dtype == torch.bfloat16 else H22
    x = d.double().abs() / norm
    e = x * (H22 + 4 * U)
    for a, b, c in coefs(coef, steps):
        A = x * x
        p = b * A + c * A * A
        dp = ((b + 2 * c * A).abs() * A + abs(c) * 3 * H * A * A) * 3 * H + 4 * U * (abs(b) * A + abs(c) * A * A)
        new = a * x + p * x
        slope = (a + 3 * b * A + 5 * c * A * A).abs()
        e = slope * e + 20 * e * e + dp * x * (1 + H) + p.abs() * x * H + 4 * U * (a * x + p.abs() * x) + H22 * new.abs()
        x = new
    return x * torch.sign(d.double()), e
