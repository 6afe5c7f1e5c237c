"""Plain 64-bit forms of the training operators, and bounds on what fp32 and bf16 arithmetic may add to them.

u = 2^-24 is fp32's half step, h(t) the half step of a result's type: 2^-24 or 2^-8.  A sum of n rounded terms, in any
order, is off by at most gamma(n) * (sum of magnitudes), gamma(n) = n u / (1 - n u).
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-37  # below fp32's normal range nothing relative holds


def gamma(n):
    return n * U / (1 - n * U)


def within(got, ref, bound, what=""):
    """|got - ref| <= bound everywhere, and finite where ref is."""
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: {(got - ref).abs().max():.3e} off at most, by {over.max():.3e} over its bound"


# ---- dense product ----------------------------------------------------------------

def rows_of(act, N):
    return 2 * N if act == "swiglu" else N


def act64(act, z):
    if act == "none":
        return z
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    g, u = z.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def slope64(act, z):
    """d act / d z for the one-argument activations."""
    if act == "none":
        return torch.ones_like(z)
    if act == "gelu":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    h = torch.sigmoid(z)
    return h + z * h * (1 - h)


def gate_err(act, z):
    """Relative error of the sigmoid behind the activation: its argument v (z, or GELU's 2 v) is rounded a few times
    (relative 4 u, so e^v moves by 4 u |v|), and exp2, 1 + ., the reciprocal and the products add a few u each."""
    v = z.abs() if act != "gelu" else 1.6 * z.abs() * (1 + 0.045 * z * z)
    return (6 * v.clamp(max=200) + 16) * U


def linear64(x, w, bias, act, residual):
    z = x.double() @ w.double().t()
    if bias is not None:
        z = z + bias.double()
    y = act64(act, z)
    return (y if residual is None else y + residual.double()), z


def linear_bounds(x, w, bias, act, residual, y_dtype, x_rounded):
    """(bound of y, bound of pre).  x_rounded: fp32 x enters rounded to bf16.  Each product of exact operands is one
    rounded addition per term of x; all partial sums are at most S = |x| |W|^T + |b|."""
    K = x.shape[1]
    S = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        S = S + bias.double().abs()
    terms = 3 if x.dtype == torch.float32 and not x_rounded else 1
    ez = gamma(terms * K + 32) * S + (2.0 ** -8 * S if x_rounded else 0)
    y, z = linear64(x, w, bias, act, None)
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        eg, eu = ez.chunk(2, 1)
        # silu's slope is below 1.1
        s = g * torch.sigmoid(g)
        ey = 1.1 * eg * (u.abs() + eu) + (s.abs() + 1.1 * eg) * eu + y.abs() * gate_err("silu", g)
    elif act == "none":
        ey = ez
    else:  # GELU's slope is below 1.13
        ey = 1.13 * ez + y.abs() * gate_err(act, z)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2 * U * (y.abs() + residual.double().abs())
    h = HALF[y_dtype]
    return ey * (1 + h) + h * y.abs() + TINY, ez * (1 + h) + h * z.abs() + TINY


def linear_grad64(dy, x, w, act, pre):
    dy, x, w = dy.double(), x.double(), w.double()
    if act == "swiglu":
        g, u = pre.double().chunk(2, 1)
        h = torch.sigmoid(g)
        dz = torch.cat([dy * u * (h + g * h * (1 - h)), dy * g * h], 1)
    elif act == "none":
        dz = dy
    else:
        dz = dy * slope64(act, pre.double())
    return dz @ w, dz.t() @ x, dz.sum(0), dz


def linear_grad_bounds(dy, x, w, act, pre, dx_dtype, dw_dtype):
    """Bounds of dx, dw, db.  dz's own error: the gate's relative error on each of the two parts of the slope.  Then
    dz enters a bf16 result rounded once (2^-8), an fp32 one as three terms; of x's and dz's terms together products
    below 2^-24 (three and three) or 2^-16 (two of x) are left out, counted double for the remainders behind them."""
    T, K = x.shape
    exact = act == "none" and dy.dtype == torch.bfloat16
    dx, dw, db, dz = linear_grad64(dy, x, w, act, pre)
    a = dy.double().abs()
    if act == "swiglu":
        g, u = pre.double().chunk(2, 1)
        h = torch.sigmoid(g)
        ez = torch.cat([a * u.abs() * (h + 2 * g.abs() * h) * (gate_err("silu", g) + 4 * U),
                        a * g.abs() * h * (gate_err("silu", g) + 4 * U)], 1)
    elif act == "none":
        ez = torch.zeros_like(dz)
    else:
        z = pre.double()
        # GELU's second part carries 2 v' = 1.6 (1 + 0.134 z^2) besides z
        lead = z.abs() * (1.6 * (1 + 0.1342 * z * z) if act == "gelu" else 1)
        h = torch.sigmoid(z) if act == "silu" else 0.5 * (1 + torch.tanh(0.79788456 * (z + 0.044715 * z ** 3)))
        ez = a * (h + 2 * lead * h) * (gate_err(act, z) + 8 * U) + a * lead * 4 * U
    R = dz.shape[1]
    xa, wa, za = x.double().abs(), w.double().abs(), dz.abs() + ez

    def one(n, dtype, sums, ezs, x_terms, x_is_f32):
        b = ezs + gamma(6 * n + 64) * sums
        if not exact and dtype == torch.bfloat16:
            b = b + 2.0 ** -8 * sums
        if x_is_f32 and x_terms == 1:
            b = b + 2.0 ** -8 * sums
        elif x_is_f32:
            b = b + 2 * (2.0 ** -16 if x_terms == 2 else 4 * 2.0 ** -24) * sums
        return b

    b_dx = one(R, dx_dtype, za @ wa, ez @ wa, 1, False)
    f = x.dtype == torch.float32
    b_dw = one(T, dw_dtype, za.t() @ xa, ez.t() @ xa, 3 if dw_dtype == torch.float32 else 1 if exact else 2, f)
    b_db = ez.sum(0) + gamma(T + 8) * za.sum(0) + TINY
    hx, hw = HALF[dx_dtype], HALF[dw_dtype]
    return b_dx * (1 + hx) + hx * dx.abs() + TINY, b_dw * (1 + hw) + hw * dw.abs() + TINY, b_db


# ---- balance loss ---------------------------------------------------------------------

def loss64(logits, ids, mask):
    """(loss [2], counts [E + 1], lse [T], takes [T]) from the definition, row by row."""
    T, E = logits.shape
    k = ids.shape[1]
    l = logits.double()
    takes = torch.tensor([bool((mask is None or mask[t]) and not (l[t] == -math.inf).all()) for t in range(T)],
                         dtype=torch.bool)
    n = int(takes.sum())
    counts = torch.zeros(E + 1, dtype=torch.int64)
    counts[E] = n
    lse = torch.full((T,), -math.inf, dtype=torch.float64)
    P = torch.zeros(E, dtype=torch.float64)
    for t in range(T):
        if not takes[t]:
            continue
        for j in range(k):
            if 0 <= int(ids[t, j]) < E:
                counts[int(ids[t, j])] += 1
        lse[t] = torch.logsumexp(l[t], 0)
        P += torch.softmax(l[t], 0)
    if n == 0:
        return torch.zeros(2, dtype=torch.float64), counts, lse, takes
    loss = torch.stack([E / (n * n * k) * (counts[:E].double() * P).sum(), (lse[takes] ** 2).mean()])
    return loss, counts, lse, takes


def route_grad64(logits, ids, w, dw, takes, counts, lse, dloss):
    T, E = logits.shape
    k = ids.shape[1]
    d = torch.zeros((T, E), dtype=torch.float64)
    c = counts[:E].double()
    n = int(counts[E])
    for t in range(T):
        if not takes[t]:
            continue
        if dloss is not None and n:
            p = torch.softmax(logits[t].double(), 0)
            A = float(dloss[0]) * E / (n * n * k)
            d[t] += p * (A * (c - (p * c).sum()) + 2 * float(dloss[1]) / n * lse[t])
        if w is not None:
            wt, g = w[t].double(), dw[t].double()
            s = (wt * g).sum()
            for j in range(k):
                if 0 <= int(ids[t, j]) < E:
                    d[t, int(ids[t, j])] += wt[j] * (g[j] - s)
    return d
