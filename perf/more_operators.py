"""Cases of what becomes of the dense weights beside the experts once their gradient is there: the gradient made
orthogonal (the update that the Muon optimiser applies), the weights' and activations' 8-bit form, and the product of both
in 8-bit integers.

`listed()` names the cases, `draw(rng)` gives more of the same ranges, `prepare(case, seed)` makes one case's inputs on
the GPU, `run(state)` makes one pass (elementary torch operations, or this package's kernels where `own` is true),
`exact(case, seed)` computes the same outputs in 64 bits, and `work(case)` counts the bytes and operations that a pass
cannot do without.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, "i8": 1}
# The odd quintic a s + b s^3 + c s^5 that five Newton-Schulz steps apply to every singular value, momentum and floor
# of the norm: the optimiser's usual values.
STEPS, COEF, BETA, EPS = 5, (3.4445, -4.7750, 2.0315), 0.95, 1e-7
LEAST = 2.0 ** -126  # of a scale: fp32's smallest normal value


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # the gradient of a small router with an odd number of experts
        {"name": "orthogonal small router", "op": "orthogonalize", "B": 1, "R": 60, "K": 544, "g": "f32", "o": "bf16",
         "momentum": False},
        # one layer's 512-expert router, with the optimiser's momentum
        {"name": "orthogonal router", "op": "orthogonalize", "B": 1, "R": 512, "K": 2048, "g": "f32", "o": "bf16",
         "momentum": True},
        # the routers of 48 layers in one call
        {"name": "orthogonal 48 routers", "op": "orthogonalize", "B": 48, "R": 512, "K": 2048, "g": "bf16", "o": "bf16",
         "momentum": True},
        # a tall matrix of odd sizes whose update is wanted in fp32
        {"name": "orthogonal ragged fp32", "op": "orthogonalize", "B": 1, "R": 1001, "K": 777, "g": "f32", "o": "f32",
         "momentum": False},
        # the largest: a wide square block
        {"name": "orthogonal wide block", "op": "orthogonalize", "B": 1, "R": 4096, "K": 4096, "g": "bf16", "o": "bf16",
         "momentum": False},
        # a prompt chunk's activations to 8 bits, the last tokens padding
        {"name": "quantize chunk", "op": "quantize", "T": 8192, "K": 2048, "x": "bf16", "pad": True},
        # a trained matrix of odd height to 8 bits, from its fp32 copy
        {"name": "quantize weights", "op": "quantize", "T": 1001, "K": 4096, "x": "f32", "pad": False},
        # one decoded token through a shared expert's gate and up rows
        {"name": "int8 1 token swiglu", "op": "linear", "T": 1, "K": 2048, "N": 512, "act": "swiglu", "x": "bf16",
         "y": "bf16", "bias": False, "res": "", "pad": False},
        # a verify step of three tokens through its down rows, added to the residual stream
        {"name": "int8 verify down", "op": "linear", "T": 3, "K": 512, "N": 2048, "act": "none", "x": "bf16",
         "y": "f32", "bias": True, "res": "f32", "pad": False},
        # an odd batch with fp32 activations
        {"name": "int8 ragged gelu", "op": "linear", "T": 777, "K": 1056, "N": 1001, "act": "gelu", "x": "f32",
         "y": "f32", "bias": True, "res": "", "pad": True},
        # a prompt chunk through a shared expert's gate and up rows, its 8-bit codes made before (another product
        # takes them too)
        {"name": "int8 chunk swiglu", "op": "linear", "T": 8192, "K": 2048, "N": 512, "act": "swiglu", "x": "i8",
         "y": "bf16", "bias": False, "res": "", "pad": True},
        # a wide dense block with everything in the epilogue
        {"name": "int8 chunk wide silu", "op": "linear", "T": 8192, "K": 4096, "N": 4096, "act": "silu", "x": "bf16",
         "y": "bf16", "bias": True, "res": "bf16", "pad": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v):
    return v | 1 if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["orthogonalize", "orthogonalize", "quantize", "linear", "linear", "linear"])
    if op == "orthogonalize":
        R, K = _odd(rng, _log(rng, 16, 4096)), _odd(rng, _log(rng, 16, 4096))
        B = rng.choice([1, 1, _log(rng, 2, 48)])
        o = rng.choice(["bf16", "bf16", "f32"])
        most = 4096 ** 3 // (3 if o == "f32" else 1)  # (an fp32 result costs several passes of the matrix units)
        while B * min(R, K) ** 2 * max(R, K) > most:
            B, R, K = max(1, B // 2), max(16, R * 3 // 4), max(16, K * 3 // 4)
        return {"op": op, "B": B, "R": R, "K": K, "g": rng.choice(["f32", "bf16"]), "o": o,
                "momentum": rng.random() < 0.6}
    T = max(1, min(8192, _odd(rng, _log(rng, 1, 8192))))
    K = 32 * _log(rng, 1, 256)
    if op == "quantize":
        return {"op": op, "T": T, "K": K, "x": rng.choice(["f32", "bf16"]), "pad": rng.random() < 0.5}
    N = max(1, min(8192, _odd(rng, _log(rng, 16, 8192))))
    act = rng.choice(["none", "gelu", "silu", "swiglu"])
    while T * K * N * (2 if act == "swiglu" else 1) > 8192 * 4096 * 4096:
        T, N = max(1, T * 2 // 3), max(1, N * 2 // 3)
    return {"op": op, "T": T, "K": K, "N": N, "act": act, "x": rng.choice(["f32", "bf16", "bf16", "i8"]),
            "y": rng.choice(["f32", "bf16"]), "bias": rng.random() < 0.5, "res": rng.choice(["", "f32", "bf16"]),
            "pad": rng.random() < 0.3}


def work(c):
    if c["op"] == "orthogonalize":
        m, n, B = min(c["R"], c["K"]), max(c["R"], c["K"]), c["B"]
        # X X^T and its square are symmetric, so half of each is enough
        flops = B * STEPS * (m * m * n + m ** 3 + 2 * m * m * n)
        return {"bytes": B * m * n * (BYTES[c["g"]] + BYTES[c["o"]] + (8 if c["momentum"] else 0)), "flops": flops}
    T, K = c["T"], c["K"]
    if c["op"] == "quantize":
        return {"bytes": T * K * (BYTES[c["x"]] + 1) + 4 * T, "flops": 3 * T * K}
    N = c["N"]
    R = 2 * N if c["act"] == "swiglu" else N
    b = T * K * BYTES[c["x"]] + R * K + R * 4 + T * N * BYTES[c["y"]]
    b += (R * 4 if c["bias"] else 0) + (T * N * BYTES[c["res"]] if c["res"] else 0) + (4 * T if c["x"] == "i8" else 0)
    return {"bytes": b, "flops": 2 * T * R * K}


# ---- inputs -----------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    s = dict(c)
    if c["op"] == "orthogonalize":
        B, R, K = c["B"], c["R"], c["K"]
        r = max(1, min(R, K) // 8)
        # a gradient: a few strong directions over the noise of a batch
        strong = torch.bmm(normal(B, R, r), normal(B, r, K)) / math.sqrt(r)
        s["grad"] = ((strong + 0.3 * normal(B, R, K)) * 1e-3).to(DTYPES[c["g"]])
        s["moment"] = normal(B, R, K, scale=5e-4) if c["momentum"] else None
        return s
    T, K = c["T"], c["K"]
    # activations: some channels far larger than the others
    x = normal(T, K) * torch.exp(0.7 * normal(K))
    if c["op"] == "quantize" and not c["pad"]:  # weights: rows of similar size
        x = normal(T, K, scale=1.0 / math.sqrt(K))
    if c["pad"]:
        x[T - max(1, T // 20):] = 0.0
    if c["op"] == "quantize":
        s["in"] = x.to(DTYPES[c["x"]])
        return s
    N = c["N"]
    R = 2 * N if c["act"] == "swiglu" else N
    s["x_scale"] = None
    if c["x"] == "i8":
        codes, s["x_scale"] = _plain_codes(x)
        s["in"] = codes.to(torch.int8)
    else:
        s["in"] = x.to(DTYPES[c["x"]])
    codes, s["w_scale"] = _plain_codes(normal(R, K, scale=1.0 / math.sqrt(K)))
    s["weight"] = codes.to(torch.int8)
    s["b"] = normal(R) if c["bias"] else None
    s["residual"] = normal(T, N).to(DTYPES[c["res"]]) if c["res"] else None
    return s


# ---- one pass -----------------------------------------------------------------------

def run(s):
    if own:
        return _run_kernels(s)
    return {"orthogonalize": _plain_orthogonalize, "quantize": _plain_quantize, "linear": _plain_linear}[s["op"]](s)


def _run_kernels(s):
    import expert_routed_ffn_amd as moe

    if s["op"] == "orthogonalize":
        o = moe.orthogonalize(s["grad"], momentum=s["moment"], beta=BETA, steps=STEPS, eps=EPS, o_dtype=DTYPES[s["o"]])
        return {"o": o} if s["moment"] is None else {"o": o, "momentum": s["moment"]}
    if s["op"] == "quantize":
        codes, scale = moe.quantize_rows(s["in"])
        return {"values": codes * scale[:, None], "scale": scale}
    return {"y": moe.linear_q8(s["in"], s["weight"], s["w_scale"], x_scale=s["x_scale"], bias=s["b"], act=s["act"],
                               residual=s["residual"], y_dtype=DTYPES[s["y"]])}


def _plain_orthogonalize(s):
    x = s["grad"].float()
    if s["moment"] is not None:
        s["moment"].mul_(BETA).add_(x, alpha=1.0 - BETA)
        x = BETA * s["moment"] + (1.0 - BETA) * x
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
    tall = s["R"] > s["K"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEF
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    o = (x.transpose(1, 2) if tall else x).to(DTYPES[s["o"]]).contiguous()
    return {"o": o} if s["moment"] is None else {"o": o, "momentum": s["moment"]}


def _plain_codes(x):
    """Codes (as fp32) and scales of the rows; both quotients in 64 bits, as values may lie next to a border."""
    x = x.float()
    scale = (x.abs().amax(1).double() / 127.0).float().clamp(min=LEAST)
    return torch.round(x.double() / scale.double()[:, None]).float(), scale


def _plain_quantize(s):
    codes, scale = _plain_codes(s["in"])
    return {"values": codes * scale[:, None], "scale": scale}


def _plain_sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _plain_linear(s):
    codes, scale = (s["in"].float(), s["x_scale"]) if s["x"] == "i8" else _plain_codes(s["in"])
    z = torch.mm(codes, s["weight"].float().t()) * scale[:, None] * s["w_scale"]
    if s["b"] is not None:
        z = z + s["b"]
    N = s["N"]
    if s["act"] == "none":
        y = z
    elif s["act"] == "gelu":
        y = z * _plain_sigmoid(1.5957691216057308 * (z + 0.044715 * z * z * z))
    elif s["act"] == "silu":
        y = z * _plain_sigmoid(z)
    else:
        y = z[:, :N] * _plain_sigmoid(z[:, :N]) * z[:, N:]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(DTYPES[s["y"]])}


# ---- the same in 64 bits --------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    f = torch.float64
    if c["op"] == "orthogonalize":
        g, out = s["grad"].to(f), {}
        if s["moment"] is not None:
            out["momentum"] = BETA * s["moment"].to(f) + (1 - BETA) * g
            g = (1 - BETA) * g + BETA * out["momentum"]
        g = g / (torch.linalg.matrix_norm(g)[:, None, None] + EPS)
        # The steps' polynomials are all polynomials of the first Gram matrix and commute: their product is gathered
        # on the shorter side, and the matrix is multiplied once.
        wide = c["R"] <= c["K"]
        gram = torch.matmul(g, g.mT) if wide else torch.matmul(g.mT, g)
        eye = torch.eye(min(c["R"], c["K"]), dtype=f, device="cuda").expand_as(gram)
        total = eye
        for _ in range(STEPS):
            p = COEF[0] * eye + torch.matmul(gram, COEF[1] * eye + COEF[2] * gram)
            total, gram = torch.matmul(total, p), torch.matmul(p, torch.matmul(gram, p))
        out["o"] = torch.matmul(total, g) if wide else torch.matmul(g, total)
        return out
    if c["op"] == "quantize":
        codes, scale = _codes64(s["in"])
        return {"values": codes * scale, "scale": scale[:, 0]}
    codes, scale = (s["in"].to(f), s["x_scale"].to(f)[:, None]) if c["x"] == "i8" else _codes64(s["in"])
    z = torch.matmul(codes, s["weight"].to(f).t().contiguous()) * (scale * s["w_scale"].to(f))
    z = z if s["b"] is None else z + s["b"].to(f)
    if c["act"] == "gelu":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    elif c["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif c["act"] == "swiglu":
        gate, up = z.chunk(2, 1)
        z = gate * torch.sigmoid(gate) * up
    return {"y": z if s["residual"] is None else z + s["residual"].to(f)}


def _codes64(x):
    # a row's scale is itself an fp32 value: the one nearest to a 127th of the largest magnitude
    x = x.to(torch.float64)
    scale = torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True) / 127
    scale = scale.to(torch.float32).to(torch.float64).clamp(min=LEAST)
    return torch.round(x / scale), scale
