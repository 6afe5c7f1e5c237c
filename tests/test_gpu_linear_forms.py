"""GPU: the dense product and its gradient in each form that their plan has: tile shape, reduction whole or cut, fp32
activations split at the fragments or as planes.  Each test asserts the form that it is there for, so that other rates in
the plan cannot leave a form untested without a word.  All sizes are ragged: last steps of fewer than 64 k, columns off the
tiles (and odd, where a row may be), rows past the last tile.

Operands are whole numbers whose products and sums fp32 holds exactly (the magnitudes under every sum stay below 2^24), or
one operand has a single +-1 in each reduction and the other is any fp32 value, which must come back bit for bit: that takes
all three of its bf16 terms.  Results are then compared for equality; bf16 ones with the exact value rounded once.
"""
import pytest
import torch

from tests._train_ref import HALF, U, gate_err, rows_of, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _whole(shape, most, g, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def _equal(got, exact, what):
    assert exact.abs().max() < 1 << 24, what
    assert torch.equal(got, exact.float().to(got.dtype)), what


def _ones(rows, cols, g, dtype):
    """[rows, cols] of zeros with one +-1 in each column; the row of each and its sign."""
    at = torch.randint(0, rows, (cols,), generator=g, device="cuda")
    at[0], at[-1] = rows - 1, rows - 1  # the end of the reduction among them
    sign = 2.0 * torch.randint(0, 2, (cols,), generator=g, device="cuda") - 1
    m = torch.zeros((rows, cols), device="cuda")
    m[at, torch.arange(cols, device="cuda")] = sign
    return m.to(dtype), at, sign


# x and y types, the form's tile, whether its reduction is cut, launches from planes
FORWARD = [
    (100, 96, 33, "none", BF16, BF16, 64, False, 0), (100, 2080, 33, "none", BF16, BF16, 64, True, 0),
    (2050, 96, 1003, "none", BF16, BF16, 128, False, 0), (1025, 8224, 201, "none", BF16, F32, 128, True, 0),
    (2050, 1056, 4094, "none", BF16, F32, 256, False, 0), (1025, 16352, 1003, "none", BF16, BF16, 256, True, 0),
    (100, 2080, 33, "swiglu", BF16, F32, 64, True, 0), (65, 8224, 515, "swiglu", BF16, BF16, 128, True, 0),
    (1025, 1056, 4094, "swiglu", BF16, BF16, 256, False, 0), (1025, 8224, 1003, "swiglu", BF16, BF16, 256, True, 0),
    (100, 96, 33, "none", F32, F32, 64, False, 0), (100, 1056, 33, "none", F32, F32, 64, True, 0),
    (4001, 96, 2047, "none", F32, F32, 128, False, 1), (1025, 1056, 2047, "none", F32, F32, 128, True, 1),
    (4001, 544, 4094, "none", F32, F32, 256, False, 1), (1025, 8224, 1003, "none", F32, F32, 256, True, 1),
    (1025, 1056, 1003, "swiglu", F32, F32, 128, True, 1), (4001, 544, 2047, "swiglu", F32, F32, 256, False, 1),
    (1025, 4128, 1003, "swiglu", F32, F32, 256, True, 1),
    (100, 96, 33, "none", F32, BF16, 64, False, 0), (100, 2080, 33, "none", F32, BF16, 64, True, 0),
    (4001, 96, 4094, "none", F32, BF16, 128, False, 2), (4001, 8224, 2047, "none", F32, BF16, 256, True, 2),
    (4001, 96, 2047, "swiglu", F32, BF16, 128, False, 2), (4001, 544, 4094, "swiglu", F32, BF16, 256, False, 2),
    (4001, 4128, 2047, "swiglu", F32, BF16, 256, True, 2)]


@pytest.mark.parametrize("T,K,N,act,xt,yt,tile,cut,planes", FORWARD)
def test_forward(moe, T, K, N, act, xt, yt, tile, cut, planes):
    form = moe.linear_form(T, K, N, act, xt, yt)
    assert (form["tile"], form["parts"] > 1, form["planes"]) == (tile, cut, planes)
    assert form["terms"] == (1 if xt == BF16 else 3 if yt == F32 else 2)
    g, R = _gen(T + K + N), rows_of(act, N)
    most = 1000 if xt == F32 else 127  # times 16,352 at most: below 2^24
    x, w = _whole((T, K), most, g, xt), _whole((R, K), 1, g, BF16)
    bias, res = _whole((R,), 999, g, F32), _whole((T, N), 100, g, yt)
    pre = torch.empty((T, R), dtype=yt, device="cuda")
    y = moe.linear(x, w, bias=bias, act=act, residual=res, y_dtype=yt, pre=pre)
    again = res.clone()
    moe.linear(x, w, bias=bias, act=act, residual=again, y=again)  # in place
    assert torch.equal(again, y)
    z = x.double() @ w.double().t() + bias.double()
    _equal(pre, z, "pre")
    if act == "none":
        _equal(y, z + res.double(), "y")
    else:
        a, u = z.chunk(2, 1)
        v = a * torch.sigmoid(a) * u
        # the sigmoid's error; sigmoids below the normal range become 0; the sum with the residual and y's rounding
        e = v.abs() * gate_err("silu", a) + (a * u).abs() * 2.0 ** -126 + 2 * U * (v.abs() + res.double().abs())
        v = v + res.double()
        within(y, v, (e * (1 + HALF[yt]) + HALF[yt] * v.abs()).cpu(), "y")


@pytest.mark.parametrize("T,K,N,act,xt,yt,tile,cut,planes", [c for c in FORWARD if c[4:6] == (F32, F32)])
def test_forward_holds_all_of_fp32(moe, T, K, N, act, xt, yt, tile, cut, planes):
    g, R = _gen(T + K + N + 1), rows_of(act, N)
    x = torch.randn((T, K), generator=g, device="cuda")
    wt, at, sign = _ones(K, R, g, BF16)
    pre = torch.empty((T, R), device="cuda")
    y = moe.linear(x, wt.t().contiguous(), act=act, pre=pre)
    assert torch.equal(pre, x[:, at] * sign)
    if act == "none":
        assert torch.equal(y, pre)


# dy, x, dx and dw types, the form's tile, whether dw's and dx's reductions are cut
BACKWARD = [
    (100, 96, 33, "BBBB", 64, False, False), (2050, 96, 33, "BBBB", 64, True, False), (100, 96, 2047, "BBBB", 64, False, True),
    (300, 8224, 201, "BBBB", 128, False, False), (4001, 2080, 33, "BBBB", 128, True, False),
    (300, 1056, 2047, "BBBB", 128, False, True), (2050, 8224, 1003, "BBBB", 256, False, False),
    (8193, 2080, 2047, "BBBB", 256, True, False),
    (515, 96, 2047, "BFBB", 64, True, True), (4001, 96, 2047, "BFBB", 128, True, True),
    (515, 8224, 2047, "BFBB", 256, False, False), (4001, 4128, 1003, "BFBB", 256, True, False),
    (300, 96, 1003, "FBBF", 64, True, True), (300, 8224, 515, "FBBF", 128, False, False),
    (1025, 8224, 33, "FBBF", 128, True, False), (1025, 8224, 1003, "FBBF", 256, False, False),
    (1025, 4128, 4094, "FBBF", 256, False, True), (4001, 1056, 4094, "FBBF", 256, True, True),
    (65, 96, 33, "FFFF", 64, False, False), (300, 96, 201, "FFFF", 64, True, True),
    (65, 8224, 201, "FFFF", 128, False, False), (1025, 544, 2047, "FFFF", 128, True, True),
    (515, 8224, 2047, "FFFF", 256, False, False), (515, 4128, 4094, "FFFF", 256, False, True),
    (4001, 8224, 201, "FFFF", 256, True, False), (2050, 2080, 2047, "FFFF", 256, True, True)]


def _types(code):
    return [F32 if c == "F" else BF16 for c in code]


@pytest.mark.parametrize("T,K,N,types,tile,dw_cut,dx_cut", BACKWARD)
def test_backward(moe, T, K, N, types, tile, dw_cut, dx_cut):
    gt, xt, dxt, dwt = _types(types)
    form = moe.linear_backward_form(T, K, N, "none", gt, xt, dxt, dwt)
    assert (form["tile"], form["dw_parts"] > 1, form["dx_parts"] > 1) == (tile, dw_cut, dx_cut)
    g = _gen(T + K + N)
    runs = [(1000 if gt == F32 else 2, 1)] + ([(1, 1000)] if xt == F32 else [])
    for dy_most, x_most in runs:  # 1,000 * 8,193 and 2 * 1,000 * 4,094 stay below 2^24
        dy, x, w = _whole((T, N), dy_most, g, gt), _whole((T, K), x_most, g, xt), _whole((N, K), 2, g, BF16)
        dx, dw, db = moe.linear_backward(dy, x, w, dx_dtype=dxt, dw_dtype=dwt)
        _equal(dx, dy.double() @ w.double(), "dx")
        _equal(dw, dy.double().t() @ x.double(), "dw")
        _equal(db, dy.double().sum(0), "db")


@pytest.mark.parametrize("T,K,N,types,tile,dw_cut,dx_cut", [c for c in BACKWARD if c[3] in ("FBBF", "FFFF")])
def test_backward_holds_all_of_fp32(moe, T, K, N, types, tile, dw_cut, dx_cut):
    gt, xt, dxt, dwt = _types(types)
    g = _gen(T + K + N + 1)
    dy = torch.randn((T, N), generator=g, device="cuda")
    w, r_of, w_sign = _ones(N, K, g, BF16)
    x, t_of, x_sign = _ones(T, K, g, xt)
    dx, dw, _ = moe.linear_backward(dy, x, w, dx_dtype=dxt, dw_dtype=dwt)
    # (a bf16 dx takes two terms, which round to the value's own bf16 but for ties; those are left to the test above)
    if dxt == F32:
        assert torch.equal(dx, dy[:, r_of] * w_sign)
    assert torch.equal(dw, dy[t_of].t() * x_sign)
    if xt == F32:
        x = torch.randn((T, K), generator=g, device="cuda")
        dy, t_of, sign = _ones(T, N, g, F32)
        _, dw, _ = moe.linear_backward(dy, x, w, need=("dw",), dw_dtype=dwt)
        assert torch.equal(dw, x[t_of] * sign[:, None])


def test_largest_rows_and_columns(moe):
    """K and N at their largest, SwiGLU's 32,768 rows of w among them: no row, column or piece is left out or taken twice."""
    K = N = 16384
    g = _gen(5)
    for T in (64, 66):
        x = torch.randn((T, K), generator=g, device="cuda")
        wt, at, sign = _ones(K, 2 * N, g, BF16)
        pre = torch.empty((T, 2 * N), device="cuda")
        moe.linear(x, wt.t().contiguous(), act="swiglu", pre=pre)
        assert torch.equal(pre, x[:, at] * sign)
        dy = torch.randn((T, N), generator=g, device="cuda")
        w, r_of, w_sign = _ones(N, K, g, BF16)
        ones, t_of, x_sign = _ones(T, K, g, F32)
        dx, dw, db = moe.linear_backward(dy, ones, w, dx_dtype=F32)
        assert torch.equal(dx, dy[:, r_of] * w_sign)
        assert torch.equal(dw, dy[t_of].t() * x_sign)
        bound = (T + 8) * U * dy.double().abs().sum(0)
        within(db, dy.double().sum(0), bound.cpu(), "db")
