"""GPU: what the dense product and its gradient round, and what they do not.

The exact tests use whole numbers whose products and sums fp32 holds exactly (below 2^24), with operands of 12 bits that one
bf16 does not hold: a bf16 result is then the exact sum rounded once, to the nearest and ties to even, bit for bit.  An
operand that was rounded to bf16 on the way would show in most elements.
"""
import pytest
import torch

from tests._train_ref import linear_grad64, linear_grad_bounds, rows_of, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _whole(shape, most, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def _rounded(exact):
    """A float64 tensor of values that fp32 holds, rounded once to bf16."""
    assert exact.abs().max() < 1 << 24
    return exact.float().to(BF16)


# more than 2^14 values of dz, fewer and more tokens than a part of the reduction, odd columns, each tile shape
@pytest.mark.parametrize("T,K,N", [(300, 96, 200), (1000, 64, 33), (4000, 512, 520), (3000, 2048, 1001), (1, 64, 8000)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_bf16_gradients_of_fp32_dy_are_rounded_once(moe, T, K, N, xt):
    dy = _whole((T, N), 2047, T + N, F32)
    x, w = _whole((T, K), 1, K, xt), _whole((N, K), 2, N, BF16)
    dx, dw, db = moe.linear_backward(dy, x, w, dx_dtype=BF16, dw_dtype=BF16)
    rx, rw, rb, _ = linear_grad64(dy, x, w, "none", None)
    assert torch.equal(dx, _rounded(rx))
    assert torch.equal(dw, _rounded(rw))
    assert torch.equal(db.double(), rb)


# the same behind an activation, where dz is no whole number.  The bounds of the fp32 results carry dz's own error and that
# of the sums; beside those a result is off by half a step of bf16 and by what two terms leave of dz, 2^-17 of it.
@pytest.mark.parametrize("T,K,N,act,gt", [(400, 96, 65, "swiglu", BF16), (300, 224, 201, "gelu", F32),
                                          (500, 64, 300, "silu", BF16)])
def test_bf16_gradients_behind_an_activation_are_rounded_once(moe, T, K, N, act, gt):
    g = torch.Generator().manual_seed(T + K)
    R = rows_of(act, N)
    x, dy = torch.randn((T, K), generator=g).to(BF16), torch.randn((T, N), generator=g).to(gt)
    w = (torch.randn((R, K), generator=g) / K ** 0.5).to(BF16)
    pre = torch.randn((T, R), generator=g).to(gt)
    dx, dw, _ = moe.linear_backward(dy.cuda(), x.cuda(), w.cuda(), act=act, pre=pre.cuda(), dx_dtype=BF16, dw_dtype=BF16)
    rx, rw, _, dz = linear_grad64(dy, x, w, act, pre)
    bx, bw, _ = linear_grad_bounds(dy, x, w, act, pre, F32, F32)
    za = dz.abs()
    within(dx, rx, bx + 2.0 ** -8 * (rx.abs() + bx) + 2.0 ** -17 * (za @ w.double().abs()), "dx")
    within(dw, rw, bw + 2.0 ** -8 * (rw.abs() + bw) + 2.0 ** -17 * (za.t() @ x.double().abs()), "dw")


# dy in bf16 without an activation is dz as it stands, and fp32 x is what would be rounded
@pytest.mark.parametrize("T,K,N", [(1, 64, 40), (3, 96, 8), (6, 2048, 512), (300, 96, 200), (4000, 512, 520), (2000, 1024, 33)])
def test_bf16_weight_gradient_takes_fp32_activations_unrounded(moe, T, K, N):
    dy, x, w = _whole((T, N), 2, N, BF16), _whole((T, K), 2047, K, F32), _whole((N, K), 1, T, BF16)
    dx, dw, db = moe.linear_backward(dy, x, w, dx_dtype=BF16, dw_dtype=BF16)
    rx, rw, rb, _ = linear_grad64(dy, x, w, "none", None)
    assert torch.equal(dw, _rounded(rw))
    assert torch.equal(dx, _rounded(rx)) and torch.equal(db.double(), rb)


# fewest tokens that take tiles, reductions cut into parts, rows past the last tile, an odd number of tokens above and below
# a tile's half, columns off the tile, the largest
@pytest.mark.parametrize("T,K,N", [(64, 96, 33), (65, 96, 33), (65, 4096, 512), (301, 544, 515), (2000, 64, 9), (1001, 4096, 1024),
                                   (4001, 2080, 2047), (8192, 4096, 4096)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_bf16_product_of_fp32_activations_is_rounded_once(moe, T, K, N, act):
    if act == "swiglu" and T == 8192:
        N = 1024
    R = rows_of(act, N)
    x, w = _whole((T, K), 2047, T, F32), _whole((R, K), 1, N, BF16)
    bias, res = _whole((R,), 1000, K, F32), _whole((T, N), 100, K + 1, BF16)
    pre = torch.empty((T, R), dtype=BF16, device="cuda")
    y = moe.linear(x, w, bias=bias, act=act, residual=res, y_dtype=BF16, pre=pre)
    z = x.double() @ w.double().t() + bias.double()
    assert torch.equal(pre, _rounded(z))
    if act == "none":
        assert torch.equal(y, _rounded(z + res.double()))


def test_a_token_keeps_its_value_in_a_larger_batch(moe):
    x, w = _whole((200, 256), 2047, 1, F32), _whole((70, 256), 2, 2, BF16)
    few, many = moe.linear(x[:64], w, y_dtype=BF16), moe.linear(x, w, y_dtype=BF16)
    assert torch.equal(few, many[:64])


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slopes_far_out(moe, act, gt):
    """The activation's slope is 1 far above zero and 0 far below it, up to the type's largest value: dz is dy or zero there,
    and the products with the unit matrix give it back."""
    far = torch.tensor([1e3, 1e6, 1e12, 4e19, 6e19, 1e25, 1e37, torch.finfo(gt).max], dtype=torch.float64)
    pre = torch.cat([far, -far]).repeat(70, 2).to(gt).cuda()
    dy = _whole((70, 32), 9, 3, gt)
    eye = torch.eye(32, dtype=BF16, device="cuda")
    x = _whole((70, 32), 2, 4, BF16)
    dx, dw, db = moe.linear_backward(dy, x, eye, act=act, pre=pre, dx_dtype=F32)
    dz = torch.where(pre > 0, dy, torch.zeros_like(dy)).double()
    assert torch.equal(dx.double(), dz)
    assert torch.equal(dw.double(), dz.t() @ x.double())
    assert torch.equal(db.double(), dz.sum(0))


def test_swiglu_slope_of_a_closed_gate_is_zero(moe):
    """Where the gate's slope is 0 its dz is 0, however large dy times the up value (here past fp32's range)."""
    T, N = 70, 32
    pre = torch.cat([torch.full((T, N), -300.0), torch.full((T, N), 1e30)], 1).cuda()
    dy = torch.full((T, N), 1e30, device="cuda")
    x, w = _whole((T, 64), 2, 1, BF16), _whole((2 * N, 64), 2, 2, BF16)
    dx, dw, db = moe.linear_backward(dy, x, w, act="swiglu", pre=pre, dx_dtype=F32)
    assert not dx.any() and not dw.any() and not db.any()
