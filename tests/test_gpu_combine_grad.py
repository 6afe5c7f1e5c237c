"""GPU: the combine's gradient against its definition in 64 bits.

dw is a sum of H products of fp32 values: |error| <= gamma(H + 8) sum |dout y|.  dy is one product: half a step of its
type, after half a step of fp32."""
import pytest
import torch

from tests._train_ref import HALF, TINY, U, gamma, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _inputs(T, k, H, yt, gt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, k, H), generator=g).to(yt), torch.softmax(torch.randn((T, k), generator=g), 1),
            torch.randn((T, H), generator=g).to(gt))


def _check(y, w, dout, dw, dy):
    yd, gd = y.double(), dout.double()[:, None, :]
    if dw is not None:
        within(dw, (yd * gd).sum(2), gamma(y.shape[2] + 8) * (yd * gd).abs().sum(2) + TINY, "dw")
    if dy is not None:
        ref = w.double()[:, :, None] * gd
        within(dy, ref, (HALF[y.dtype] + 2 * U) * ref.abs() + TINY, "dy")


@pytest.mark.parametrize("T,k,H", [(1, 1, 4), (2, 16, 32), (5, 3, 36), (12, 10, 2048), (33, 9, 2052), (70, 8, 96),
                                   (300, 2, 4096), (3, 16, 16384)])
@pytest.mark.parametrize("yt,gt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_combine_backward(moe, T, k, H, yt, gt):
    y, w, dout = _inputs(T, k, H, yt, gt, seed=T + k + H)
    dw, dy = moe.combine_backward(y.cuda(), w.cuda(), dout.cuda())
    assert dw.dtype == F32 and dy.dtype == yt
    _check(y, w, dout, dw, dy)


def test_parts_equal_the_whole(moe):
    y, w, dout = (t.cuda() for t in _inputs(40, 10, 520, BF16, F32, seed=1))
    dw, dy = moe.combine_backward(y, w, dout)
    only_w = moe.combine_backward(y, w, dout, need=("dw",))
    only_y = moe.combine_backward(y, w, dout, need=("dy",))
    assert only_w[1] is None and only_y[0] is None
    assert torch.equal(only_w[0], dw) and torch.equal(only_y[1], dy)
    # a token's result does not depend on its neighbours
    some = moe.combine_backward(y[7:9], w[7:9], dout[7:9])
    assert torch.equal(some[0], dw[7:9]) and torch.equal(some[1], dy[7:9])


def test_no_rows_and_nothing_past_the_end(moe):
    y, w, dout = (t.cuda() for t in _inputs(6, 3, 64, F32, F32, seed=2))
    dw, dy = moe.combine_backward(y[:0], w[:0], dout[:0])
    assert dw.shape == (0, 3) and dy.shape == (0, 3, 64)
    dw, dy = torch.full((8, 3), 5.0, device="cuda"), torch.full((8, 3, 64), 5.0, device="cuda")
    moe.combine_backward(y, w, dout, dw=dw[1:7], dy=dy[1:7])
    torch.cuda.synchronize()
    for t in (dw, dy):
        assert (t[0] == 5).all() and (t[7] == 5).all()
    _check(y.cpu(), w.cpu(), dout.cpu(), dw[1:7], dy[1:7])


def test_differences(moe):
    """The gradient against central differences of the combine itself (linear in w and y, so differences are exact up
    to the rounding of its fp32 sums)."""
    y, w, dout = _inputs(4, 3, 64, F32, F32, seed=3)
    dw, dy = moe.combine_backward(y.cuda(), w.cuda(), dout.cuda())

    def loss(y, w):
        return float((moe.combine(y.cuda().contiguous(), w.cuda().contiguous()).cpu().double() * dout.double()).sum())

    mag = float(((w[:, :, None] * y).abs().sum(1).double() * dout.double().abs()).sum())
    g = torch.Generator().manual_seed(4)
    for _ in range(3):
        vy, vw, eps = torch.randn(y.shape, generator=g), torch.randn(w.shape, generator=g), 0.25
        num = (loss(y + eps * vy, w) - loss(y - eps * vy, w)) / (2 * eps)
        assert abs(num - float((dy.cpu().double() * vy.double()).sum())) <= 64 * U * (mag + 1) / eps * 4
        num = (loss(y, w + eps * vw) - loss(y, w - eps * vw)) / (2 * eps)
        assert abs(num - float((dw.cpu().double() * vw.double()).sum())) <= 64 * U * (mag + 1) / eps * 16


def test_most_tokens(moe):
    """T * k = 2^24 with k = 1: as many tokens as a call takes.  Small whole numbers: every product and sum is exact."""
    T, H = 1 << 24, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    y = torch.randint(-3, 4, (T, 1, H), generator=g, device="cuda").to(BF16)
    w = torch.randint(-3, 4, (T, 1), generator=g, device="cuda").float()
    dout = torch.randint(-3, 4, (T, H), generator=g, device="cuda").to(BF16)
    dw, dy = moe.combine_backward(y, w, dout)
    assert torch.equal(dw[:, 0], (y[:, 0].float() * dout.float()).sum(1))
    assert torch.equal(dy[:, 0].float(), w * dout.float())


@pytest.mark.parametrize("T,k,H", [(3, 2, 64), (300, 9, 96), (300, 4, 36)])
@pytest.mark.parametrize("yt,gt", [(F32, BF16), (BF16, F32)])
def test_what_an_output_does_not_need_may_be_null(moe, T, k, H, yt, gt):
    """Through the C interface: dw alone without w, dy alone without y."""
    import ctypes

    from expert_routed_ffn_amd import _lib

    y, w, dout = (t.cuda() for t in _inputs(T, k, H, yt, gt, seed=T + H))
    want = moe.combine_backward(y, w, dout)
    dw, dy = torch.empty_like(w), torch.empty_like(y)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for a_y, a_w, a_dw, a_dy in [(y.data_ptr(), None, dw.data_ptr(), None), (None, w.data_ptr(), None, dy.data_ptr())]:
        assert int(_lib.lib.moe_combine_backward(a_y, _lib._dtype_code(y), a_w, dout.data_ptr(), _lib._dtype_code(dout), T, k, H,
                                                 a_dw, a_dy, stream)) == _lib.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(dw, want[0]) and torch.equal(dy, want[1])
