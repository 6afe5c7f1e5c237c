"""GPU: the orthogonalised update's gradient and moment on both ways, the moment against 64 bits value by value and the
result against what the new moment and the gradient give in 64 bits."""
import pytest
import torch

from tests._newton_ref import newton64, newton_bound
from tests._train_ref import HALF, U

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _near(got, u, o_dtype):
    """An fp32 result within newton_bound; a bf16 one within the documented 2e-3 of its norm and its rounding (at most half
    a step of each value, and at most what the reference's own rounding is and 2e-3 again)."""
    ref = newton64(u)
    off, n = (got.double().cpu() - ref).norm(), ref.norm()
    if o_dtype == F32:
        most = newton_bound(u, F32) * (1 + HALF[F32]) + HALF[F32] * n
    else:
        most = 2 * 2e-3 * n + (ref.to(BF16).double() - ref).norm()
    assert off <= most, (float(off / n), float(most / n))


def _gradients(B, R, K, seed):
    """Three strong directions over noise."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, R, 3), generator=g) @ torch.randn((B, 3, K), generator=g) + 0.1 * torch.randn((B, R, K), generator=g)


# Both sides above 64, and numbers of values that are neither whole blocks of 2,048 nor multiples of 4
SIZES = [(81, 67), (131, 97), (67, 131), (65, 65), (69, 1001)]


def _check_momentum(moe, B, R, K, gt, o_dtype, nesterov):
    beta = 0.9
    gr, m = _gradients(B, R, K, R + K).to(gt), 0.5 * _gradients(B, R, K, R * K)
    # neighbours of the moment's memory, which stay as they are
    held = torch.full((B * R * K + 64,), 7.0, device="cuda")
    moment = held[32:-32].view(B, R, K)
    moment.copy_(m)
    o = moe.orthogonalize(gr.cuda(), momentum=moment, beta=beta, nesterov=nesterov, o_dtype=o_dtype)
    new = moment.cpu().double()
    want = beta * m.double() + (1 - beta) * gr.double()
    # beta and 1 - beta are rounded to fp32, then one product and one fused sum
    assert ((new - want).abs() <= 3 * U * (beta * m.double().abs() + (1 - beta) * gr.double().abs())).all()
    assert (held[:32] == 7).all() and (held[-32:] == 7).all()
    u = beta * new + (1 - beta) * gr.double() if nesterov else new
    for b in {0, B - 1}:
        _near(o[b], u[b], o_dtype)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("R,K", SIZES)
def test_momentum_above_a_short_side_of_64(moe, R, K, gt, nesterov):
    for B in (1, 3):
        for o_dtype in (BF16, F32):
            _check_momentum(moe, B, R, K, gt, o_dtype, nesterov)


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("R,K", SIZES)
def test_gradients_above_a_short_side_of_64(moe, R, K, gt):
    u = _gradients(1, R, K, 3)[0].to(gt)
    for o_dtype in (BF16, F32):
        _near(moe.orthogonalize(u.cuda(), o_dtype=o_dtype), u.float(), o_dtype)


# A short side up to 64 and a long one whose stretches of 64 are more than the 32 workgroups that share a Gram matrix, so that
# a workgroup brings several: 33 stretches (the last of one column) are 16 workgroups of two and one of one, 65 are 21 of three
# and one of two, 66 are 22 of three, 256 are 32 of eight
LONG = [(60, 2049), (2049, 60), (33, 4100), (4161, 17), (64, 16384), (16384, 1), (48, 6145)]


@pytest.mark.parametrize("R,K", LONG)
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_long_sides_beside_short_ones(moe, R, K, o_dtype):
    u = _gradients(2, R, K, R + K)
    o = moe.orthogonalize(u.cuda(), o_dtype=o_dtype)
    for b in range(2):
        _near(o[b], u[b], o_dtype)


@pytest.mark.parametrize("R,K", LONG)
@pytest.mark.parametrize("gt,o_dtype,nesterov", [(F32, BF16, True), (BF16, F32, False)])
def test_momentum_of_long_sides_beside_short_ones(moe, R, K, gt, o_dtype, nesterov):
    _check_momentum(moe, 3, R, K, gt, o_dtype, nesterov)
