"""GPU: how exact a bf16 orthogonalised update is where its fewer bits could show.

The rule of these tests: with o' the result before its rounding and |o' - ref| <= d |ref|, the way from a value to the nearest
bf16 changes by no more than the value does, so a bf16 result is off by at most 2 d |ref| + |bf16(ref) - ref|.  d is what is
documented for the kind of matrix."""
import pytest
import torch

from tests._newton_ref import coefs, newton64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rounded(o, ref, d, what=""):
    """The rule above; o and ref on the same device."""
    off, n = float((o.double() - ref).norm()), float(ref.norm())
    most = 2 * d * n + float((ref.to(BF16).double() - ref).norm())
    assert off <= most, f"{what}: off {off / n:.2e} of its norm, allowed {most / n:.2e}"


# One step of a large a among others: A's smallest values, and any noise beside them, grow by a^2 in it.
BY_STEP = [[(19.0, -15.9, 0.0), (3.9, -0.4, 0.01), (1.5, -0.1, 0.0)],
           [(2.136, -1.435, 0.318), (2.728, -0.947, 0.028), (15.119, -5.444, 0.192), (3.219, -3.441, 0.659), (1.616, -0.792, 0.285)],
           [(1.32, -0.136, 0.013), (2.313, -1.821, 0.416), (2.436, -1.962, 0.793), (14.339, -13.85, 2.38), (3.256, -2.761, 1.183),
            (1.61, -0.963, 0.019)]]


@pytest.mark.parametrize("R,K", [(24, 24), (33, 36), (64, 64), (64, 700), (700, 40)])
@pytest.mark.parametrize("coef", BY_STEP)
def test_steps_of_large_growth_on_a_short_side(moe, R, K, coef):
    g = _gen(R + K)
    u = torch.randn((8, R, 1), generator=g) @ torch.randn((8, 1, K), generator=g) + 1e-3 * torch.randn((8, R, K), generator=g)
    for x in u:  # singular values stay in the documented range
        s = torch.linalg.svdvals(x.double() / x.double().norm())
        for a, b, c in coefs(coef, len(coef)):
            assert (b * s ** 2 + c * s ** 4).abs().max() < 16
            s = (a * s + b * s ** 3 + c * s ** 5).abs()
            assert s.max() < 4
    o = moe.orthogonalize(u.cuda(), coef=coef, steps=len(coef)).cpu()
    for b in range(8):
        _rounded(o[b], newton64(u[b], steps=len(coef), coef=coef), 2e-3, f"matrix {b}")
