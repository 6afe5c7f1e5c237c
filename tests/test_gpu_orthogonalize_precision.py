"""GPU: how exact a bf16 orthogonalised update is where its fewer bits could show.

The rule of these tests: o' is the result before its rounding and |o' - ref| <= d |ref|, with the d that is documented for the
kind of matrix.  The rounding moves each value by at most half a step of the result's last place, so |o - ref| is at most
d |ref| + |half steps|; and the way from a value to the nearest bf16 changes by no more than the value does, so it is at most
2 d |ref| + |bf16(ref) - ref|, too."""
import pytest
import torch

from tests._newton_ref import coefs, newton64, newton_bound
from tests._train_ref import HALF
from tests.test_gpu_orthogonalize import FORMS, _check_spread

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
    """The rules above; o and ref on the same device."""
    off, n = float((o.double() - ref).norm()), float(ref.norm())
    half = torch.where(o == 0, 0.0, torch.ldexp(torch.ones_like(ref), torch.frexp(o.double())[1] - 9))
    most = min(2 * d * n + float((ref.to(BF16).double() - ref).norm()), d * n + float(half.norm()))
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


# Norms of the rows that are not 0, of norm 1 together: the first two kinds are those where A's diagonal in 11 bits did most.
ROWS = [(0.48889417, 0.61683972, 0.61683972), (0.50231472, 0.50231472, 0.50231472, 0.49299061), (1.0,), (0.25,) * 16]


@pytest.mark.parametrize("R,K", [(100, 700), (700, 100), (512, 2048)])
@pytest.mark.parametrize("norms", ROWS)
def test_gradients_of_few_rows(moe, R, K, norms):
    """A router whose tokens went to few experts: its other rows are 0.  Where rows have nothing in common A is diagonal, holding
    their squared norms, and a rounding of these to 11 bits grows to 7e-3 on the way: of 0.61684, 0.8112 instead of 0.8054
    would come, of 0.50231 0.7587 instead of 0.7534."""
    g = _gen(R)
    m, n = min(R, K), max(R, K)
    u = torch.zeros((8, m, n), dtype=torch.float64)
    for x in u:
        rows = torch.linalg.qr(torch.randn((n, len(norms)), generator=g, dtype=torch.float64))[0].t()
        x[torch.randperm(m, generator=g)[:len(norms)]] = rows * torch.tensor(norms).double()[:, None]
    u = (u if R <= K else u.mT).float().contiguous()
    o = moe.orthogonalize(u.cuda(), eps=0.0).cpu()
    for b in range(8):
        _rounded(o[b], newton64(u[b], eps=0.0), 2e-3, f"matrix {b}")
        assert not o[b][u[b] == 0].any()


@pytest.mark.parametrize("n", [65, 100, 128, 256, 343, 384, 512, 1024])
def test_equal_singular_values(moe, n):
    """What is off in one direction is off in all of them."""
    u = torch.linalg.qr(torch.randn((n, n), generator=_gen(n), dtype=torch.float64))[0].float().contiguous()
    _rounded(moe.orthogonalize(u.cuda()).cpu(), newton64(u), 3e-3)


# Two sizes of values, so many of each, of norm 1 together, and values of one size.
VALUES = [(1, 0.478627245, 2, 0.62085255), (2, 0.61157397, 1, 0.50195072), (1, 0.502671066, 1, 0.86447776), (3, 0.27338099, 2, 0.62281157),
          (43, 1.0, 0, 0.0), (343, 1.0, 0, 0.0), (8, 1.0, 0, 0.0)]


@pytest.mark.parametrize("i,x,j,y", VALUES)
def test_single_values(moe, i, x, j, y):
    """One value in each row and column: each passes through the steps by itself, and all its roundings go one way.  The sizes are
    where a replay of the arithmetic is furthest off."""
    g = _gen(i + j)
    u = torch.zeros((400, 500))
    u[torch.randperm(400, generator=g)[:i + j], torch.randperm(500, generator=g)[:i + j]] = torch.tensor([x] * i + [y] * j)
    o = moe.orthogonalize(u.cuda(), eps=0.0).cpu()
    _rounded(o, newton64(u, eps=0.0), 2e-2)
    assert not o[u == 0].any()


# ---- the ends of the documented range --------------------------------------------------------

@pytest.mark.parametrize("o_dtype", [BF16, F32])
@pytest.mark.parametrize("top", [3.9994, 3.9999])
def test_singular_values_just_below_4(moe, top, o_dtype):
    """A holds their squares, to 15.9992, on its diagonal."""
    d = torch.tensor([1.0, 0.9, 0.5, 0.1])
    u = torch.zeros((70, 90))
    u[[3, 68, 41, 17], [89, 2, 40, 64]] = d
    n = float(d.double().norm())
    coef = [(top * n, 0.0, 0.0), (0.1, -0.005, 0.0)]  # the largest value, 1 / n, becomes top
    o = moe.orthogonalize(u.cuda(), steps=2, coef=coef, eps=0.0, o_dtype=o_dtype).cpu()
    ref = newton64(u, steps=2, coef=coef, eps=0.0)
    most = newton_bound(u, o_dtype, steps=2, coef=coef, eps=0.0) * (1 + HALF[o_dtype]) + HALF[o_dtype] * ref.norm()
    assert (o.double() - ref).norm() <= most
    assert int((o != 0).sum()) == 4


@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_a_polynomial_just_below_16_off_the_diagonal(moe, o_dtype):
    """Singular values 0.12 and 0.06 along (1, 1) and (1, -1) of two rows, where b s^2 + c s^4 is 15.998 and -15.998: b A + c A^2 then
    holds 15.998 off its diagonal alone."""
    top = 15.998
    s, t = 0.12, 0.06
    c = (top + top * (s / t) ** 2) / (s ** 4 - s ** 2 * t ** 2)
    b = (-top - c * t ** 4) / t ** 2
    u = torch.zeros((70, 90), dtype=torch.float64)
    u[[5, 66], 80] = s / 2 ** 0.5
    u[5, 7], u[66, 7] = t / 2 ** 0.5, -t / 2 ** 0.5
    coef, eps = [(17.0, b, c)], 1.0 - (s * s + t * t) ** 0.5  # |u| + eps is 1
    u = u.float()
    o = moe.orthogonalize(u.cuda(), steps=1, coef=coef, eps=eps, o_dtype=o_dtype).cpu()
    ref = newton64(u, steps=1, coef=coef, eps=eps)
    assert abs(ref.norm() - ((33 * s) ** 2 + t ** 2) ** 0.5) < 0.02
    most = newton_bound(u, o_dtype, steps=1, coef=coef, eps=eps) * (1 + HALF[o_dtype]) + HALF[o_dtype] * ref.norm()
    assert (o.double() - ref).norm() <= most


@pytest.mark.parametrize("R,K", [(40, 70), (70, 90)])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_zeros_with_the_smallest_eps(moe, R, K, o_dtype):
    """1 / eps is past the range of 64 bits below 5.6e-309, and 2^13 / eps below 4.6e-305."""
    u = torch.zeros((3, R, K))
    u[1] = torch.randn((R, K), generator=_gen(R)) * 1e-40
    want = moe.orthogonalize(u.cuda(), eps=0.0, o_dtype=o_dtype)
    assert want[1].isfinite().all() and want[1].any()
    for eps in (1e-300, 1e-306, 1e-310, 5e-324):
        o = moe.orthogonalize(u.cuda(), eps=eps, o_dtype=o_dtype)
        assert not o[0].any() and not o[2].any(), eps
        assert torch.equal(o[1], want[1]), eps


# ---- every form ------------------------------------------------------------------------------

def _newton64_gpu(u):
    """newton64 of a batch, with the usual coefficients, by 64-bit products on the GPU."""
    x = u.double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    tall = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if tall else x
    for a, b, c in coefs(None, 5):
        gram = torch.bmm(x, x.mT.contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x.mT.contiguous() if tall else x


# What reaches every kernel of a bf16 result above a short side of 64: forms as in test_gpu_orthogonalize.py, and whether X
# is past the caches (over 8 bytes a padded value and 256 MB).
BF16_FORMS = [(B, R, K) for B, R, K, o_dtype, *form in FORMS if o_dtype == BF16 and form[0]] + [
    (48, 512, 2048), (100, 256, 2048), (1000, 130, 130)]


@pytest.mark.parametrize("B,R,K", BF16_FORMS)
@pytest.mark.parametrize("kind", ["strong over noise", "low rank"])
def test_strong_and_low_rank_in_every_form(moe, B, R, K, kind):
    """What X's second term is for: rounded to 11 bits before each step these come out 3 to 7% off, as what is weak grows 485-fold
    and the rounding's noise with it."""
    g = torch.Generator(device="cuda").manual_seed(R + K)
    r = 3 if kind == "strong over noise" else 2
    left, right = (torch.randn(s, generator=g, device="cuda") for s in ((B, R, r), (B, r, K)))
    u = torch.bmm(left, right)
    if kind == "strong over noise":
        u += 0.01 * torch.randn((B, R, K), generator=g, device="cuda")
    o = moe.orthogonalize(u)
    for b in {0, B // 2, B - 1}:
        _rounded(o[b], _newton64_gpu(u[b:b + 1])[0], 2e-3, f"matrix {b}")


@pytest.mark.parametrize("R,K", [(16384, 16384), (65, 16384), (16384, 65), (16384, 8000)])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_longest_sides(moe, R, K, o_dtype):
    """Values at every place, one in each row and column of the shorter side (their bounds are in _newton_ref.scalar_bound)."""
    _check_spread(moe, 1, R, K, o_dtype, seed=R + K)
