"""GPU: the orthogonalised update against a 64-bit form.

Bounds are derived in tests/_newton_ref.py.  Matrices with one value in each row and column are checked value by value and
zero by zero (every place of every tile shape, and both orders of sides); dense ones by the norm of their error."""
import pytest
import torch

from tests._newton_ref import newton64, newton_bound, scalar_bound
from tests._train_ref import HALF, U

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


def _near(got, u, o_dtype, what="", **kw):
    ref = newton64(u, **kw)
    off = (got.double().cpu() - ref).norm()
    h = HALF[o_dtype]
    most = newton_bound(u, o_dtype, **kw) * (1 + h) + h * ref.norm()
    assert torch.isfinite(got).all(), what
    assert off <= most, f"{what}: off {off:.3e}, {off / ref.norm():.2e} of its norm; bound {most:.3e}"
    return float(off / ref.norm())


def _dense(R, K, kind, seed):
    g = _gen(seed)
    n = torch.randn((R, K), generator=g)
    if kind == "even":
        return n
    r = max(1, min(R, K) // 8)
    low = torch.randn((R, r), generator=g) @ torch.randn((r, K), generator=g)
    return low / r ** 0.5 + (0.1 * n if kind == "strong" else 0)


# the shorter side around 16, 32, 48 and 64 (sums on the shorter side up to there), the longer one around stretches of 64 and
# the 32 workgroups that share them (a stretch each; more are in test_gpu_orthogonalize_moment.py)
SIZES = [(15, 17), (17, 100), (33, 49), (48, 1025), (49, 64), (64, 1024), (2000, 60), (1, 1), (1, 50), (50, 1), (3, 5), (16, 16), (60, 137), (64, 64), (65, 63), (129, 40), (100, 300), (257, 200), (200, 321)]


@pytest.mark.parametrize("R,K", SIZES)
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_dense(moe, R, K, o_dtype):
    for i, kind in enumerate(["even", "strong", "low"]):
        u = _dense(R, K, kind, seed=R + K + i)
        o = moe.orthogonalize(u.cuda(), o_dtype=o_dtype)
        assert o.shape == (R, K) and o.dtype == o_dtype
        _near(o, u, o_dtype, f"{kind}")
        one = moe.orthogonalize(u.cuda(), o_dtype=o_dtype, steps=1)
        _near(one, u, o_dtype, f"{kind}, one step", steps=1)


def test_bf16_gradients(moe):
    for R, K in [(60, 137), (137, 60), (64, 128)]:
        u = _dense(R, K, "strong", 3).to(BF16)
        _near(moe.orthogonalize(u.cuda()), u.float(), BF16)
        _near(moe.orthogonalize(u.cuda(), o_dtype=F32), u.float(), F32)


def test_low_rank_gradients_stay_clean(moe):
    """Two strong directions among 128: X in one fp16 term would leave an error of 5% or more here, as a step multiplies
    what is small by 3.44 and five of them by 485.  With the sum over both terms the first X's roundings (2^-22 of its norm
    1) come to at most 485 * 2^-22 = 1.2e-4 beside a result of norm 0.96 or more; a bf16 result is held to the 2e-3 that
    are documented for it, and its rounding."""
    g = _gen(5)
    u = torch.randn((128, 2), generator=g) @ torch.randn((2, 512), generator=g)
    assert _near(moe.orthogonalize(u.cuda()), u, BF16) < 2e-3 + 2.0 ** -8
    assert _near(moe.orthogonalize(u.cuda(), o_dtype=F32), u, F32) < 2e-4


@pytest.mark.parametrize("R,K", [(8, 8), (16, 40), (17, 17), (24, 24), (33, 36), (64, 64), (200, 24), (64, 700), (65, 65), (128, 200)])
@pytest.mark.parametrize("strong,noise", [(1, 1.0), (1, 0.3), (1, 0.1), (1, 0.03), (1, 0.01), (3, 0.1), (3, 0.01)])
def test_strong_directions_over_noise(moe, R, K, strong, noise):
    """What is weak grows most on the way, and noise of the strong directions' size with it.  bf16: with o' the result before its
    rounding and |o' - ref| <= 2e-3 |ref| as documented; the way from a value to the nearest bf16 changes by no more than the
    value does, so the rounding adds at most |bf16(ref) - ref| + |o' - ref|.  fp32: newton_bound."""
    g = _gen(R + K + strong)
    u = torch.randn((16, R, strong), generator=g) @ torch.randn((16, strong, K), generator=g) / strong ** 0.5
    u = u + noise * torch.randn((16, R, K), generator=g)
    o, f = moe.orthogonalize(u.cuda()).double().cpu(), moe.orthogonalize(u.cuda(), o_dtype=F32)
    for b in range(16):
        ref = newton64(u[b])
        most = 2 * 2e-3 * ref.norm() + (ref.to(BF16).double() - ref).norm()
        assert (o[b] - ref).norm() <= most, (b, float((o[b] - ref).norm() / ref.norm()))
        _near(f[b], u[b], F32)


# (B, R, K, o): rows of the tiles of A and P, of P X, and whether their K-steps bring two pieces
FORMS = [(1, 64, 128, BF16, 0, 0, 0, 0), (7, 500, 33, F32, 0, 0, 0, 0), (1, 190, 130, BF16, 32, 32, 1, 1),
         (2, 130, 190, F32, 32, 32, 1, 1), (2, 5000, 70, BF16, 32, 64, 1, 0), (2, 70, 5000, F32, 32, 64, 1, 0),
         (1, 70, 5000, BF16, 32, 64, 1, 1), (1, 5000, 70, F32, 32, 64, 1, 1), (24, 70, 5000, BF16, 32, 128, 1, 0),
         (24, 5000, 70, F32, 32, 128, 1, 0), (48, 190, 130, BF16, 64, 64, 0, 0), (48, 130, 190, F32, 64, 64, 0, 0),
         (1, 1000, 12000, BF16, 64, 128, 1, 0), (3, 513, 515, F32, 64, 64, 1, 1), (3, 4097, 1025, BF16, 64, 256, 0, 0), (8, 2050, 700, F32, 64, 256, 1, 0),
         (24, 700, 512, BF16, 128, 128, 0, 0), (3, 1100, 1100, BF16, 128, 128, 0, 0), (3, 1101, 1100, F32, 128, 128, 0, 0),
         (8, 700, 2050, BF16, 128, 256, 0, 0), (24, 515, 513, BF16, 192, 64, 0, 0), (24, 513, 515, F32, 192, 64, 0, 0),
         (8, 1100, 1100, BF16, 192, 128, 0, 0), (48, 1030, 700, BF16, 192, 256, 0, 0), (48, 700, 1030, F32, 192, 256, 0, 0),
         (4, 2050, 2100, BF16, 256, 128, 0, 0), (24, 1500, 1700, BF16, 256, 256, 0, 0), (8, 1700, 1500, F32, 256, 256, 0, 0)]


def _spread(B, R, K, seed):
    """B matrices with one value in each row and column of the shorter side; the values and where they lie."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = min(R, K)
    u = torch.zeros((B, R, K), device="cuda")
    d = (torch.rand((B, m), generator=g, device="cuda") + 0.05) * (2.0 * torch.randint(0, 2, (B, m), generator=g, device="cuda") - 1)
    rows = torch.stack([torch.randperm(R, generator=g, device="cuda")[:m] for _ in range(B)])
    cols = torch.stack([torch.randperm(K, generator=g, device="cuda")[:m] for _ in range(B)])
    at = torch.arange(B, device="cuda")[:, None]
    u[at, rows, cols] = d
    return u, d, (at, rows, cols)


def _check_spread(moe, B, R, K, o_dtype, seed):
    u, d, at = _spread(B, R, K, seed)
    o = moe.orthogonalize(u, o_dtype=o_dtype)
    got = o[at].double().cpu()
    h = HALF[o_dtype]
    for b in range(B):
        ref, e = scalar_bound(d[b].cpu(), float(d[b].double().norm()) + 1e-7, o_dtype)
        over = (got[b] - ref).abs() - (e * (1 + h) + h * ref.abs())
        assert (over <= 0).all(), (b, float(over.max()))
    o[at] = 0
    assert not o.any()


@pytest.mark.parametrize("B,R,K", [(1, 1, 1), (1, 5, 70), (3, 70, 5), (2, 64, 64), (2, 65, 129), (1, 200, 320), (5, 33, 191)])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_places(moe, B, R, K, o_dtype):
    _check_spread(moe, B, R, K, o_dtype, seed=B + R + K)


@pytest.mark.parametrize("B,R,K,o_dtype,gram,apply,gram_paired,apply_paired", FORMS)
def test_places_in_every_form(moe, B, R, K, o_dtype, gram, apply, gram_paired, apply_paired):
    form = moe.orthogonalize_form(B, R, K, o_dtype)
    assert tuple(form.values()) == (gram, apply, gram_paired, apply_paired), form
    _check_spread(moe, B, R, K, o_dtype, seed=R)


@pytest.mark.parametrize("B,R,K,o_dtype", [f[:4] for f in FORMS])
def test_dense_in_every_form(moe, B, R, K, o_dtype):
    """The last matrix of the batch, against 64-bit products on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(R + K)
    u = torch.randn((B, R, K), generator=g, device="cuda")
    o = moe.orthogonalize(u, o_dtype=o_dtype)[-1].double()
    x = u[-1].double()
    x = x / (x.norm() + 1e-7)
    x = x.t().contiguous() if R > K else x
    a, b, c = (float(torch.tensor(v)) for v in (3.4445, -4.7750, 2.0315))
    for _ in range(5):
        gr = x @ x.t()
        x = a * x + (b * gr + c * gr @ gr) @ x
    x = x.t() if R > K else x
    h = HALF[o_dtype]
    off, n = float((o - x).norm()), float(x.norm())
    assert off <= newton_bound(u[-1], o_dtype) * (1 + h) + h * n, off / n


def test_scale_does_not_matter(moe):
    """Powers of two on the gradient change no bit without eps; the norm of squares past fp32's range among them."""
    u = _dense(70, 90, "strong", 8).cuda()
    want = moe.orthogonalize(u, eps=0.0, o_dtype=F32)
    for s in (2.0 ** -100, 2.0 ** 100, 2.0 ** -60, 2.0 ** 3):
        assert torch.equal(moe.orthogonalize(u * s, eps=0.0, o_dtype=F32), want), s
    # with eps, small gradients stay small: X = u / (|u| + eps)
    small = (u / u.norm() * 1e-7).cpu()
    _near(moe.orthogonalize(small.cuda(), o_dtype=F32), small, F32)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("R,K", [(60, 137), (131, 64)])
def test_momentum(moe, nesterov, gt, R, K):
    g = _gen(9)
    m = torch.randn((2, R, K), generator=g)
    gr = torch.randn((2, R, K), generator=g).to(gt)
    beta = 0.95
    moment = m.cuda()
    o = moe.orthogonalize(gr.cuda(), momentum=moment, beta=beta, nesterov=nesterov, o_dtype=F32)
    want = beta * m.double() + (1 - beta) * gr.double()
    # beta and 1 - beta are rounded to fp32, then one product and one fused sum
    assert ((moment.cpu().double() - want).abs() <= 3 * U * (beta * m.double().abs() + (1 - beta) * gr.double().abs())).all()
    u = beta * moment.cpu().double() + (1 - beta) * gr.double() if nesterov else moment.cpu().double()
    for b in range(2):
        _near(o[b], u[b], F32)
    # beta 0: the gradient itself
    moment = torch.full_like(moment, 3.0)
    assert torch.equal(moe.orthogonalize(gr.cuda(), momentum=moment, beta=0.0, nesterov=nesterov, o_dtype=F32),
                       moe.orthogonalize(gr.cuda(), o_dtype=F32))
    assert torch.equal(moment.cpu(), gr.float())


def test_coefficients_and_steps(moe):
    u = _dense(48, 80, "even", 1)
    one = (1.5, -0.5, 0.0)
    many = [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    _near(moe.orthogonalize(u.cuda(), coef=one, steps=12, o_dtype=F32), u, F32, coef=one, steps=12)
    _near(moe.orthogonalize(u.cuda(), coef=many, steps=3, o_dtype=F32), u, F32, coef=many, steps=3)
    _near(moe.orthogonalize(u.cuda(), coef=many, steps=3), u, BF16, coef=many, steps=3)
    # more steps of the usual quintic than the sums on the shorter side hold in 32 bits, and than they hold in 64
    for steps in (6, 7, 9):
        _near(moe.orthogonalize(u.cuda(), steps=steps, o_dtype=F32), u, F32, steps=steps)
        _near(moe.orthogonalize(u.cuda(), steps=steps), u, BF16, steps=steps)
    # twelve cubic steps end near an orthogonal matrix
    o = moe.orthogonalize(u.cuda(), coef=one, steps=16, o_dtype=F32).double().cpu()
    assert (o @ o.t() - torch.eye(48, dtype=torch.float64)).abs().max() < 1e-3


@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_singular_values_up_to_the_documented_range(moe, o_dtype):
    """X's singular values to just below 4 and b s^2 + c s^4 to just below 16 on the way, on matrices of one value in each row and
    column, where A and P hold the squares themselves: they stay finite and as exact as others."""
    d = torch.tensor([1.0, 0.9, 0.5, 0.1])
    u = torch.zeros((70, 90))
    u[[3, 68, 41, 17], [89, 2, 40, 64]] = d
    n = float(d.double().norm())
    top = 3.99 * n  # takes the largest value, 1 / n, to 3.99
    for coef in ([(top, 0.0, 0.0), (0.1, -0.005, 0.0)], [(top, 0.0, 0.0), (-15.0, 1.004, 0.0)],
                 [(top, 0.0, 0.0), (1.0, -1.004, 0.0)], [(top, 0.0, 0.0), (-15.0, 0.0, 0.063)]):
        o = moe.orthogonalize(u.cuda(), steps=len(coef), coef=coef, eps=0.0, o_dtype=o_dtype)
        got = o.cpu()[[3, 68, 41, 17], [89, 2, 40, 64]].double()
        ref, e = scalar_bound(d, n, o_dtype, steps=len(coef), coef=coef)
        h = HALF[o_dtype]
        assert ((got - ref).abs() <= e * (1 + h) + h * ref.abs()).all(), (got, ref)
        assert int((o != 0).sum()) == 4


@pytest.mark.parametrize("R,K", [(40, 70), (70, 90)])
def test_zero_and_nonfinite_matrices_stay_alone(moe, R, K):
    u = torch.stack([_dense(R, K, "strong", s) for s in range(6)])
    clean = moe.orthogonalize(u.cuda())
    u[1] = 0.0
    u[2, 3, 5] = float("nan")
    u[4, R - 1, K - 1] = float("inf")
    for eps in (1e-7, 0.0):
        o = moe.orthogonalize(u.cuda(), eps=eps)
        assert not o[1].any()
        assert o[2].isnan().all() and o[4].isnan().all()
        if eps:
            assert torch.equal(o[[0, 3, 5]], clean[[0, 3, 5]])


def test_same_bits_every_time_and_in_a_workspace_of_garbage(moe):
    for R, K in [(60, 137), (300, 200)]:
        u = _dense(R, K, "strong", 2).cuda()
        want = moe.orthogonalize(u)
        ws = torch.full((moe.orthogonalize_workspace_bytes(1, R, K),), 0xFF, dtype=torch.uint8, device="cuda")  # (NaNs)
        o = torch.full((R + 2, K), 7.0, dtype=BF16, device="cuda")
        moe.orthogonalize(u, o=o[1:-1], ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(o[1:-1], want) and (o[0] == 7).all() and (o[-1] == 7).all()


@pytest.mark.parametrize("R,K", [(37, 51), (81, 67)])
def test_views_off_alignment(moe, R, K):
    u = _dense(R, K, "strong", 4)
    big = torch.full((R * K + 2,), 7.0, device="cuda")
    big[1:-1] = u.reshape(-1).cuda()
    mom = torch.full((R * K + 2,), 7.0, device="cuda")
    mom[1:-1] = 0.25
    out = torch.full((R * K + 2,), 7.0, dtype=BF16, device="cuda")
    moe.orthogonalize(big[1:-1].view(R, K), momentum=mom[1:-1].view(R, K), o=out[1:-1].view(R, K))
    m2 = torch.full((R, K), 0.25, device="cuda")
    want = moe.orthogonalize(u.cuda(), momentum=m2)
    assert torch.equal(out[1:-1].view(R, K), want) and torch.equal(mom[1:-1].view(R, K), m2)
    for b in (big, mom, out):
        assert b[0] == 7 and b[-1] == 7


def test_no_matrices(moe):
    o = moe.orthogonalize(torch.empty((0, 8, 8)).cuda())
    assert o.shape == (0, 8, 8) and o.dtype == BF16


def test_streams_and_graph(moe):
    g = torch.Generator(device="cuda").manual_seed(1)
    for B, R, K in [(1, 60, 137), (3, 200, 70)]:
        u = torch.randn((B, R, K), generator=g, device="cuda")
        m0 = torch.randn((B, R, K), generator=g, device="cuda")
        m = m0.clone()
        want = moe.orthogonalize(u, momentum=m)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        m1 = m0.clone()
        torch.cuda.synchronize()
        o1 = moe.orthogonalize(u, momentum=m1, stream=s)
        s.synchronize()
        assert torch.equal(o1, want) and torch.equal(m1, m)
        o = torch.zeros_like(want)
        ws = torch.empty(moe.orthogonalize_workspace_bytes(B, R, K), dtype=torch.uint8, device="cuda")
        mg = m0.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.orthogonalize(u, momentum=mg, o=o, ws=ws)
        mg.copy_(m0)
        me = m0.clone()
        for k in range(3):
            u.copy_(torch.randn((B, R, K), generator=g, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, moe.orthogonalize(u, momentum=me)) and torch.equal(mg, me), k
            torch.cuda.synchronize()
