"""GPU: the dense product with bias, activation and residual, and its gradient, against 64-bit forms.

Bounds are derived in tests/_train_ref.py from the number of rounded additions, the terms fp32 operands enter as, and
half a step of each result's type."""
import pytest
import torch

from tests._train_ref import (linear64, linear_bounds, linear_grad64, linear_grad_bounds, rows_of, within)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _inputs(T, K, N, act, xt, seed, bias=True, res=None):
    g = torch.Generator().manual_seed(seed)
    R = rows_of(act, N)
    x = torch.randn((T, K), generator=g).to(xt)
    w = (torch.randn((R, K), generator=g) / K ** 0.5).to(BF16)
    b = torch.randn((R,), generator=g) if bias else None
    r = torch.randn((T, N), generator=g).to(res) if res is not None else None
    return x, w, b, r


def _c(t):
    return None if t is None else t.cuda()


# T around the switch from few tokens to tiles and around tile edges; K one step, off and on the tile's K-step of 64;
# N below, off and over the tile and the 16 rows of the few-token kernel
SHAPES = [(1, 32, 1), (1, 2048, 40), (2, 96, 7), (3, 512, 130), (16, 544, 33), (17, 64, 16), (33, 160, 19),
          (64, 320, 200), (65, 32, 1), (65, 1024, 72), (127, 96, 129), (129, 64, 3), (200, 224, 257), (384, 128, 260)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
def test_linear(moe, T, K, N, act):
    for i, (xt, yt, res, bias) in enumerate([(BF16, BF16, None, True), (BF16, F32, F32, False), (F32, F32, BF16, True),
                                             (F32, BF16, BF16, True)]):
        x, w, b, r = _inputs(T, K, N, act, xt, seed=T + K + N + i, bias=bias, res=res)
        pre = torch.empty((T, w.shape[0]), dtype=yt, device="cuda")
        y = moe.linear(x.cuda(), w.cuda(), bias=_c(b), act=act, residual=_c(r), y_dtype=yt, pre=pre)
        ref_y, ref_z = linear64(x, w, b, act, r)
        by, bz = linear_bounds(x, w, b, act, r, yt, x_rounded=xt == F32 and yt == BF16 and T > 64)
        assert y.dtype == yt
        within(y, ref_y, by, f"y {xt} {yt}")
        within(pre, ref_z, bz, f"pre {xt} {yt}")


GRAD_SHAPES = [(1, 32, 1), (3, 96, 7), (16, 64, 64), (65, 160, 19), (63, 32, 130), (128, 544, 8), (200, 224, 201),
               (700, 96, 36), (160, 64, 96), (96, 32, 32)]


@pytest.mark.parametrize("T,K,N", GRAD_SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
def test_linear_backward(moe, T, K, N, act):
    for i, (xt, gt, dxt, dwt) in enumerate([(BF16, BF16, BF16, F32), (BF16, F32, F32, F32), (F32, F32, F32, F32),
                                            (F32, BF16, BF16, BF16), (BF16, F32, BF16, BF16)]):
        x, w, _, _ = _inputs(T, K, N, act, xt, seed=T + K + N + 50 + i)
        g = torch.Generator().manual_seed(T + i)
        dy = torch.randn((T, N), generator=g).to(gt)
        pre = (2 * torch.randn((T, w.shape[0]), generator=g)).to(gt)
        dx, dw, db = moe.linear_backward(dy.cuda(), x.cuda(), w.cuda(), act=act, pre=_c(pre), dx_dtype=dxt, dw_dtype=dwt)
        rx, rw, rb, _ = linear_grad64(dy, x, w, act, pre)
        bx, bw, bb = linear_grad_bounds(dy, x, w, act, pre, dxt, dwt)
        assert dx.dtype == dxt and dw.dtype == dwt and db.dtype == F32
        within(dx, rx, bx, f"dx {xt} {gt} {dxt}")
        within(dw, rw, bw, f"dw {xt} {gt} {dwt}")
        within(db, rb, bb, f"db {xt} {gt}")


def test_fp32_operands_are_held_to_full_precision(moe):
    """Values whose low mantissa bits matter: products that cancel to 2^-20 of their size come out right."""
    T, K, N = 130, 64, 16
    g = torch.Generator().manual_seed(1)
    half = torch.randn((T, K // 2), generator=g)
    x = torch.cat([half * (1 + 2.0 ** -20), -half], 1)
    row = (torch.randn((N, K // 2), generator=g)).to(BF16)
    w = torch.cat([row, row], 1)
    ref = x.double() @ w.double().t()
    S = x.double().abs() @ w.double().abs().t()
    for n in (5, T):  # both kernels
        y = moe.linear(x[:n].cuda(), w.cuda())
        within(y, ref[:n], (3 * K + 32) * 2.0 ** -24 * S[:n], "y")
    # the gradient: dz = x^T against an all-equal W column pattern cancels in the same way
    dy = x.t().contiguous()                      # [K, T] gradients of K rows
    cols = torch.randn((T, 32), generator=g).to(BF16)
    dx, _, _ = moe.linear_backward(dy.cuda(), torch.zeros((K, 32), dtype=BF16).cuda(), cols.cuda(), dx_dtype=F32,
                                   need=("dx",))
    S = dy.double().abs() @ cols.double().abs()
    within(dx, dy.double() @ cols.double(), (3 * T + 64) * 2.0 ** -24 * S, "dx")
    both = dx.cpu().double()[:K // 2] + dx.cpu().double()[K // 2:]  # = 2^-20 of the first half's
    assert (both - 2.0 ** -20 * (half.t().double() @ cols.double())).abs().max() <= ((6 * T + 128) * 2.0 ** -24 * S).max()


def test_large_and_small_magnitudes(moe):
    x, w, b, _ = _inputs(100, 64, 24, "none", F32, seed=3)
    x[::3] *= 1e30
    x[1::3] *= 1e-25
    y = moe.linear(x.cuda(), w.cuda())
    ref, _ = linear64(x, w, None, "none", None)
    by, _ = linear_bounds(x, w, None, "none", None, F32, False)
    within(y, ref, by, "y")
    for act in ("gelu", "silu"):  # far tails: no NaN, the right limits
        z = torch.tensor([[-1e4, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 1e4]]).repeat(70, 4)
        eye = torch.eye(32).to(BF16)
        y = moe.linear(z.cuda(), eye.cuda(), act=act)
        ref, _ = linear64(z, eye, None, act, None)
        by, _ = linear_bounds(z, eye, None, act, None, F32, False)
        within(y, ref, by, act)


def test_a_nonfinite_row_stays_in_its_row(moe):
    x, w, b, _ = _inputs(150, 96, 40, "silu", BF16, seed=4)
    clean = moe.linear(x.cuda(), w.cuda(), act="silu")
    x[17, 3], x[140, 90] = float("nan"), float("inf")
    y = moe.linear(x.cuda(), w.cuda(), act="silu")
    keep = [t for t in range(150) if t not in (17, 140)]
    assert torch.equal(y[keep], clean[keep])
    assert y[17].isnan().all() and not torch.isfinite(y[140]).all()
    dy = torch.randn((150, 40), generator=torch.Generator().manual_seed(0)).to(BF16)
    pre = torch.randn((150, 40), generator=torch.Generator().manual_seed(1)).to(BF16)
    a = moe.linear_backward(dy.cuda(), x.nan_to_num(0, 0, 0).cuda(), w.cuda(), act="silu", pre=pre.cuda(), need=("dx",))[0]
    dy[9, 2] = float("nan")
    d = moe.linear_backward(dy.cuda(), x.nan_to_num(0, 0, 0).cuda(), w.cuda(), act="silu", pre=pre.cuda(), need=("dx",))[0]
    keep = [t for t in range(150) if t != 9]
    assert torch.equal(d[keep], a[keep]) and d[9].isnan().all()


def test_residual_in_place(moe):
    for T in (5, 90):
        x, w, b, r = _inputs(T, 128, 68, "gelu", BF16, seed=T, res=F32)
        r = r.cuda()
        want = moe.linear(x.cuda(), w.cuda(), bias=b.cuda(), act="gelu", residual=r, y_dtype=F32)
        got = moe.linear(x.cuda(), w.cuda(), bias=b.cuda(), act="gelu", residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("T", [7, 150])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_views_off_alignment_and_nothing_past_the_end(moe, T, act):
    """Outputs, bias, residual and gradients that start at odd elements: the same values, and the elements around them
    untouched."""
    K, N = 96, 36
    x, w, b, r = _inputs(T, K, N, act, BF16, seed=T, res=BF16)
    R = w.shape[0]

    def odd(t, dtype):
        big = torch.full((t[0] * t[1] + 2,) if isinstance(t, tuple) else (t.numel() + 2,), 7.0, dtype=dtype, device="cuda")
        view = big[1:-1].view(t if isinstance(t, tuple) else t.shape)
        if not isinstance(t, tuple):
            view.copy_(t)
        return big, view

    bb, vb = odd(b, F32)
    br, vr = odd(r, BF16)
    by, vy = odd((T, N), BF16)
    bp, vp = odd((T, R), BF16)
    moe.linear(x.cuda(), w.cuda(), bias=vb, act=act, residual=vr, y=vy, pre=vp)
    pre = torch.empty((T, R), dtype=BF16, device="cuda")
    y = moe.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, residual=r.cuda(), pre=pre)
    assert torch.equal(vy, y) and torch.equal(vp, pre)
    bd, vd = odd(torch.randn((T, N), generator=torch.Generator().manual_seed(2)).to(BF16), BF16)
    bg, vg = odd((1, R), F32)
    got = moe.linear_backward(vd, x.cuda(), w.cuda(), act=act, pre=vp, db=vg.view(R))
    want = moe.linear_backward(vd.clone(), x.cuda(), w.cuda(), act=act, pre=pre)
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    for big in (bb, br, by, bp, bd, bg):
        assert big[0] == 7 and big[-1] == 7
    rows = torch.full((T + 4, K), 7.0, dtype=BF16, device="cuda")
    moe.linear_backward(vd, x.cuda(), w.cuda(), act=act, pre=vp, need=("dx",), dx=rows[2:-2])
    torch.cuda.synchronize()
    assert torch.equal(rows[2:-2], want[0]) and (rows[:2] == 7).all() and (rows[-2:] == 7).all()


def test_no_rows(moe):
    x, w, b, _ = _inputs(0, 64, 12, "none", BF16, seed=0)
    assert moe.linear(x.cuda(), w.cuda(), bias=b.cuda()).shape == (0, 12)
    dx, dw, db = moe.linear_backward(torch.empty((0, 12), dtype=BF16).cuda(), x.cuda(), w.cuda(),
                                     dw=torch.full((12, 64), 3.0).cuda(), db=torch.full((12,), 3.0).cuda())
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_each_output_alone_equals_all_together(moe):
    """What is asked for beside an output does not change it, apart from how a reduction is cut into parts."""
    x, w, _, _ = _inputs(300, 96, 40, "swiglu", BF16, seed=5)
    g = torch.Generator().manual_seed(6)
    dy, pre = torch.randn((300, 40), generator=g).to(BF16), torch.randn((300, 80), generator=g).to(BF16)
    args = [t.cuda() for t in (dy, x, w)]
    every = moe.linear_backward(*args, act="swiglu", pre=pre.cuda())
    bounds = linear_grad_bounds(dy, x, w, "swiglu", pre, BF16, F32)
    refs = linear_grad64(dy, x, w, "swiglu", pre)
    for i, name in enumerate(("dx", "dw", "db")):
        one = moe.linear_backward(*args, act="swiglu", pre=pre.cuda(), need=(name,))
        assert [t is None for t in one] == [j != i for j in range(3)]
        within(one[i], refs[i], bounds[i], name)
        within(every[i], refs[i], bounds[i], name)


def test_repeatable_and_on_another_stream(moe):
    x, w, b, r = _inputs(500, 256, 64, "gelu", F32, seed=8, res=F32)
    x, w, b, r = x.cuda(), w.cuda(), b.cuda(), r.cuda()
    pre = torch.empty((500, 64), device="cuda")
    y = moe.linear(x, w, bias=b, act="gelu", residual=r, pre=pre)
    dx, dw, db = moe.linear_backward(r, x, w, act="gelu", pre=pre)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2 = moe.linear(x, w, bias=b, act="gelu", residual=r, stream=s)
    back = moe.linear_backward(r, x, w, act="gelu", pre=pre, stream=s)
    s.synchronize()
    assert torch.equal(y, y2)
    for a, c in zip((dx, dw, db), back):
        assert torch.equal(a, c)


def test_prompt_chunk(moe):
    """The 8,192-token chunk through 2,048 x 512 SwiGLU rows and its gradient, against 64-bit products on the GPU."""
    T, K, N = 8192, 2048, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF16)
    w = (torch.randn((2 * N, K), generator=g, device="cuda") / K ** 0.5).to(BF16)
    dy = torch.randn((T, N), generator=g, device="cuda").to(BF16)
    pre = torch.empty((T, 2 * N), dtype=BF16, device="cuda")
    y = moe.linear(x, w, act="swiglu", pre=pre)
    ry, rz = linear64(x, w, None, "swiglu", None)
    by, bz = linear_bounds(x, w, None, "swiglu", None, BF16, False)
    within(y, ry, by.cpu(), "y")
    within(pre, rz, bz.cpu(), "pre")
    dx, dw, db = moe.linear_backward(dy, x, w, act="swiglu", pre=pre)
    rx, rw, rb, _ = linear_grad64(dy, x, w, "swiglu", pre)
    bx, bw, bb = linear_grad_bounds(dy, x, w, "swiglu", pre, BF16, F32)
    within(dx, rx, bx.cpu(), "dx")
    within(dw, rw, bw.cpu(), "dw")
    within(db, rb, bb.cpu(), "db")


def _big(T, K, N, act, xt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = rows_of(act, N)
    return (torch.randn((T, K), generator=g, device="cuda").to(xt),
            (torch.randn((R, K), generator=g, device="cuda") / K ** 0.5).to(BF16),
            torch.randn((R,), generator=g, device="cuda"), torch.randn((T, N), generator=g, device="cuda"), g)


# sizes that take 128 x 128 and 256 x 256 tiles, with last steps of 32 k, odd columns and rows past the last tile
@pytest.mark.parametrize("T,K,N,act,xt,yt", [(2100, 544, 1001, "silu", BF16, BF16), (2100, 544, 1003, "swiglu", BF16, F32),
                                             (4000, 1056, 1500, "none", F32, F32), (4000, 4128, 4094, "gelu", BF16, BF16),
                                             (4000, 2080, 2047, "swiglu", BF16, BF16)])
def test_large_tiles(moe, T, K, N, act, xt, yt):
    x, w, b, r, _ = _big(T, K, N, act, xt, seed=N)
    pre = torch.empty((T, w.shape[0]), dtype=yt, device="cuda")
    y = moe.linear(x, w, bias=b, act=act, residual=r, y_dtype=yt, pre=pre)
    ry, rz = linear64(x, w, b, act, r)
    by, bz = linear_bounds(x, w, b, act, r, yt, False)
    within(y, ry, by.cpu(), "y")
    within(pre, rz, bz.cpu(), "pre")


# both products on 128 x 128 tiles with dW's reduction cut (and odd columns), and on 256 x 256 tiles from fp32
@pytest.mark.parametrize("T,K,N,act,xt,gt,dxt,dwt", [(4000, 2048, 1001, "silu", BF16, BF16, BF16, F32),
                                                     (8200, 2048, 515, "swiglu", BF16, BF16, BF16, BF16),
                                                     (3000, 1024, 2000, "none", F32, F32, F32, F32)])
def test_large_tiles_gradient(moe, T, K, N, act, xt, gt, dxt, dwt):
    x, w, _, r, g = _big(T, K, N, act, xt, seed=N)
    dy, pre = r.to(gt), torch.randn((T, w.shape[0]), generator=g, device="cuda").to(gt)
    dx, dw, db = moe.linear_backward(dy, x, w, act=act, pre=pre, dx_dtype=dxt, dw_dtype=dwt)
    rx, rw, rb, _ = linear_grad64(dy, x, w, act, pre)
    bx, bw, bb = linear_grad_bounds(dy, x, w, act, pre, dxt, dwt)
    within(dx, rx, bx.cpu(), "dx")
    within(dw, rw, bw.cpu(), "dw")
    within(db, rb, bb.cpu(), "db")


@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_infinities_stay_where_they_are(moe, T, xt):
    """An infinite activation makes its own products infinite and no others, also in the last, partial step of a
    reduction and for the rows and columns next to it."""
    x, w, _, _ = _inputs(T, 96, 33, "none", xt, seed=T)
    x[T - 1, 95] = float("inf")
    y = moe.linear(x.cuda(), w.cuda()).cpu()
    assert torch.isfinite(y[:T - 1]).all()
    want = torch.where(w[:, 95] > 0, float("inf"), torch.where(w[:, 95] < 0, -float("inf"), float("nan"))).float()
    assert torch.equal(y[T - 1].float().nan_to_num(7, 1e38, -1e38), want.nan_to_num(7, 1e38, -1e38))
    dy = torch.randn((T, 33), generator=torch.Generator().manual_seed(1)).to(BF16)
    dx, dw, _ = moe.linear_backward(dy.cuda(), x.cuda(), w.cuda(), need=("dx", "dw"))
    assert torch.isfinite(dx).all() and torch.isfinite(dw[:, :95]).all() and not torch.isfinite(dw[:, 95]).any()
    assert torch.equal(torch.isinf(dw[:, 95]).cpu(), dy[T - 1] != 0)


# fp32 activations split inside the tiles: the reduction cut into parts that end on and off its last, partial step, both
# halves of a SwiGLU tile, one term and three; and, for the largest, as planes of one term
@pytest.mark.parametrize("T,K,N,act,yt", [(65, 4128, 201, "gelu", F32), (100, 2080, 515, "swiglu", F32),
                                          (300, 2080, 1030, "silu", BF16), (66, 8224, 33, "swiglu", BF16),
                                          (1000, 1056, 999, "none", F32), (4000, 4128, 4094, "none", BF16)])
def test_fp32_activations_on_tiles(moe, T, K, N, act, yt):
    x, w, b, r, _ = _big(T, K, N, act, F32, seed=N + T)
    pre = torch.empty((T, w.shape[0]), dtype=yt, device="cuda")
    y = moe.linear(x, w, bias=b, act=act, residual=r, y_dtype=yt, pre=pre)
    ry, rz = linear64(x, w, b, act, r)
    by, bz = linear_bounds(x, w, b, act, r, yt, yt == BF16)
    within(y, ry, by.cpu(), "y")
    within(pre, rz, bz.cpu(), "pre")


@pytest.mark.parametrize("T,K,N,act,xt,gt", [(1, 224, 111, "swiglu", BF16, BF16), (6, 256, 19, "gelu", BF16, F32),
                                             (2, 96, 40, "none", F32, F32), (1, 64, 8000, "silu", F32, BF16)])
def test_few_values_of_dz_are_not_rounded(moe, T, K, N, act, xt, gt):
    """bf16 gradients of few tokens are the rounded exact ones but for fp32's part of the error: half a step of bf16,
    and what two terms leave of dz (and of fp32 x), 2^-16 of the sums' magnitudes each, counted double."""
    x, w, _, r = _inputs(T, K, N, act, xt, seed=N, res=gt)
    pre = torch.randn((T, w.shape[0]), generator=torch.Generator().manual_seed(N + 1)).to(gt)
    dx, dw, _ = moe.linear_backward(r.cuda(), x.cuda(), w.cuda(), act=act, pre=pre.cuda(), dx_dtype=BF16, dw_dtype=BF16)
    rx, rw, _, dz = linear_grad64(r, x, w, act, pre)
    # bounds of the fp32 results, whose dz carries the activation's own error
    bx, bw, _ = linear_grad_bounds(r, x, w, act, pre, F32, F32)
    za = dz.abs()
    within(dx, rx, bx + 2.0 ** -8 * (rx.abs() + bx) + 2 * 2.0 ** -16 * (za @ w.double().abs()), "dx")
    within(dw, rw, bw + 2.0 ** -8 * (rw.abs() + bw) + 4 * 2.0 ** -16 * (za.t() @ x.double().abs()), "dw")
