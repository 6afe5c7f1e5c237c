"""GPU: rows to 8-bit codes, and the dense product of 8-bit integers, against 64-bit forms.

Codes and scales are compared for equality.  The product's bounds are derived in tests/_q8_ref.py; where scales are powers
of two and no bias is added its results are exact and are compared for equality too."""
import pytest
import torch

from tests._q8_ref import codes64, q8_64, q8_bound
from tests._train_ref import rows_of, within

pytestmark = pytest.mark.gpu
F32, BF16, I8 = torch.float32, torch.bfloat16, torch.int8


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- codes ----------------------------------------------------------------------------

def _check_codes(moe, x):
    q, s = moe.quantize_rows(x.cuda())
    rq, rs = codes64(x)
    assert q.dtype == I8 and s.dtype == F32
    assert torch.equal(s.cpu().nan_to_num(-1.0), rs.nan_to_num(-1.0))
    assert torch.equal(q.cpu(), rq)


# K around every change of kernel; T around a workgroup's four rows
@pytest.mark.parametrize("K", [32, 96, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 16384])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes(moe, K, dtype):
    for T in (1, 3, 4, 5, 130):
        x = torch.randn((T, K), generator=_gen(T + K)) * torch.exp(2 * torch.randn((T, 1), generator=_gen(K)))
        _check_codes(moe, x.to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes_of_ties_and_of_values_beside_them(moe, dtype):
    """Scales of 2^k and others, with every half between two codes and its neighbours on either side."""
    rows = []
    for i, s in enumerate([1.0, 2.0 ** -20, 2.0 ** 30, 0.75, 1.0 / 3, 1.1754944e-38, 3.0e-38, 2.0e36, 0.0078125]):
        s = torch.tensor(s, dtype=F32)
        half = (torch.arange(-127, 127).double() + 0.5) * s.double()
        near = half.float()
        x = torch.cat([near, torch.nextafter(near, torch.tensor(float("inf"))),
                       torch.nextafter(near, torch.tensor(-float("inf"))), s * 127 * torch.ones(6)])
        rows.append(x)
    x = torch.stack(rows)
    assert x.shape[1] == 768
    _check_codes(moe, x.to(dtype))


def test_codes_beside_a_border_by_the_thousand(moe):
    """Row sizes at random: the fp32 values next to each half of the row's own scale."""
    g = _gen(11)
    top = torch.rand((400, 1), generator=g) + 1.0
    s = (top.double() / 127).float()
    n = torch.randint(-126, 126, (400, 1023), generator=g)
    x = ((n.double() + 0.5) * s.double()).float()
    x = torch.nextafter(x, x + torch.randint(-1, 2, x.shape, generator=g).float())
    x = torch.cat([x, top], 1)
    _check_codes(moe, x)


@pytest.mark.parametrize("K", [64, 2048, 16384])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes_of_zero_tiny_huge_and_nonfinite_rows(moe, K, dtype):
    x = torch.randn((12, K), generator=_gen(K))
    x[1] = 0.0
    x[2] *= 1e-40
    x[3] *= 1e-38
    x[4] = x[4].clamp(-3, 3) * 1e38
    x[5, K - 1] = float("nan")
    x[6, 0] = float("inf")
    x[7, K // 2] = -float("inf")
    x[8] = float("nan")
    x[9] = -0.0
    x[10] = 0.0
    x[10, 3] = 1e-45
    _check_codes(moe, x.to(dtype))


def test_codes_write_their_rows_only(moe):
    x = torch.randn((6, 96), generator=_gen(1)).cuda()
    q = torch.full((10, 96), 9, dtype=I8, device="cuda")
    s = torch.full((10,), 9.0, device="cuda")
    moe.quantize_rows(x, q=q[2:8], scale=s[2:8])
    torch.cuda.synchronize()
    assert (q[:2] == 9).all() and (q[8:] == 9).all() and (s[:2] == 9).all() and (s[8:] == 9).all()
    rq, rs = codes64(x)
    assert torch.equal(q[2:8].cpu(), rq) and torch.equal(s[2:8].cpu(), rs)
    a, b = moe.quantize_rows(x[:0])
    assert a.shape == (0, 96) and b.shape == (0,)


# ---- the product -----------------------------------------------------------------------

def _inputs(T, K, N, act, seed, bias=True, res=None):
    g = _gen(seed)
    R = rows_of(act, N)
    x = torch.randn((T, K), generator=g) * torch.exp(0.5 * torch.randn((K,), generator=g))
    w, sw = codes64(torch.randn((R, K), generator=g) / K ** 0.5)
    b = torch.randn((R,), generator=g) if bias else None
    r = torch.randn((T, N), generator=g).to(res) if res is not None else None
    return x, w, sw, b, r


def _c(t):
    return None if t is None else t.cuda()


# T around the switch from few tokens to tiles, from 16 to 32 to 64 tokens, and from coding in the product's launch to
# one before it; K below, off and on the step of 64 values, and of 128; N below, off and over 8, 16 and the tile
SHAPES = [(1, 32, 1), (1, 2048, 40), (2, 96, 7), (3, 512, 130), (16, 544, 33), (16, 1024, 9), (5, 4096, 24), (17, 64, 16),
          (33, 160, 19), (32, 512, 11), (33, 512, 18), (64, 256, 10), (64, 320, 200), (65, 32, 1), (65, 1024, 72), (127, 96, 129), (129, 64, 3), (200, 224, 257),
          (384, 128, 260)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "swiglu"])
def test_linear_q8(moe, T, K, N, act):
    for i, (xt, yt, res, bias) in enumerate([(BF16, BF16, None, True), (BF16, F32, F32, False), (F32, F32, BF16, True),
                                             (I8, BF16, BF16, True), (I8, F32, None, False)]):
        x, w, sw, b, r = _inputs(T, K, N, act, seed=T + K + N + i, bias=bias, res=res)
        if xt != I8:
            x = x.to(xt)
        qx, sx = codes64(x)
        y = moe.linear_q8(qx.cuda() if xt == I8 else x.cuda(), w.cuda(), sw.cuda(), x_scale=sx.cuda() if xt == I8 else None,
                          bias=_c(b), act=act, residual=_c(r), y_dtype=yt)
        assert y.dtype == yt
        ref, _ = q8_64(qx, sx, w, sw, b, act, r)
        within(y, ref, q8_bound(qx, sx, w, sw, b, act, r, yt), f"{xt} {yt}")


# each form of the plan: tile, whether the reduction is cut
FORMS = [(65, 96, 33, "none", 64, False), (65, 8224, 33, "none", 64, True), (2050, 96, 1003, "none", 128, False),
         (1025, 16352, 201, "none", 128, True), (2050, 2080, 4094, "none", 256, False),
         (2050, 16352, 1003, "none", 256, True), (65, 96, 33, "swiglu", 64, False), (65, 8224, 33, "swiglu", 64, True),
         (1025, 96, 1003, "swiglu", 128, False), (65, 16352, 515, "swiglu", 128, True),
         (1025, 2080, 4094, "swiglu", 256, False), (1025, 16352, 1003, "swiglu", 256, True)]


@pytest.mark.parametrize("T,K,N,act,tile,cut", FORMS)
def test_forms_are_exact(moe, T, K, N, act, tile, cut):
    """Codes of any size with scales of 1: sums below 2^24 come back as they are.  SwiGLU's gate rows are those of a
    large constant, so that its silu is the gate itself; both factors are powers of two or small."""
    form = moe.linear_q8_form(T, K, N, act, I8)
    assert form["tile"] == tile and (form["parts"] > 1) == cut, form
    g = torch.Generator(device="cuda").manual_seed(T + K)
    x = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=I8)
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda", dtype=I8)
    one = torch.ones((T,), device="cuda")
    exact = (x.double() @ w.double().t())
    assert exact.abs().max() < 1 << 24
    if act == "swiglu":
        gate = torch.zeros_like(w)
        bias = torch.zeros((2 * N,), device="cuda")
        bias[:N] = 128.0  # silu(128) is 128 in fp32
        y = moe.linear_q8(x, torch.cat([gate, w]), torch.ones((2 * N,), device="cuda"), x_scale=one, bias=bias, act=act,
                          y_dtype=F32)
        assert torch.equal(y.double(), exact * 128.0)
        # and the gate's own rows: an up value of 1, gates so large that silu is the identity, or 0 below
        bias = torch.zeros((2 * N,), device="cuda")
        bias[N:] = 1.0
        y = moe.linear_q8(x, torch.cat([w, gate]), torch.full((2 * N,), 2.0 ** 10, device="cuda"), x_scale=one, bias=bias,
                          act=act, y_dtype=F32)
        assert torch.equal(y.double(), exact.clamp(min=0) * 2.0 ** 10)
    else:
        y = moe.linear_q8(x, w, torch.ones((N,), device="cuda"), x_scale=one, y_dtype=F32)
        assert torch.equal(y.double(), exact)


@pytest.mark.parametrize("T", [1, 16, 64, 65, 300])
def test_largest_sums(moe, T):
    """16,384 products of -128 * -128, the largest that a sum can be: 2^28, and 2^28 - 2^14 + 127 * 128 beside it."""
    K, N = 16384, 20
    x = torch.full((T, K), -128, dtype=I8, device="cuda")
    w = torch.full((N, K), -128, dtype=I8, device="cuda")
    w[1, 5] = 127
    one = torch.ones((T,), device="cuda")
    y = moe.linear_q8(x, w, torch.ones((N,), device="cuda"), x_scale=one, y_dtype=F32)
    want = torch.full((T, N), 2.0 ** 28)
    want[:, 1] = torch.tensor(float(2 ** 28 - 2 ** 14 - 127 * 128)).float()
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("T", [3, 40, 100])
def test_scales_far_apart(moe, T):
    """Scales whose product alone leaves fp32's range on either side, while the result does not."""
    K, N = 64, 40
    x, w, sw, _, _ = _inputs(T, K, N, "none", seed=T)
    qx, sx = codes64(x)
    for a, b in [(1e-30, 1e-12), (1e30, 1e-30), (1e-36, 1e33), (1e20, 1e10), (2.0 ** -126, 2.0 ** 100)]:
        s, t = torch.full((T,), a), torch.full((N,), b)
        for p, q in ((s, t), (t.new_full((T,), b), s.new_full((N,), a))):
            y = moe.linear_q8(qx.cuda(), w.cuda(), q.cuda(), x_scale=p.cuda(), y_dtype=F32)
            ref, _ = q8_64(qx, p, w, q, None, "none", None)
            # (results below the normal range are off by its last place)
            within(y, ref, 4 * 2.0 ** -24 * ref.abs() + 2.0 ** -149, f"{a} {b}")


@pytest.mark.parametrize("T", [3, 40, 100])
def test_scales_of_either_sign_and_below_the_normal_range(moe, T):
    """Scales that a caller made: negative ones, the large ones among them, whose product with a sum passes fp32's range while the
    result does not; and one below 2^-126, of which fp32 holds multiples of 2^-149, exact beside sums this small."""
    K, N = 64, 40
    x, w, sw, _, _ = _inputs(T, K, N, "none", seed=T)
    qx, sx = codes64(x)
    for a, b in [(-1e36, 1e-30), (1e36, -1e-30), (-1e36, -1e-30), (-2.0, 0.5), (2.0 ** -140, 2.0 ** 100), (-2.0 ** -140, 2.0 ** 100)]:
        s, t = torch.full((T,), a), torch.full((N,), b)
        for p, q in ((s, t), (t.new_full((T,), b), s.new_full((N,), a))):
            y = moe.linear_q8(qx.cuda(), w.cuda(), q.cuda(), x_scale=p.cuda(), y_dtype=F32)
            ref, _ = q8_64(qx, p, w, q, None, "none", None)
            within(y, ref, 4 * 2.0 ** -24 * ref.abs(), f"{a} {b}")


@pytest.mark.parametrize("T", [6, 48, 150])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_a_nonfinite_row_stays_in_its_row(moe, T, xt):
    x, w, sw, b, _ = _inputs(T, 96, 40, "silu", seed=4)
    x = x.to(xt)
    clean = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="silu")
    x[1, 3], x[T - 1, 90] = float("nan"), float("inf")
    y = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="silu")
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(y[keep], clean[keep])
    assert y[1].isnan().all() and y[T - 1].isnan().all()


@pytest.mark.parametrize("xt", [F32, BF16])
def test_a_token_gives_the_same_in_every_batch(moe, xt):
    """One token, a few, and a tiled batch: the codes are the same and the sums exact, so the results are too."""
    x, w, sw, b, _ = _inputs(300, 2080, 72, "gelu", seed=9)
    x = x.to(xt)
    whole = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="gelu", y_dtype=F32)
    q, s = moe.quantize_rows(x.cuda())
    for n in (1, 7, 16, 17, 40, 64, 65, 299):
        part = moe.linear_q8(x[:n].cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="gelu", y_dtype=F32)
        assert torch.equal(part, whole[:n]), n
        part = moe.linear_q8(q[:n], w.cuda(), sw.cuda(), x_scale=s[:n], bias=b.cuda(), act="gelu", y_dtype=F32)
        assert torch.equal(part, whole[:n]), n


def test_zero_rows_give_the_bias(moe):
    for T in (4, 100):
        x, w, sw, b, r = _inputs(T, 64, 24, "none", seed=2, res=F32)
        x[1] = 0.0
        y = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), residual=r.cuda(), y_dtype=F32)
        assert torch.equal(y[1].cpu(), b + r[1])


def test_residual_in_place(moe):
    for T in (5, 40, 90):
        x, w, sw, b, r = _inputs(T, 128, 68, "gelu", seed=T, res=F32)
        r = r.cuda()
        want = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="gelu", residual=r, y_dtype=F32)
        got = moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), act="gelu", residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("T", [7, 50, 150])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_views_off_alignment_and_nothing_past_the_end(moe, T, act):
    """Scales, bias, residual and y that start at odd elements: the same values, and the elements around y untouched."""
    K, N = 96, 36
    x, w, sw, b, r = _inputs(T, K, N, act, seed=T, res=BF16)

    def odd(t):
        big = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device="cuda")
        big[1:-1] = t.reshape(-1).cuda()
        return big, big[1:-1].view(t.shape)

    (_, vs), (_, vb), (_, vr) = odd(sw), odd(b), odd(r)
    by, vy = odd(torch.zeros((T, N), dtype=BF16))
    q, s = moe.quantize_rows(x.cuda())
    _, vx = odd(s.cpu())
    moe.linear_q8(q, w.cuda(), vs, x_scale=vx, bias=vb, act=act, residual=vr, y=vy)
    y = moe.linear_q8(q, w.cuda(), sw.cuda(), x_scale=s, bias=b.cuda(), act=act, residual=r.cuda())
    assert torch.equal(vy, y) and by[0] == 7 and by[-1] == 7


def test_no_rows(moe):
    x, w, sw, b, _ = _inputs(0, 64, 12, "none", seed=0)
    assert moe.linear_q8(x.cuda(), w.cuda(), sw.cuda(), bias=b.cuda()).shape == (0, 12)


def test_streams_and_graph(moe):
    """Calls on a stream of their own and replays of a captured one give what an eager call does."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, K, N, act in [(1, 2048, 512, "swiglu"), (40, 512, 200, "none"), (100, 8224, 33, "gelu")]:
        R = rows_of(act, N)
        x = torch.randn((T, K), generator=g, device="cuda").to(BF16)
        w, sw = moe.quantize_rows(torch.randn((R, K), generator=g, device="cuda") / K ** 0.5)
        want = moe.linear_q8(x, w, sw, act=act)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        y1 = moe.linear_q8(x, w, sw, act=act, stream=s)
        s.synchronize()
        assert torch.equal(y1, want)
        y = torch.zeros_like(want)
        ws = torch.empty(max(1, moe.linear_q8_workspace_bytes(T, K, N, act)), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.linear_q8(x, w, sw, act=act, y=y, ws=ws)
        for k in range(3):
            fresh = torch.randn((T, K), generator=g, device="cuda").to(BF16)
            x.copy_(fresh)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, moe.linear_q8(x, w, sw, act=act)), (T, k)
            torch.cuda.synchronize()
