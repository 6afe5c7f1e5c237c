"""GPU: the training operators on tensors of more than 2^31 elements (offsets past 32 bits, signed and in bytes).

Operands are small whole numbers, of which every product and sum is exact in fp32 (below 2^24), so results are compared
for equality, by blocks of rows; the reference products are float64.  Only the balance loss has rounded values: its lse is
held to the bound that the balance tests derive.
"""
import pytest
import torch

from tests._train_ref import U

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _whole(shape, seed, most=2, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for rows in out.split(1 << 18):  # (int64 draws of a whole tensor would take four times its size)
        rows.copy_(torch.randint(-most, most + 1, rows.shape, generator=g, device="cuda", dtype=torch.int8))
    return out


def _blocks(T, size=1 << 16):
    """Blocks of rows: the first, the two around 2^31 elements' half way, and the last."""
    return [slice(0, size), slice(T // 2, T // 2 + size), slice(T - size, T)]


T = 1 << 20


def test_linear_long_input(moe):
    K, N = 2080, 24  # x: 2.18e9 elements
    x, w = _whole((T, K), 1), _whole((N, K), 2)
    assert x.numel() > 1 << 31
    bias = torch.arange(N, device="cuda", dtype=F32)
    y = moe.linear(x, w, bias=bias, y_dtype=F32)
    for b in _blocks(T):
        assert torch.equal(y[b].double(), x[b].double() @ w.double().t() + bias.double())
    dy = _whole((T, N), 3)
    dx, dw, db = moe.linear_backward(dy, x, w)
    for b in _blocks(T):  # sums below 24 * 4 = 96: exact in bf16
        assert torch.equal(dx[b].double(), dy[b].double() @ w.double())
    ref = torch.zeros((N, K), dtype=torch.float64, device="cuda")
    for i in range(0, T, 1 << 16):
        ref += dy[i:i + (1 << 16)].double().t().contiguous() @ x[i:i + (1 << 16)].double()
    assert torch.equal(dw.double(), ref)  # sums below 4 * 2^20
    assert torch.equal(db.double(), dy.double().sum(0))


def test_linear_long_output(moe):
    K, N = 64, 2057  # y: 2.16e9 elements, rows of odd length
    x, w = _whole((T, K), 4, most=1), _whole((N, K), 5, most=1)
    y = moe.linear(x, w)
    assert y.numel() > 1 << 31
    for b in _blocks(T):  # sums of at most 64: exact in bf16
        assert torch.equal(y[b].double(), x[b].double() @ w.double().t())
    dx, dw, db = moe.linear_backward(y, x, w, dx_dtype=F32)
    for b in _blocks(T):  # sums of at most 2057 * 64
        assert torch.equal(dx[b].double(), y[b].double() @ w.double())
    ref, sums = torch.zeros((N, K), dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(sums)
    for i in range(0, T, 1 << 16):
        d = y[i:i + (1 << 16)].double()
        ref += d.t().contiguous() @ x[i:i + (1 << 16)].double()
        sums += d.sum(0)
        size += d.abs().sum(0)
    assert size.max() < 1 << 24  # the magnitudes under every sum of dw (|x| <= 1) and db: each partial sum is exact
    assert torch.equal(dw.double(), ref)
    assert torch.equal(db.double(), sums)


def test_combine_backward_long(moe):
    n, k, H = (1 << 17) + 3, 16, 1032  # y: 2.16e9 elements
    y, dout = _whole((n * k, H), 6).view(n, k, H), _whole((n, H), 7)
    w = _whole((n, k), 8, dtype=F32)
    assert y.numel() > 1 << 31
    dw, dy = moe.combine_backward(y, w, dout)
    for b in _blocks(n, 1 << 12):
        assert torch.equal(dw[b], (y[b].float() * dout[b].float()[:, None]).sum(2))
        assert torch.equal(dy[b].float(), w[b][:, :, None] * dout[b].float()[:, None])


def test_balance_long(moe):
    n, E, k = (1 << 22) + 5, 516, 2  # logits: 2.16e9 elements
    logits = _whole((n, E), 9, most=4, dtype=F32)
    assert logits.numel() > 1 << 31
    t = torch.arange(n, device="cuda")
    ids = torch.stack([t % E, (t + 7) % E], 1).to(torch.int32)
    loss, counts, lse = moe.balance_loss(logits, ids)
    assert int(counts[E]) == n
    assert torch.equal(counts[:E].long(), torch.bincount(ids.flatten().long(), minlength=E))
    w = torch.full((n, k), 0.5, device="cuda")
    dw = _whole((n, k), 10, dtype=F32)
    d = moe.route_backward(logits, ids, w=w, dw=dw, lse=lse, counts=counts, dloss=torch.zeros(2, device="cuda"))
    for b in _blocks(n):
        ref = torch.logsumexp(logits[b].double(), 1)
        assert (lse[b].double() - ref).abs().max() <= (60 + E + 32) * U + 4 * U * (11 + 4 + 8)
        # w (dw - sum w dw) with halves and small whole numbers: exact, and a loss part of zero
        gate = 0.5 * (dw[b] - 0.5 * dw[b].sum(1, keepdim=True))
        want = torch.zeros_like(logits[b]).scatter_(1, ids[b].long(), gate)
        assert torch.equal(d[b], want)
    alone = moe.route_backward(logits, ids, lse=lse, counts=counts, dloss=torch.tensor([1.0, 0.0], device="cuda"))
    p = torch.softmax(logits[-1000:].double(), 1)
    c = counts[:E].double()
    s = (p * c).sum(1, keepdim=True)
    ref = p * (E / (n * n * k) * (c - s))
    # p's relative error and the sum's, on both parts of the difference
    bound = p * (E / (n * n * k)) * (2 * (60 + E + 32) * U + 2 * E * U) * (c + 2 * s) + 1e-37
    assert ((alone[-1000:].double() - ref).abs() <= bound).all()
