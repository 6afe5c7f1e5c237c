"""GPU: the dense weights' way from gradient to 8-bit serving, as a program goes it: linear and linear_backward of a shared
expert, the update made orthogonal with momentum, rows to 8 bits, and the products on them.  Each part is checked against
64 bits on what the part before it gave."""
import pytest
import torch

from tests._newton_ref import newton64, newton_bound
from tests._q8_ref import codes64, q8_64, q8_bound
from tests._train_ref import HALF, U, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
T, H, I = 150, 256, 96
LR = 0.02


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


class Shared:
    """A shared expert being trained: fp32 weights, their bf16 copies, and one momentum each."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn((T, H), generator=g).to(BF16).cuda()
        self.dout = torch.randn((T, H), generator=g).cuda()
        self.w = [(torch.randn(s, generator=g) / s[1] ** 0.5).cuda() for s in ((2 * I, H), (H, I))]
        self.low = [w.to(BF16) for w in self.w]
        self.momentum = [torch.zeros_like(w) for w in self.w]

    def step(self, moe, stream=None):
        """One step; the gradients and updates of both matrices."""
        up, down = self.low
        pre = torch.empty((T, 2 * I), dtype=BF16, device="cuda")
        h = moe.linear(self.x, up, act="swiglu", pre=pre, stream=stream)
        dh, d_down, _ = moe.linear_backward(self.dout, h, down, need=("dx", "dw"), stream=stream)
        _, d_up, _ = moe.linear_backward(dh, self.x, up, act="swiglu", pre=pre, need=("dw",), stream=stream)
        grads = (d_up, d_down)
        o = [moe.orthogonalize(g, momentum=m, stream=stream) for g, m in zip(grads, self.momentum)]
        for w, low, u in zip(self.w, self.low, o):
            w.add_(u, alpha=-LR * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
            low.copy_(w)
        return grads, o

    def serve(self, moe, n, stream=None):
        """The first n tokens through the 8-bit form, the residual x."""
        (qu, su), (qd, sd) = [moe.quantize_rows(w, stream=stream) for w in self.w]
        h = moe.linear_q8(self.x[:n], qu, su, act="swiglu", y_dtype=F32, stream=stream)
        y = moe.linear_q8(h, qd, sd, residual=self.x[:n], stream=stream)
        return (qu, su, qd, sd), h, y


def test_from_gradient_to_served_weights(moe):
    s = Shared(1)
    before = [torch.zeros_like(w) for w in s.w]
    for k in range(3):
        old = [w.clone() for w in s.w]
        grads, o = s.step(moe)
        for g, m, b, u, w, v in zip(grads, s.momentum, before, o, s.w, old):
            want = 0.95 * b.double() + 0.05 * g.double()
            assert ((m.double() - want).abs() <= 4 * U * (b.double().abs() + g.double().abs())).all()
            upd = (0.95 * m.double() + 0.05 * g.double()).cpu()
            ref = newton64(upd)
            off = (u.double().cpu() - ref).norm()
            assert off <= newton_bound(upd, BF16) * (1 + HALF[BF16]) + HALF[BF16] * ref.norm(), k
            step = -LR * max(1.0, w.shape[0] / w.shape[1]) ** 0.5 * u.double()
            assert ((w.double() - v.double() - step).abs() <= 4 * U * (v.double().abs() + step.abs())).all()
        before = [m.clone() for m in s.momentum]
    for n in (1, 12, 40, T):
        (qu, su, qd, sd), h, y = s.serve(moe, n)
        for q, sc, w in ((qu, su, s.w[0]), (qd, sd, s.w[1])):
            rq, rs = codes64(w)
            assert torch.equal(q.cpu(), rq) and torch.equal(sc.cpu(), rs)
        qx, sx = codes64(s.x[:n])
        ref, _ = q8_64(qx, sx, qu.cpu(), su.cpu(), None, "swiglu", None)
        within(h, ref, q8_bound(qx, sx, qu.cpu(), su.cpu(), None, "swiglu", None, F32), f"h {n}")
        qh, sh = codes64(h)
        x = s.x[:n].cpu()
        ref, _ = q8_64(qh, sh, qd.cpu(), sd.cpu(), None, "none", x)
        within(y, ref, q8_bound(qh, sh, qd.cpu(), sd.cpu(), None, "none", x, F32), f"y {n}")
        # and against the weights themselves: a code is off by half a scale, of the activations as of the weights
        hd, wd = h.double().cpu(), s.w[1].double().cpu()
        most = (0.5 * sh.double()[:, None] * wd.abs().sum(1) + hd.abs().sum(1, keepdim=True) * 0.5 * sd.double().cpu()
                + I * 0.25 * sh.double()[:, None] * sd.double().cpu())
        within(y, hd @ wd.t() + x.double(), most * (1 + 1e-6) + 1e-5, f"unquantised {n}")


def test_two_streams_at_once(moe):
    """Two experts trained and served on streams of their own give what each gives alone."""
    alone = [Shared(s) for s in (2, 3)]
    want = []
    for a in alone:
        for _ in range(2):
            a.step(moe)
        want.append(([w.clone() for w in a.w], a.serve(moe, T)[2]))
    torch.cuda.synchronize()
    both, streams = [Shared(s) for s in (2, 3)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(2):
        for b, s in zip(both, streams):
            with torch.cuda.stream(s):
                b.step(moe)
    for i, (b, s) in enumerate(zip(both, streams)):
        with torch.cuda.stream(s):
            got[i] = b.serve(moe, T)[2]
    torch.cuda.synchronize()
    for b, y, (w, v) in zip(both, got, want):
        assert all(torch.equal(x, z) for x, z in zip(b.w, w)) and torch.equal(y, v)


def test_captured_step(moe):
    """A step and the serving pass in one graph, replayed, against eager ones."""
    eager, held = Shared(4), Shared(4)
    held.step(moe)  # (first use outside the capture)
    eager.step(moe)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.step(moe)
        out = held.serve(moe, T)[2]
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        eager.step(moe)
        y = eager.serve(moe, T)[2]
        torch.cuda.synchronize()
        assert torch.equal(out, y), k
        for a, b in zip(held.w + held.momentum, eager.w + eager.momentum):
            assert torch.equal(a, b), k


# ---- more than 2^31 elements ----------------------------------------------------------

def test_far_rows_of_the_8_bit_calls(moe):
    rows, K, N = 1 << 20, 2080, 2112
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((rows, K), dtype=BF16, device="cuda")
    tail = torch.randn((70, K), generator=g, device="cuda").to(BF16)
    x[-70:] = tail
    assert x.numel() > 1 << 31 and rows * N > 1 << 31
    q, s = moe.quantize_rows(x)
    rq, rs = codes64(tail)
    assert torch.equal(q[-70:].cpu(), rq) and torch.equal(s[-70:].cpu(), rs)
    assert not q[:-70].any() and (s[:-70] == 2.0 ** -126).all()
    w, sw = moe.quantize_rows(torch.randn((N, K), generator=g, device="cuda") / K ** 0.5)
    want = moe.linear_q8(tail, w, sw)
    y = moe.linear_q8(q, w, sw, x_scale=s)
    assert torch.equal(y[-70:], want) and not y[:-70].any()
    del y, q
    y = moe.linear_q8(x, w, sw)
    assert torch.equal(y[-70:], want) and not y[:-70].any()


@pytest.mark.parametrize("B,R,K", [(2060, 1024, 1024), (540000, 63, 64)])
def test_far_matrices(moe, B, R, K):
    u = torch.zeros((B, R, K), dtype=BF16, device="cuda")
    assert u.numel() > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    u[-1] = torch.randn((R, K), generator=g, device="cuda").to(BF16)
    o = moe.orthogonalize(u)
    one = u[-1].float().cpu()
    ref = newton64(one)
    assert (o[-1].double().cpu() - ref).norm() <= newton_bound(one, BF16) * (1 + HALF[BF16]) + HALF[BF16] * ref.norm()
    assert not o[:-1].any()
