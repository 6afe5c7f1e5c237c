"""GPU: the training operators together, as a training step of a layer with frozen low-bit experts uses them.

The step: router logits from a dense product with bias, top-k, quantized experts, a shared expert (SwiGLU, then down)
whose output is the combine's residual; loss = <out, target> + losses of the router.  The gradients of the router's
weights and bias, of the shared expert's weights and of its input are compared with 64-bit automatic differentiation
of the same step on the same expert outputs, and with central differences of that 64-bit step.
"""
import math

import pytest
import torch

import synth
from tests._parity import to_dev, to_dev_x

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _layer(moe, T):
    w = synth.Workload(f"train_step_{T}", E=16, k=4, H=256, I=128, T=T, bits=4, x_dtype="bf16", zipf_s=0.8)
    layer = moe.ExpertLayer(w.E, w.H, w.I, w.bits, to_dev(w.experts()))
    g = torch.Generator().manual_seed(T)
    p = {"wr": (torch.randn((w.E, w.H), generator=g) / 16).to(BF16), "br": torch.randn((w.E,), generator=g) / 4,
         "w1": (torch.randn((2 * w.I, w.H), generator=g) / 16).to(BF16),
         "w2": (torch.randn((w.H, w.I), generator=g) / 11).to(BF16)}
    p = {n: t.cuda() for n, t in p.items()}
    x = to_dev_x(w.x())
    target = (torch.randn((T, w.H), generator=g) / T).cuda()
    mask = (torch.rand((T,), generator=g) > 0.1).cuda()
    return w, layer, p, x, target, mask


def _step(moe, w, layer, p, x, target, mask, dloss, ws=None):
    """One forward and backward pass; every tensor that it makes."""
    logits = moe.linear(x, p["wr"], bias=p["br"], y_dtype=F32)
    pre = torch.empty((w.T, 2 * w.I), dtype=BF16, device=x.device)
    h = moe.linear(x, p["w1"], act="swiglu", pre=pre)
    shared = moe.linear(h, p["w2"], y_dtype=F32)
    ids, gate, d, y, out = moe.layer_forward(layer, x, logits, w.k, residual=shared, path="mfma")
    loss, counts, lse = moe.balance_loss(logits, ids, mask=mask)
    dout = target
    dgate, dy = moe.combine_backward(y, gate, dout)
    dlogits = moe.route_backward(logits, ids, w=gate, dw=dgate, lse=lse, counts=counts, dloss=dloss)
    dx_r, dwr, dbr = moe.linear_backward(dlogits, x, p["wr"], dx_dtype=F32)
    dh, dw2, _ = moe.linear_backward(dout, h, p["w2"], need=("dx", "dw"), dx_dtype=BF16)
    dx_s, dw1, _ = moe.linear_backward(dh, x, p["w1"], act="swiglu", pre=pre, need=("dx", "dw"), dx_dtype=F32)
    return dict(logits=logits, ids=ids, gate=gate, y=y, out=out, loss=loss, counts=counts, dlogits=dlogits, dwr=dwr, dbr=dbr,
                dw1=dw1, dw2=dw2, dx_r=dx_r, dx_s=dx_s, dy=dy)


def _step64(wr, br, w1, w2, x, held, ids, y, target, mask, dloss):
    """The scalar that the step differentiates, in 64 bits, with the routing and the expert outputs held, and the gate
    weights of rows that the mask leaves out held at `held`: those rows give the router no gradient."""
    logits = x @ wr.t() + br
    gate = torch.where(mask[:, None], torch.softmax(torch.gather(logits, 1, ids), 1), held)
    g, u = (x @ w1.t()).chunk(2, 1)
    out = (g * torch.sigmoid(g) * u) @ w2.t() + (gate[:, :, None] * y).sum(1)
    E, k = wr.shape[0], ids.shape[1]
    n = mask.sum()
    counts = torch.zeros(E, dtype=torch.float64).index_add_(0, ids[mask].reshape(-1),
                                                            torch.ones(int(n) * k, dtype=torch.float64))
    p = torch.softmax(logits[mask], 1)
    bal = E / (n * n * k) * (counts * p.sum(0)).sum()
    z = (torch.logsumexp(logits[mask], 1) ** 2).mean()
    return (out * target).sum() + dloss[0] * bal + dloss[1] * z


@pytest.mark.parametrize("T", [40, 300])
def test_training_step_gradients(moe, T):
    w, layer, p, x, target, mask = _layer(moe, T)
    dloss = torch.tensor([0.5, 0.05], device="cuda")
    r = _step(moe, w, layer, p, x, target, mask, dloss)
    torch.cuda.synchronize()
    leaves = [p[n].cpu().double().requires_grad_() for n in ("wr", "br", "w1", "w2")]
    held = r["gate"].cpu().double()
    fixed = (r["ids"].cpu().long(), r["y"].cpu().double(), target.cpu().double(), mask.cpu(), dloss.cpu().double())
    xd = x.cpu().double().requires_grad_()
    total = _step64(*leaves, xd, held, *fixed)
    grads = torch.autograd.grad(total, leaves + [xd])
    # Each gradient is a product of operands of which at most three were rounded to bf16 on the way (h, dh, dz, pre:
    # 2^-8 each at most, on independent elements), so a relative distance of 4 * 2^-8 in the 2-norm bounds it; the
    # router's chain is fp32 throughout except x and the fp16 products inside y, which are held.
    for name, got, ref, tol in [("dwr", r["dwr"], grads[0], 1e-4), ("dbr", r["dbr"], grads[1], 1e-4),
                                ("dw1", r["dw1"], grads[2], 4 * 2.0 ** -8), ("dw2", r["dw2"], grads[3], 4 * 2.0 ** -8),
                                ("dx", r["dx_r"] + r["dx_s"], grads[4], 4 * 2.0 ** -8)]:
        d = (got.cpu().double() - ref).norm() / ref.norm()
        assert d <= tol, (name, float(d))
    # differences of the 64-bit step along random directions
    g = torch.Generator().manual_seed(5)
    for i, (got, tol) in enumerate([(r["dwr"], 2e-4), (r["dbr"], 2e-4), (r["dw1"], 2.0 ** -5), (r["dw2"], 2.0 ** -5)]):
        v = got.cpu().double() / got.cpu().double().norm() + 0.1 * torch.randn(leaves[i].shape, generator=g,
                                                                               dtype=torch.float64) / leaves[i].numel() ** 0.5
        eps = 1e-4
        with torch.no_grad():
            up = [l + eps * v if j == i else l for j, l in enumerate(leaves)]
            dn = [l - eps * v if j == i else l for j, l in enumerate(leaves)]
            num = (_step64(*up, xd, held, *fixed) - _step64(*dn, xd, held, *fixed)) / (2 * eps)
        assert abs(float(num) - float((got.cpu().double() * v).sum())) <= tol * abs(float(num)), i


def test_training_step_graph_replays(moe):
    """The whole step captured once and replayed with eager work between the replays: the same bits every time."""
    w, layer, p, x, target, mask = _layer(moe, 300)
    dloss = torch.tensor([0.5, 0.05], device="cuda")
    eager = _step(moe, w, layer, p, x, target, mask, dloss)
    torch.cuda.synchronize()
    names = ("logits", "out", "loss", "counts", "dlogits", "dwr", "dbr", "dw1", "dw2", "dx_r", "dx_s", "dy")
    want = {n: eager[n].clone() for n in names}
    graphs = []
    for _ in range(2):  # two graphs, each with its own memory
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            made = _step(moe, w, layer, p, x, target, mask, dloss)
        graphs.append((g, made))
    torch.cuda.synchronize()
    for r in range(3):
        for g, made in graphs:
            for n in names:
                made[n].fill_(1)
            again = _step(moe, w, layer, p, x, target, mask, dloss)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for n in names:
                assert torch.equal(made[n], want[n]), (r, n)
                assert torch.equal(again[n], want[n]), (r, n)


def test_two_steps_at_once_on_two_streams(moe):
    w, layer, p, x, target, mask = _layer(moe, 300)
    dloss = torch.tensor([0.5, 0.05], device="cuda")
    want = _step(moe, w, layer, p, x, target, mask, dloss)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(_step(moe, w, layer, p, x, target, mask, dloss))
    torch.cuda.synchronize()
    for r in got:
        for n in ("loss", "counts", "dlogits", "dwr", "dw1", "dw2", "dx_s"):
            assert torch.equal(r[n], want[n]), n
