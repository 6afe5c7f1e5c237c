"""GPU: balance loss, counts and the gradient of the logits against their definitions in 64 bits.

Tolerances.  p = e^(l - m) / s: the difference l - m is rounded (u |l - m|, at most 60 u here), the exponential adds
a few u, s is a sum of E positive terms: relative error of p at most PERR = (60 + E + 32) u.  Sums of p over rows,
counts and experts add gamma of their length; the bounds below carry those terms with the magnitudes they act on.
"""
import math

import pytest
import torch

from tests._train_ref import TINY, U, gamma, loss64, route_grad64, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_routed_ffn_amd as m
    return m


def _inputs(T, E, k, seed, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) * 2
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(max(T, 1))])[:T].to(torch.int32)
    w = torch.softmax(torch.randn((T, k), generator=g), 1)
    dw = torch.randn((T, k), generator=g)
    mask = torch.rand((T,), generator=g) >= masked if masked else None
    return logits, ids, w, dw, mask


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check(moe, logits, ids, w, dw, mask, gate=True, loss_part=True):
    T, E = logits.shape
    k = ids.shape[1]
    dloss = torch.tensor([0.7, -0.3])
    dl, di, dw_, ddw, dm, dd = _cuda(logits, ids, w, dw, mask, dloss)
    loss, counts, lse = moe.balance_loss(dl, di, mask=dm)
    d = moe.route_backward(dl, di, w=dw_ if gate else None, dw=ddw if gate else None,
                           lse=lse if loss_part else None, counts=counts if loss_part else None,
                           dloss=dd if loss_part else None)
    torch.cuda.synchronize()
    rl, rc, rs, takes = loss64(logits, ids, mask)
    assert torch.equal(counts.cpu().long(), rc)
    assert torch.equal(lse.cpu() == -math.inf, ~takes)
    n = int(rc[E])
    perr = (60 + E + 32) * U
    # lse = m + log s: s within perr, the logarithm and the sum round once each
    within(lse.cpu()[takes], rs[takes], perr + 4 * U * (rs[takes].abs() + logits[takes].abs().amax(1) + 8), "lse")
    b0 = (perr + gamma(T + 64)) * rl[0].abs()
    b1 = (2 * perr + 8 * U) * (rs[takes].abs() + 8).mean() + gamma(T + 64) * rl[1] if n else 0.0
    if n:
        b1 = b1 + 2 * (perr + 4 * U * (logits[takes].abs().max() + 8)) * (rs[takes].abs() + 8).max()
    within(loss, rl, torch.tensor([float(b0), float(b1)]) + TINY, "loss")
    on = takes if loss_part else torch.ones(T, dtype=torch.bool)
    ref = route_grad64(logits, ids, w if gate else None, dw, on, rc, rs, dloss if loss_part else None)
    bound = torch.zeros((T, E), dtype=torch.float64)
    if loss_part and n:
        p = torch.softmax(logits[takes].double(), 1)
        c = rc[:E].double()
        A = abs(float(dloss[0])) * E / (n * n * k)
        Z = 2 * abs(float(dloss[1])) / n
        s = (p * c).sum(1, keepdim=True)
        z = rs[takes].abs()[:, None]
        bound[takes] += p * (A * (2 * perr + gamma(E + 16)) * (c + 2 * s) + Z * ((perr + 16 * U) * (z + 8) + perr * z))
    if gate:
        a = (w.double() * dw.double().abs()).sum(1, keepdim=True)
        part = w.double() * ((gamma(k + 8) + 4 * U) * (a + dw.double().abs()))
        for j in range(k):
            for t in range(T):
                e = int(ids[t, j])
                if 0 <= e < E:
                    bound[t, e] += 2 * part[t, j]
    within(d, ref, bound + 4 * U * ref.abs() + TINY, "dlogits")
    return loss, counts, lse, d


# (T, E, k): one token; the smallest router; E on each side of a lane's share and of the vector path (E % 4); the last
# size of one workgroup and the first of several; the largest E and k
CASES = [(1, 8, 2), (3, 1, 1), (4, 7, 7), (12, 512, 10), (64, 60, 6), (65, 61, 6), (100, 256, 8), (130, 257, 5),
         (300, 513, 16), (257, 1024, 16), (40, 1023, 3)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_loss_and_gradient(moe, T, E, k, masked):
    _check(moe, *_inputs(T, E, k, seed=T * 7 + E, masked=masked))


@pytest.mark.parametrize("gate,loss_part", [(True, False), (False, True)])
def test_one_part_only(moe, gate, loss_part):
    _check(moe, *_inputs(70, 96, 4, seed=5, masked=0.3), gate=gate, loss_part=loss_part)


def test_no_token_takes_part(moe):
    logits, ids, w, dw, _ = _inputs(9, 16, 3, seed=1)
    loss, counts, lse, d = _check(moe, logits, ids, w, dw, torch.zeros(9, dtype=torch.bool))
    assert not loss.any() and not counts.any() and not d.any()
    loss, counts, lse, d = _check(moe, torch.full((200, 16), -math.inf), _inputs(200, 16, 3, 2)[1],
                                  *_inputs(200, 16, 3, 2)[2:4], None)
    assert not loss.any() and not counts.any() and not d.any()


def test_no_rows(moe):
    dev = torch.device("cuda")
    loss, counts, lse = moe.balance_loss(torch.empty((0, 16), device=dev), torch.empty((0, 3), dtype=torch.int32, device=dev))
    assert loss.tolist() == [0.0, 0.0] and not counts.any() and lse.numel() == 0
    d = moe.route_backward(torch.empty((0, 16), device=dev), torch.empty((0, 3), dtype=torch.int32, device=dev), lse=lse,
                           counts=counts, dloss=torch.zeros(2, device=dev))
    assert d.shape == (0, 16)


def test_masked_rows_may_hold_anything(moe):
    """NaN, infinities and wild ids in rows that the mask leaves out change nothing; -inf and the lowest value within
    rows that count have probability 0."""
    logits, ids, w, dw, mask = _inputs(150, 48, 4, seed=9, masked=0.5)
    logits[::7, 5] = -math.inf
    logits[::5, 9] = torch.finfo(torch.float32).min
    out = ~mask
    logits[out] = float("nan")
    logits[out.nonzero()[:5, 0]] = math.inf
    ids[out] = 1 << 30
    w[out] = float("nan")
    dw[out] = math.inf
    clean = [t.clone() for t in (logits, ids, w, dw)]
    clean[0][out], clean[1][out], clean[2][out], clean[3][out] = 0.0, 0, 0.0, 0.0
    a = [t.cpu() for t in _run(moe, logits, ids, w, dw, mask)]
    b = [t.cpu() for t in _run(moe, *clean, mask)]
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    _check(moe, *clean, mask)


def _run(moe, logits, ids, w, dw, mask):
    l, i, w, dw, m = _cuda(logits, ids, w, dw, mask)
    loss, counts, lse = moe.balance_loss(l, i, mask=m)
    d = moe.route_backward(l, i, w=w, dw=dw, lse=lse, counts=counts, dloss=torch.tensor([1.0, 0.1], device="cuda"))
    return loss, counts, lse, d


def test_nan_in_a_counted_row_shows(moe):
    logits, ids, w, dw, _ = _inputs(70, 32, 2, seed=3)
    logits[11, 4] = float("nan")
    logits[12] = float("nan")
    loss, counts, lse, d = _run(moe, logits, ids, w, dw, None)
    assert loss.isnan().all() and int(counts[32]) == 70
    assert lse[11].isnan() and lse[12].isnan() and d[11].isnan().all() and d[12].isnan().all()
    rest = [t for t in range(70) if t not in (11, 12)]
    assert torch.isfinite(lse[rest]).all()


def test_wide_logits(moe):
    """Logits of hundreds: the exponentials span the whole range."""
    logits, ids, w, dw, _ = _inputs(80, 40, 3, seed=4)
    logits = logits * 100 + 1000
    perr_scale = 400.0  # |l - m| up to about 1000 but e^-120 and below is 0: 120 u against the 60 u allowed elsewhere
    loss, counts, lse, d = _run(moe, logits, ids, w, dw, None)
    rl, rc, rs, takes = loss64(logits, ids, None)
    within(lse, rs, 8 * U * rs.abs().max(), "lse")
    ref = route_grad64(logits, ids, w, dw, takes, rc, rs, torch.tensor([1.0, 0.1]))
    # 120 u on p; the losses' factors: A c <= 40 * 80 / (80^2 * 3), z <= 0.2 / 80 * lse
    size = 40 * 80 / (80 * 80 * 3) * 2 + 0.2 / 80 * rs.abs().max() + 2 * dw.abs().max()
    within(d, ref, (perr_scale + 40) * U * size, "dlogits")


def test_ids_out_of_range_and_twice(moe):
    logits, ids, w, dw, mask = _inputs(90, 24, 5, seed=8, masked=0.2)
    ids[3] = torch.tensor([4, 4, 4, 4, 4], dtype=torch.int32)
    ids[7] = torch.tensor([2, -1, 2, 24, 2], dtype=torch.int32)
    ids[20:30, 1] = -5
    mask[3] = mask[7] = True
    _check(moe, logits, ids, w, dw, mask)


def test_views_off_the_vector_path(moe):
    """Rows of a tensor that start off a 16-byte boundary give what the aligned copy gives, bit for bit."""
    logits, ids, w, dw, mask = _inputs(130, 64, 4, seed=6, masked=0.2)
    big = torch.empty(130 * 64 + 1, device="cuda")
    view = big[1:].view(130, 64)
    view.copy_(logits)
    i, w, dw, m = _cuda(ids, w, dw, mask)
    up = torch.tensor([1.0, 0.5], device="cuda")
    outs = []
    for l in (view, logits.cuda()):
        loss, counts, lse = moe.balance_loss(l, i, mask=m.to(torch.uint8))
        outs.append((loss, counts, lse, moe.route_backward(l, i, w=w, dw=dw, lse=lse, counts=counts, dloss=up)))
    rl, rc, rs, takes = loss64(logits, ids, mask)
    assert torch.equal(outs[0][1], outs[1][1])
    for o in outs:  # (the two column layouts add in different orders)
        ref = route_grad64(logits, ids, w.cpu(), dw.cpu(), takes, rc, rs, up.cpu())
        within(o[3], ref, 1e-5 * (ref.abs() + 1), "dlogits")


def test_repeatable_and_other_stream(moe):
    logits, ids, w, dw, mask = _inputs(1000, 100, 6, seed=12, masked=0.1)
    a = _run(moe, logits, ids, w, dw, mask)
    b = _run(moe, logits, ids, w, dw, mask)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    l, i, m = _cuda(logits, ids, mask)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, counts, lse = moe.balance_loss(l, i, mask=m, stream=s)
    s.synchronize()
    assert torch.equal(loss, a[0]) and torch.equal(counts, a[1]) and torch.equal(lse, a[2])


def test_nothing_written_past_the_outputs(moe):
    logits, ids, w, dw, _ = _inputs(77, 30, 3, seed=2)
    l, i, w, dw = _cuda(logits, ids, w, dw)
    out = torch.full((80, 30), 7.0, device="cuda")
    lse, counts = torch.full((90,), 7.0, device="cuda"), torch.full((40,), 7, dtype=torch.int32, device="cuda")
    loss = torch.full((4,), 7.0, device="cuda")
    moe.balance_loss(l, i, loss=loss[1:3], counts=counts[4:35], lse=lse[5:82])
    moe.route_backward(l, i, w=w, dw=dw, dlogits=out[2:79])
    torch.cuda.synchronize()
    assert (out[:2] == 7).all() and (out[79:] == 7).all()
    assert (lse[:5] == 7).all() and (lse[82:] == 7).all() and (counts[:4] == 7).all() and (counts[35:] == 7).all()
    assert loss[0] == 7 and loss[3] == 7
