"""GPU: balance loss and logits' gradient from tensors that start off the 16-byte boundaries of the vector path, under the
bounds that test_gpu_balance.py derives; and the losses of logits of hundreds."""
import pytest
import torch

import tests.test_gpu_balance as base
from tests._train_ref import TINY, U, gamma, loss64, within
from tests.test_gpu_balance import CASES, moe  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _off(t):
    """A view one element behind the start of its memory."""
    if t is None:
        return None
    big = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    view = big[1:].view(t.shape)
    view.copy_(t)
    assert view.is_contiguous() and view.data_ptr() % 16 == t.element_size()
    return view


@pytest.mark.parametrize("T,E,k", CASES + [(130, 64, 4), (300, 512, 10)])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_views_off_alignment(moe, monkeypatch, T, E, k, masked):  # noqa: F811
    monkeypatch.setattr(base, "_cuda", lambda *ts: [_off(t) for t in ts])
    base._check(moe, *base._inputs(T, E, k, seed=T * 7 + E, masked=masked))


def test_losses_of_wide_logits(moe):  # noqa: F811
    """Logits between about 600 and 1,400.  l - m is rounded, but beyond 120 below the maximum the exponential is 0, so p is
    off by at most 120 u, a few u and E u of its sum; a p that became 0 was below e^-103.  lse is off by the rounding of m and
    of one logarithm and sum, 8 u of it."""
    T, E, k = 80, 40, 3
    logits, ids, _, _, _ = base._inputs(T, E, k, seed=4)
    logits = logits * 100 + 1000
    loss, counts, lse = moe.balance_loss(logits.cuda(), ids.cuda())
    ref, ref_counts, ref_lse, _ = loss64(logits, ids, None)
    assert torch.equal(counts.cpu().long(), ref_counts)
    within(lse, ref_lse, 8 * U * ref_lse.abs(), "lse")
    perr = (120 + E + 32) * U
    b0 = (perr + gamma(T + 64)) * ref[0] + E * E * 1e-44
    b1 = (2 * 8 * U + gamma(T + 64)) * ref[1]
    within(loss, ref, torch.stack([b0, b1]) + TINY, "loss")
