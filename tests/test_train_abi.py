"""Training entry points, without a GPU: bad arguments are refused on the host before anything is enqueued, sizes of
workspaces follow the sizes of the work, and the binding names what is wrong."""
import ctypes

import pytest
import torch

import expert_routed_ffn_amd as m
from expert_routed_ffn_amd import _lib

L = _lib.lib
P = ctypes.c_void_p(0x100000)    # never read: every call below is refused, or has no rows
ODD = ctypes.c_void_p(0x100002)
F32, BF16 = _lib.MOE_F32, _lib.MOE_BF16
OK, EINVAL, EUNSUP, EWS = _lib.MOE_OK, _lib.MOE_EINVAL, _lib.MOE_EUNSUPPORTED, _lib.MOE_EWORKSPACE


def _loss(logits=P, ids=P, mask=None, T=100, E=8, k=2, loss=P, counts=P, lse=P, ws=P, nb=1 << 24):
    return int(L.moe_balance_loss(logits, ids, mask, T, E, k, loss, counts, lse, ws, nb, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(E=0), EUNSUP), (dict(E=1025), EUNSUP), (dict(k=0), EUNSUP), (dict(k=9), EUNSUP),
    (dict(k=17, E=64), EUNSUP), (dict(T=(1 << 23) + 1), EUNSUP), (dict(loss=None), EINVAL), (dict(counts=None), EINVAL),
    (dict(logits=None), EINVAL), (dict(ids=None), EINVAL), (dict(lse=None), EINVAL), (dict(logits=ODD), EINVAL),
    (dict(ws=None), EWS), (dict(nb=0), EWS), (dict(T=0, counts=None), EINVAL)])
def test_balance_loss_refusals(kw, want):
    assert _loss(**kw) == want
    assert b"moe_balance_loss" in L.moe_last_error()


def _route(logits=P, ids=P, w=P, dw=P, lse=P, counts=P, dloss=P, T=4, E=8, k=2, out=P):
    return int(L.moe_route_backward(logits, ids, w, dw, lse, counts, dloss, T, E, k, out, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(E=2000), EUNSUP), (dict(k=9), EUNSUP), (dict(out=None), EINVAL), (dict(w=None), EINVAL),
    (dict(dw=None), EINVAL), (dict(lse=None), EINVAL), (dict(counts=None), EINVAL), (dict(dloss=None), EINVAL),
    (dict(w=None, dw=None, lse=None, counts=None, dloss=None), EINVAL), (dict(ids=None), EINVAL),
    (dict(logits=None), EINVAL), (dict(out=ODD), EINVAL), (dict(T=(1 << 23) + 1), EUNSUP)])
def test_route_backward_refusals(kw, want):
    assert _route(**kw) == want
    assert b"moe_route_backward" in L.moe_last_error()


def test_route_backward_no_rows():
    assert _route(T=0) == OK


def _combine(y=P, y_t=BF16, w=P, dout=P, d_t=F32, T=4, k=2, H=64, dw=P, dy=P):
    return int(L.moe_combine_backward(y, y_t, w, dout, d_t, T, k, H, dw, dy, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(H=66), EUNSUP), (dict(k=0), EUNSUP), (dict(k=17), EUNSUP),
    (dict(y_t=5), EINVAL), (dict(d_t=-1), EINVAL), (dict(dw=None, dy=None), EINVAL), (dict(dout=None), EINVAL),
    (dict(y=None), EINVAL), (dict(w=None), EINVAL), (dict(y=ODD), EINVAL), (dict(dout=ODD), EINVAL),
    (dict(dy=ODD), EINVAL), (dict(T=(1 << 23) + 1), EUNSUP)])
def test_combine_backward_refusals(kw, want):
    assert _combine(**kw) == want
    assert b"moe_combine_backward" in L.moe_last_error()


def test_combine_backward_no_rows():
    assert _combine(T=0) == OK


def _linear(x=P, x_t=BF16, w=P, bias=None, act=0, res=None, r_t=0, T=100, K=64, N=8, y=P, y_t=BF16, pre=None, ws=P,
            nb=1 << 30):
    return int(L.moe_linear(x, x_t, w, bias, act, res, r_t, T, K, N, y, y_t, pre, ws, nb, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EUNSUP), (dict(K=48), EUNSUP), (dict(K=0), EUNSUP),
    (dict(K=16416), EUNSUP), (dict(N=0), EUNSUP), (dict(N=16385), EUNSUP), (dict(act=4), EINVAL), (dict(act=-1), EINVAL),
    (dict(x_t=2), EINVAL), (dict(y_t=2), EINVAL), (dict(res=P, r_t=3), EINVAL), (dict(x=None), EINVAL),
    (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(x=ODD), EINVAL), (dict(w=ODD), EINVAL),
    (dict(ws=ODD), EINVAL), (dict(y=ODD, y_t=F32), EINVAL), (dict(bias=ODD), EINVAL),
    (dict(x_t=F32, y_t=F32, T=8192, K=4096, N=4096, ws=None), EWS),
    (dict(x_t=F32, y_t=F32, T=8192, K=4096, N=4096, nb=16), EWS)])
def test_linear_refusals(kw, want):
    assert _linear(**kw) == want
    assert b"moe_linear" in L.moe_last_error()


def test_linear_no_rows():
    assert _linear(T=0) == OK


def _back(dy=P, dy_t=BF16, pre=P, x=P, x_t=BF16, w=P, act=2, T=100, K=64, N=8, dx=P, dx_t=BF16, dw=P, dw_t=F32, db=P,
          ws=P, nb=1 << 30):
    return int(L.moe_linear_backward(dy, dy_t, pre, x, x_t, w, act, T, K, N, dx, dx_t, dw, dw_t, db, ws, nb, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EUNSUP), (dict(K=40), EUNSUP), (dict(N=0), EUNSUP), (dict(act=9), EINVAL),
    (dict(dy_t=2), EINVAL), (dict(x_t=2), EINVAL), (dict(dx_t=2), EINVAL), (dict(dw_t=2), EINVAL),
    (dict(dx=None, dw=None, db=None), EINVAL), (dict(dy=None), EINVAL), (dict(pre=None), EINVAL), (dict(x=None), EINVAL),
    (dict(w=None), EINVAL), (dict(dx=ODD), EINVAL), (dict(dw=ODD), EINVAL), (dict(x=ODD), EINVAL), (dict(w=ODD), EINVAL),
    (dict(ws=None), EWS), (dict(nb=0), EWS)])
def test_linear_backward_refusals(kw, want):
    assert _back(**kw) == want
    assert b"moe_linear_backward" in L.moe_last_error()


def test_linear_backward_no_rows_without_sums():
    assert _back(T=0, dw=None, db=None) == OK


def _at(mb):
    return ctypes.c_void_p(mb << 20)


def test_overlapping_buffers_are_refused():
    """Buffers at made-up addresses a MB apart (all needs here are far smaller); one of them moved onto another."""
    def check(fn, names, call):
        for a, b in names:
            places = {n: _at(16 + i) for i, n in enumerate("abcdefghij")}
            places[a] = ctypes.c_void_p(places[b].value + 16)
            assert int(call(places)) == EINVAL, (fn, a, b)
            assert b"overlap" in L.moe_last_error(), (fn, a, b)

    # logits, ids, w, dw, lse, counts, dloss, dlogits = a .. h
    check("route", [("h", "a"), ("h", "b"), ("h", "c"), ("h", "d"), ("h", "e"), ("h", "f")], lambda p: L.moe_route_backward(
        p["a"], p["b"], p["c"], p["d"], p["e"], p["f"], p["g"], 64, 16, 4, p["h"], None))
    # y, w, dout, dw, dy = a .. e
    check("combine", [("e", "a"), ("e", "c"), ("d", "a"), ("d", "c"), ("d", "e")], lambda p: L.moe_combine_backward(
        p["a"], F32, p["b"], p["c"], F32, 16, 4, 64, p["d"], p["e"], None) if p["a"].value % 16 == 0 else EINVAL)
    # x, w, bias, residual, y, pre, ws = a .. g
    check("linear", [("e", "a"), ("e", "b"), ("e", "d"), ("f", "a"), ("f", "d"), ("e", "f")], lambda p: L.moe_linear(
        p["a"], BF16, p["b"], p["c"], 2, p["d"], BF16, 16, 64, 32, p["e"], BF16, p["f"], p["g"], 0, None))
    # y on the residual is allowed only as the very buffer of the same type
    assert int(L.moe_linear(_at(16), BF16, _at(17), None, 0, _at(18), F32, 16, 64, 32, _at(18), BF16, None, None, 0,
                            None)) == EINVAL
    # dy, pre, x, w, dx, dw, db = a .. g
    check("backward", [("e", "a"), ("e", "b"), ("e", "c"), ("e", "d"), ("f", "a"), ("f", "c"), ("g", "a"), ("e", "f")],
          lambda p: L.moe_linear_backward(p["a"], BF16, p["b"], p["c"], BF16, p["d"], 2, 16, 64, 32, p["e"], BF16, p["f"],
                                          F32, p["g"], _at(64), 8 << 20, None))


def test_workspaces():
    assert int(L.moe_balance_loss_workspace_bytes(0, 512)) == 0
    assert int(L.moe_balance_loss_workspace_bytes(12, 512)) == 0
    assert int(L.moe_balance_loss_workspace_bytes(8192, 512)) > 0
    assert int(L.moe_balance_loss_workspace_bytes(8192, 5000)) == 0
    assert m.linear_workspace_bytes(3, 2048, 512, "swiglu") == 0
    # fp32 activations of a tiled product become bf16 terms: three for an fp32 result, one for a bf16 one
    one = m.linear_workspace_bytes(8192, 4096, 4096, "none", torch.float32, torch.bfloat16)
    three = m.linear_workspace_bytes(8192, 4096, 4096, "none", torch.float32, torch.float32)
    assert one == 8192 * 4096 * 2 and three == 3 * one
    every = m.linear_backward_workspace_bytes(333, 544, 201, "gelu")
    assert every > m.linear_backward_workspace_bytes(333, 544, 201, "gelu", need=("dw",)) > 0
    assert 0 < m.linear_backward_workspace_bytes(333, 544, 201, "gelu", need=("db",)) < every


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


BF = torch.bfloat16


@pytest.mark.parametrize("call,error,word", [
    (lambda: m.balance_loss(_t(4), _t(4, 2, dtype=torch.int32)), ValueError, "logits"),
    (lambda: m.balance_loss(_t(4, 8, dtype=BF), _t(4, 2, dtype=torch.int32)), TypeError, "logits"),
    (lambda: m.balance_loss(_t(8, 4).t(), _t(4, 2, dtype=torch.int32)), ValueError, "contiguous"),
    (lambda: m.balance_loss(_t(4, 8), _t(4, 2, dtype=torch.int32)), ValueError, "CUDA"),
    (lambda: m.route_backward(_t(4, 8), _t(4, 2, dtype=torch.int32)), ValueError, "neither"),
    (lambda: m.route_backward(_t(4, 8), _t(4, 2, dtype=torch.int32), w=_t(4, 2)), ValueError, "together"),
    (lambda: m.route_backward(_t(4, 8), _t(4, 2, dtype=torch.int32), lse=_t(4)), ValueError, "together"),
    (lambda: m.combine_backward(_t(4, 2), _t(4, 2), _t(4, 8)), ValueError, "dimensions"),
    (lambda: m.combine_backward(_t(4, 2, 8), _t(4, 2), _t(4, 8), need=()), ValueError, "need"),
    (lambda: m.combine_backward(_t(4, 2, 8), _t(4, 2), _t(4, 8), need=("dz",)), ValueError, "need"),
    (lambda: m.combine_backward(_t(4, 2, 8, dtype=torch.float16), _t(4, 2), _t(4, 8)), TypeError, "y must be"),
    (lambda: m.linear(_t(4, 64), _t(8, 64, dtype=BF), act="relu"), ValueError, "act"),
    (lambda: m.linear(_t(4, 64), _t(7, 64, dtype=BF), act="swiglu"), ValueError, "even"),
    (lambda: m.linear(_t(4, 64, dtype=torch.float16), _t(8, 64, dtype=BF)), TypeError, "x must be"),
    (lambda: m.linear(_t(4, 64), _t(8, 64, dtype=BF)), ValueError, "CUDA"),
    (lambda: m.linear_backward(_t(4, 8), _t(4, 64), _t(8, 64, dtype=BF), act="silu"), ValueError, "pre"),
    (lambda: m.linear_backward(_t(4, 8), _t(4, 64), _t(8, 64, dtype=BF), need=("dx", "dy")), ValueError, "need"),
    (lambda: m.linear_backward(_t(4, 9), _t(4, 64), _t(8, 64, dtype=BF)), ValueError, "dy"),
])
def test_binding_refusals(call, error, word):
    with pytest.raises(error, match=word):
        call()


def test_balance_loss_overlaps_are_refused():
    # logits, ids, mask, loss, counts, lse, ws = a .. g
    def call(p):
        return int(L.moe_balance_loss(p["a"], p["b"], p["c"], 128, 64, 4, p["d"], p["e"], p["f"], p["g"], 1 << 20, None))

    for out in "defg":
        for other in "abcdefg":
            if out == other:
                continue
            places = {n: _at(16 + 2 * i) for i, n in enumerate("abcdefg")}
            places[out] = places[other]
            assert call(places) == EINVAL, (out, other)
            assert b"overlap" in L.moe_last_error(), (out, other)


@pytest.mark.parametrize("T,K,N", [(1 << 21, 64, 64), (100, 1 << 30, 64), (100, 64, 1 << 30), (100, 64, 16385)])
def test_workspaces_of_refused_sizes_are_zero(T, K, N):
    for act in ("none", "swiglu"):
        assert m.linear_workspace_bytes(T, K, N, act, torch.float32, torch.float32) == 0
        assert m.linear_backward_workspace_bytes(T, K, N, act, torch.float32, torch.float32) == 0


@pytest.mark.parametrize("name,call", [
    ("logits", lambda big: m.balance_loss(big, big.to(torch.int32))),
    ("logits", lambda big: m.route_backward(big, big.to(torch.int32), w=big, dw=big)),
    ("y", lambda big: m.combine_backward(big[:, :, None], big, big)),
    ("x", lambda big: m.linear(big, _t(8, 64, dtype=BF))),
    ("x", lambda big: m.linear_backward(big, big, _t(8, 64, dtype=BF)))])
def test_rows_past_32_bits_are_refused(name, call):
    """One row more than 2^32 would otherwise pass for a single one.  (Meta tensors: no memory behind the rows.)"""
    big = torch.empty(((1 << 32) + 1, 1), device="meta")
    with pytest.raises(ValueError, match=name + r".*2\^31"):
        call(big)


@pytest.mark.parametrize("T,K,N", [(100, 16, 64), (100, 33, 64), (100, 48, 64), (65, 4104, 512), (8192, 4112, 4096),
                                   (8192, 0, 4096), (8192, 4096, 0), (-1, 64, 64), (0, 64, 64)])
def test_workspaces_of_unsupported_shapes_are_zero(T, K, N):
    """What the calls refuse (K that is no multiple of 32 among it) or have no rows for needs no workspace."""
    for act in ("none", "swiglu"):
        assert m.linear_workspace_bytes(T, K, N, act, torch.float32, torch.float32) == 0
        assert m.linear_backward_workspace_bytes(T, K, N, act, torch.float32, torch.float32) == 0


@pytest.mark.parametrize("act,x_t,y_t", [(4, F32, F32), (-1, F32, F32), (0, 2, F32), (0, F32, 2), (0, -1, F32)])
def test_workspaces_of_unknown_types_are_zero(act, x_t, y_t):
    assert int(L.moe_linear_workspace_bytes(8192, 4096, 4096, 0, F32, F32)) > 0
    assert int(L.moe_linear_workspace_bytes(8192, 4096, 4096, act, x_t, y_t)) == 0
    for types in [(x_t, y_t, F32, F32), (F32, F32, x_t, y_t)]:
        assert int(L.moe_linear_backward_workspace_bytes(8192, 4096, 4096, act, *types, 7)) == 0


def test_dense_workspaces_that_overlap_are_refused():
    # x, w, bias, residual, y, pre = a .. f, ws = g; places 64 MB apart
    nb = m.linear_workspace_bytes(500, 2048, 1024, "silu", torch.float32, torch.float32)
    assert 0 < nb < 32 << 20

    def linear(p):
        return int(L.moe_linear(p["a"], F32, p["b"], p["c"], 2, p["d"], F32, 500, 2048, 1024, p["e"], F32, p["f"], p["g"], nb,
                                None))

    # dy, pre, x, w, dx, dw, db = a .. f and h, ws = g
    nb_back = m.linear_backward_workspace_bytes(333, 544, 201, "gelu", dx_dtype=BF)
    assert 0 < nb_back < 32 << 20

    def backward(p):
        return int(L.moe_linear_backward(p["a"], BF16, p["b"], p["c"], BF16, p["d"], 1, 333, 544, 201, p["e"], BF16, p["f"], F32,
                                         p["h"], p["g"], nb_back, None))

    for call, others in [(linear, "abcdef"), (backward, "abcdefh")]:
        for other in others:
            for by in (0, 256):
                places = {n: _at(64 + 64 * i) for i, n in enumerate("abcdefgh")}
                places["g"] = ctypes.c_void_p(places[other].value + by)
                assert call(places) == EINVAL, (call, other)
                assert b"overlap" in L.moe_last_error(), (call, other)


def test_forms():
    for T, K, N in [(0, 64, 64), (-1, 64, 64), (100, 48, 64), (100, 64, 0)]:
        with pytest.raises(m.MoeError):
            m.linear_form(T, K, N)
        with pytest.raises(m.MoeError):
            m.linear_backward_form(T, K, N)
    form = (ctypes.c_int32 * 4)()
    assert int(L.moe_linear_form(100, 64, 64, 0, F32, 2, form)) == EINVAL
    assert int(L.moe_linear_form(100, 64, 64, 0, F32, F32, None)) == EINVAL
    assert int(L.moe_linear_backward_form(100, 64, 64, 0, F32, F32, 5, F32, 7, form)) == EINVAL
    assert int(L.moe_linear_backward_form(100, 64, 64, 4, F32, F32, F32, F32, 7, form)) == EINVAL
    assert m.linear_form(64, 64, 64) == {"tile": 0, "parts": 1, "terms": 1, "planes": 0}
    assert m.linear_form(64, 64, 64, x_dtype=torch.float32)["terms"] == 3
    assert m.linear_backward_form(100, 64, 64, need=("db",)) == {"tile": 0, "dw_parts": 0, "dx_parts": 0, "terms": 1}
    only = m.linear_backward_form(100, 64, 64, dy_dtype=torch.float32, need=("dx",))
    assert only["dw_parts"] == 0 and only["dx_parts"] >= 1 and only["terms"] == 2
