"""8-bit entry points, without a GPU: bad arguments are refused on the host before anything is enqueued, workspaces follow
the sizes of the work, and the binding names what is wrong."""
import ctypes

import pytest
import torch

import expert_routed_ffn_amd as m
from expert_routed_ffn_amd import _lib

L = _lib.lib
P = ctypes.c_void_p(0x100000)    # never read: every call below is refused, or has no rows
ODD = ctypes.c_void_p(0x100002)
F32, BF16, I8 = _lib.MOE_F32, _lib.MOE_BF16, _lib.MOE_I8
OK, EINVAL, EUNSUP, EWS = _lib.MOE_OK, _lib.MOE_EINVAL, _lib.MOE_EUNSUPPORTED, _lib.MOE_EWORKSPACE


def _at(mb):
    return ctypes.c_void_p(mb << 20)


def _rows(x=_at(1), x_t=BF16, T=4, K=64, q=_at(2), scale=_at(3)):
    return int(L.moe_quantize_rows(x, x_t, T, K, q, scale, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EUNSUP), (dict(K=0), EUNSUP), (dict(K=48), EUNSUP), (dict(K=16416), EUNSUP),
    (dict(x_t=2), EINVAL), (dict(x_t=-1), EINVAL), (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(x=ODD), EINVAL), (dict(q=ODD), EINVAL), (dict(scale=ODD), EINVAL), (dict(q=_at(1)), EINVAL),
    (dict(scale=_at(1)), EINVAL), (dict(scale=_at(2)), EINVAL)])
def test_quantize_rows_refusals(kw, want):
    assert _rows(**kw) == want
    assert b"moe_quantize_rows" in L.moe_last_error()


def test_no_rows():
    assert _rows(T=0) == OK
    assert _linear(T=0) == OK


def _linear(x=_at(1), x_t=I8, xs=_at(2), w=_at(3), ws=_at(4), bias=None, act=0, res=None, r_t=0, T=4, K=64, N=8, y=_at(5),
            y_t=BF16, work=_at(64), nb=1 << 30):
    return int(L.moe_linear_q8(x, x_t, xs, w, ws, bias, act, res, r_t, T, K, N, y, y_t, work, nb, None))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), EINVAL), (dict(T=(1 << 20) + 1), EUNSUP), (dict(K=48), EUNSUP), (dict(K=0), EUNSUP), (dict(K=16416), EUNSUP),
    (dict(N=0), EUNSUP), (dict(N=16385), EUNSUP), (dict(act=4), EINVAL), (dict(act=-1), EINVAL), (dict(x_t=3), EINVAL),
    (dict(y_t=2), EINVAL), (dict(res=P, r_t=2), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(xs=None), EINVAL), (dict(x_t=BF16), EINVAL), (dict(y=None), EINVAL), (dict(x=ODD), EINVAL),
    (dict(w=ODD), EINVAL), (dict(xs=ODD), EINVAL), (dict(ws=ODD), EINVAL), (dict(work=ODD), EINVAL),
    (dict(y=ODD, y_t=F32), EINVAL), (dict(bias=ODD), EINVAL), (dict(x_t=BF16, xs=None, T=100, work=None), EWS),
    (dict(x_t=F32, xs=None, T=100, nb=16), EWS)])
def test_linear_q8_refusals(kw, want):
    assert _linear(**kw) == want
    assert b"moe_linear_q8" in L.moe_last_error()


def test_overlapping_buffers_are_refused():
    # x, x_scale, w, w_scale, bias, residual, y, ws = a .. h, 64 MB apart
    nb = m.linear_q8_workspace_bytes(500, 8192, 64, "silu", torch.float32)
    assert 0 < nb < 32 << 20

    def codes(p):
        return int(L.moe_linear_q8(p["a"], I8, p["b"], p["c"], p["d"], p["e"], 2, p["f"], F32, 500, 8192, 64, p["g"], BF16,
                                   p["h"], nb, None))

    def floats(p):
        return int(L.moe_linear_q8(p["a"], F32, None, p["c"], p["d"], p["e"], 2, p["f"], F32, 500, 8192, 64, p["g"], BF16,
                                   p["h"], nb, None))

    assert m.linear_q8_workspace_bytes(500, 8192, 64, "silu", torch.int8) > 0  # a cut reduction: ws is written there too
    for call, inputs in ((codes, "abcdef"), (floats, "acdef")):
        for out in "gh":
            for other in inputs + ("h" if out == "g" else "g"):
                places = {n: _at(64 + 64 * i) for i, n in enumerate("abcdefgh")}
                places[out] = ctypes.c_void_p(places[other].value + 256)
                if other in "bde":  # (vectors of a few hundred values)
                    places[out] = places[other]
                assert call(places) == EINVAL, (out, other)
                assert b"overlap" in L.moe_last_error(), (out, other)
    # y on the residual is allowed only as the very buffer of the same type
    assert _linear(res=_at(5), r_t=F32) == EINVAL


@pytest.mark.parametrize("T,K,N", [(1 << 21, 64, 64), (100, 48, 64), (100, 1 << 30, 64), (100, 64, 16385), (0, 64, 64), (-1, 64, 64),
                                   (100, 64, 0)])
def test_workspaces_of_refused_sizes_are_zero(T, K, N):
    for act in ("none", "swiglu"):
        for t in (torch.float32, torch.bfloat16, torch.int8):
            assert m.linear_q8_workspace_bytes(T, K, N, act, t) == 0


def test_workspaces():
    assert m.linear_q8_workspace_bytes(3, 2048, 512, "swiglu") == 0
    assert m.linear_q8_workspace_bytes(8192, 2048, 512, "swiglu", torch.int8) == 0
    assert m.linear_q8_workspace_bytes(8192, 2048, 512, "swiglu") == 8192 * (2048 + 4)
    assert int(L.moe_linear_q8_workspace_bytes(100, 64, 64, 4, BF16)) == 0
    assert int(L.moe_linear_q8_workspace_bytes(100, 64, 64, 0, 3)) == 0


def test_forms():
    for T, K, N in [(0, 64, 64), (-1, 64, 64), (100, 48, 64), (100, 64, 0)]:
        with pytest.raises(m.MoeError):
            m.linear_q8_form(T, K, N)
    form = (ctypes.c_int32 * 3)()
    assert int(L.moe_linear_q8_form(100, 64, 64, 0, 3, form)) == EINVAL
    assert int(L.moe_linear_q8_form(100, 64, 64, 0, BF16, None)) == EINVAL
    assert m.linear_q8_form(1, 2048, 512, "swiglu") == {"tile": 0, "parts": 1, "coded_before": 0}
    assert m.linear_q8_form(64, 256, 64) == {"tile": 0, "parts": 1, "coded_before": 0}
    assert m.linear_q8_form(64, 288, 64) == {"tile": 0, "parts": 1, "coded_before": 1}
    assert m.linear_q8_form(64, 64, 64, x_dtype=torch.int8)["coded_before"] == 0
    assert m.linear_q8_form(100, 64, 64)["tile"] == 64


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


I = torch.int8


@pytest.mark.parametrize("call,error,word", [
    (lambda: m.quantize_rows(_t(4)), ValueError, "dimensions"),
    (lambda: m.quantize_rows(_t(4, 64, dtype=torch.float16)), TypeError, "x must be"),
    (lambda: m.quantize_rows(_t(64, 4).t()), ValueError, "contiguous"),
    (lambda: m.quantize_rows(_t(4, 64)), ValueError, "CUDA"),
    (lambda: m.linear_q8(_t(4, 64), _t(8, 64, dtype=I), _t(8), act="relu"), ValueError, "act"),
    (lambda: m.linear_q8(_t(4, 64), _t(7, 64, dtype=I), _t(7), act="swiglu"), ValueError, "even"),
    (lambda: m.linear_q8(_t(4, 64, dtype=torch.float16), _t(8, 64, dtype=I), _t(8)), TypeError, "x must be"),
    (lambda: m.linear_q8(_t(4, 64), _t(8, 64, dtype=I), _t(8)), ValueError, "CUDA"),
    (lambda: m.quantize_rows(torch.empty(((1 << 32) + 1, 1), device="meta")), ValueError, r"2\^31"),
    (lambda: m.linear_q8_workspace_bytes(4, 64, 8, x_dtype=torch.float16), TypeError, "dtype"),
    (lambda: m.linear_q8_workspace_bytes(4, 64, 8, act="relu"), ValueError, "act"),
])
def test_binding_refusals(call, error, word):
    with pytest.raises(error, match=word):
        call()
