"""The orthogonalised update's entry points, without a GPU: bad arguments are refused on the host before anything is
enqueued, workspaces follow the sizes of the work, and the binding names what is wrong."""
import ctypes

import pytest
import torch

import expert_routed_ffn_amd as m
from expert_routed_ffn_amd import _lib

L = _lib.lib
F32, BF16, I8 = _lib.MOE_F32, _lib.MOE_BF16, _lib.MOE_I8
OK, EINVAL, EUNSUP, EWS = _lib.MOE_OK, _lib.MOE_EINVAL, _lib.MOE_EUNSUPPORTED, _lib.MOE_EWORKSPACE
ODD = ctypes.c_void_p(0x100001)
INF, NAN = float("inf"), float("nan")


def _at(mb):
    return ctypes.c_void_p(mb << 20)


def _call(g=_at(1), g_t=F32, mom=None, beta=0.95, nesterov=1, B=2, R=40, K=60, steps=5, coef=None, eps=1e-7, o=_at(2),
          o_t=BF16, ws=_at(64), nb=1 << 30):
    return int(L.moe_orthogonalize(g, g_t, mom, beta, nesterov, B, R, K, steps, coef, eps, o, o_t, ws, nb, None))


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), EINVAL), (dict(R=0), EUNSUP), (dict(K=0), EUNSUP), (dict(R=-5), EUNSUP), (dict(R=16385), EUNSUP),
    (dict(K=16385), EUNSUP), (dict(B=33, R=16384, K=16384), EUNSUP), (dict(B=2147483647, R=64, K=128), EUNSUP), (dict(steps=0), EUNSUP),
    (dict(steps=17), EUNSUP), (dict(g_t=I8), EINVAL), (dict(o_t=I8), EINVAL), (dict(o_t=-1), EINVAL), (dict(beta=1.0), EINVAL),
    (dict(beta=-0.1), EINVAL), (dict(beta=NAN), EINVAL), (dict(eps=-1e-9), EINVAL), (dict(eps=INF), EINVAL),
    (dict(eps=NAN), EINVAL), (dict(g=None), EINVAL), (dict(o=None), EINVAL), (dict(g=ODD), EINVAL), (dict(o=ODD), EINVAL),
    (dict(mom=ODD), EINVAL), (dict(ws=ODD), EINVAL), (dict(ws=None), EWS), (dict(nb=1024), EWS),
    (dict(o=_at(1)), EINVAL), (dict(mom=_at(1)), EINVAL), (dict(mom=_at(2)), EINVAL), (dict(ws=_at(1)), EINVAL),
    (dict(ws=_at(2)), EINVAL), (dict(mom=_at(64)), EINVAL),
    (dict(coef=(ctypes.c_float * 15)(*([1.0] * 14), NAN)), EINVAL), (dict(coef=(ctypes.c_float * 15)(INF, *([1.0] * 14))), EINVAL)])
def test_refusals(kw, want):
    assert _call(**kw) == want
    assert b"moe_orthogonalize" in L.moe_last_error()


def test_no_matrices():
    assert _call(B=0) == OK
    assert _call(B=0, R=0) == EUNSUP


def test_workspaces():
    assert m.orthogonalize_workspace_bytes(0, 64, 64) == 0
    assert m.orthogonalize_workspace_bytes(-1, 64, 64) == 0
    assert m.orthogonalize_workspace_bytes(1, 16385, 64) == 0
    assert m.orthogonalize_workspace_bytes(1, 0, 64) == 0
    assert m.orthogonalize_workspace_bytes(33, 16384, 16384) == 0
    assert int(L.moe_orthogonalize_workspace_bytes(1, 64, 64, I8)) == 0
    one, two = m.orthogonalize_workspace_bytes(1, 512, 2048), m.orthogonalize_workspace_bytes(1, 512, 2048, torch.float32)
    # X twice in two terms of 2 bytes; A and P
    assert one > 8 * 512 * 2048 + 4 * 512 * 512 and two >= one + 4 * 512 * 512
    assert m.orthogonalize_workspace_bytes(1, 2048, 512) == one
    assert m.orthogonalize_workspace_bytes(32, 16384, 16384) > 1 << 36


def test_forms():
    for a in [(0, 64, 64), (-1, 64, 64), (1, 0, 64), (1, 64, 16385)]:
        with pytest.raises(m.MoeError):
            m.orthogonalize_form(*a)
    form = (ctypes.c_int32 * 4)()
    assert int(L.moe_orthogonalize_form(1, 64, 64, I8, form)) == EINVAL
    assert int(L.moe_orthogonalize_form(1, 64, 64, BF16, None)) == EINVAL
    assert m.orthogonalize_form(1, 60, 544) == {"gram": 0, "apply": 0, "gram_paired": 0, "apply_paired": 0}
    assert m.orthogonalize_form(1, 544, 65) == {"gram": 32, "apply": 32, "gram_paired": 1, "apply_paired": 1}


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,error,word", [
    (lambda: m.orthogonalize(_t(4)), ValueError, "dimensions"),
    (lambda: m.orthogonalize(_t(2, 2, 4, 4)), ValueError, "dimensions"),
    (lambda: m.orthogonalize(_t(4, 8, dtype=torch.float16)), TypeError, "g must be"),
    (lambda: m.orthogonalize(_t(8, 4).t()), ValueError, "contiguous"),
    (lambda: m.orthogonalize(_t(4, 8)), ValueError, "CUDA"),
    (lambda: m.orthogonalize(torch.empty(((1 << 32) + 1, 1), device="meta")), ValueError, r"2\^31"),
    (lambda: m.orthogonalize_workspace_bytes(1, 64, 64, torch.int8), TypeError, "dtype"),
])
def test_binding_refusals(call, error, word):
    with pytest.raises(error, match=word):
        call()


def test_coefficients_of_the_binding():
    one, many = (3.0, -2.0, 0.5), [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5)]
    assert _lib._newton_coefs(one, 3) == [3.0, -2.0, 0.5] * 3
    assert _lib._newton_coefs(many, 2) == [1.5, -0.5, 0.0, 2.0, -1.5, 0.5]
    assert _lib._newton_coefs(torch.tensor(many), 2) == _lib._newton_coefs(many, 2)
    assert _lib._newton_coefs(torch.tensor(one, dtype=torch.float64), 1) == list(one)
    assert len(_lib._newton_coefs(one, 1 << 30)) == 3 * 16  # the call refuses that many steps before it reads any
    for coef, steps in [((), 5), ((1.0, 2.0), 5), (many, 3), (many, 1), ([(1.0, 2.0)], 1), ([one, 1.0], 2)]:
        with pytest.raises(ValueError, match="coef"):
            _lib._newton_coefs(coef, steps)
