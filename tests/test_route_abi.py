"""Argument checks of the routing entry points on the CPU (refused before any HIP call), and the gradient's formula
against differences."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import _Routing, lib
from tests import layer_ref as ref

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


@pytest.mark.parametrize("kw,status", [
    (dict(l=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(T=-1), INVALID),
    (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(type=2), INVALID), (dict(score=2), INVALID),
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(kept=0), INVALID), (dict(kept=5), INVALID),
    (dict(best=0), INVALID), (dict(best=3), INVALID), (dict(kept=1, k=5), INVALID), (dict(E=2048), UNSUPPORTED),
    (dict(E=130, k=65, groups=1, kept=1), UNSUPPORTED), (dict(E=130, k=1, groups=65), UNSUPPORTED),
    (dict(T=1 << 26), UNSUPPORTED), (dict(l=FAKE + 2), ALIGNMENT), (dict(l=FAKE + 1, type=1), ALIGNMENT),
    (dict(bias=FAKE + 2), ALIGNMENT), (dict(ids=FAKE + 2), ALIGNMENT), (dict(w=FAKE + 1), ALIGNMENT)])
def test_route_refusals(kw, status):
    a = dict(l=FAKE, type=0, bias=FAKE, ids=FAKE, w=FAKE, T=4, E=16, k=4, score=1, groups=4, kept=2, best=2) | kw
    r = _Routing(a["score"], a["groups"], a["kept"], a["best"], 1, 1.0)
    assert lib.dg_moe_route(P(a["l"]), a["type"], P(a["bias"]), ctypes.byref(r), P(a["ids"]), P(a["w"]), a["T"], a["E"],
                            a["k"], None) == status
    assert lib.dg_last_error().decode()
    if not {"groups", "kept", "best", "bias"} & set(kw):
        assert lib.dg_moe_route_backward(P(a["l"]), a["type"], P(a["ids"]), P(a["w"]), ctypes.byref(r), P(FAKE), a["T"],
                                         a["E"], a["k"], None) == status


def test_route_null_and_nothing():
    f, r = P(FAKE), _Routing(0, 1, 1, 1, 1, 1.0)
    assert lib.dg_moe_route(f, 0, None, None, f, f, 4, 16, 2, None) == INVALID
    assert lib.dg_moe_route_backward(f, 0, f, f, None, f, 4, 16, 2, None) == INVALID
    assert lib.dg_moe_route_backward(f, 0, f, f, ctypes.byref(r), None, 4, 16, 2, None) == INVALID
    assert lib.dg_moe_route_backward(f, 0, f, f, ctypes.byref(r), P(FAKE + 2), 4, 16, 2, None) == ALIGNMENT
    assert lib.dg_moe_route(None, 0, None, ctypes.byref(r), None, None, 0, 16, 2, None) == 0
    assert lib.dg_moe_route_backward(None, 0, None, None, ctypes.byref(r), None, 0, 16, 2, None) == 0


def test_route_binding_refuses_wrong_tensors():
    l, i, w = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    with pytest.raises(ValueError):
        dg.dg_moe_route(l, None, i, w)                              # host tensors
    with pytest.raises(TypeError):
        dg.dg_moe_route(l.half(), None, i, w)
    with pytest.raises(ValueError):
        dg.dg_moe_route(l, None, i.reshape(-1), w)
    with pytest.raises(ValueError):
        dg.dg_moe_route_backward(l, i, w, l)
    from moe_grouped_gemm_scales_amd.dg import _routing
    with pytest.raises(ValueError):
        _routing("relu", 1, 1, 1, True, 1.0)
    with pytest.raises(ValueError):
        _routing("softmax", 2 ** 32 + 1, 1, 1, True, 1.0)           # would wrap to one group


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient_against_differences(score, renormalise):
    g = torch.Generator().manual_seed(2)
    T, E, k, step = 3, 7, 3, 1e-6
    l, dw = torch.randn((T, E), generator=g, dtype=torch.float64), torch.randn((T, k), generator=g, dtype=torch.float64)
    ids, _ = ref.route(l, None, k, score)

    def loss(l):
        p = torch.gather(ref.scores(l, score), 1, ids.long())
        return float((1.5 * (p / p.sum(1, keepdim=True) if renormalise else p) * dw).sum())

    got, _ = ref.route_backward(l, ids, dw, score, renormalise, 1.5)
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(l)
            d[t, e] = step
            assert abs((loss(l + d) - loss(l - d)) / (2 * step) - float(got[t, e])) < 1e-8


def test_negative_groups_do_not_wrap():
    """-2^32 + 1 groups are refused by the library as -1, not taken as one."""
    from moe_grouped_gemm_scales_amd.dg import _routing
    assert _routing("softmax", 1 - 2 ** 32, 1, 1, True, 1.0)._obj.groups < 0
    assert _routing("softmax", 1, 1 - 2 ** 32, 2 - 2 ** 32, True, 1.0)._obj.group_best < 0


def test_settings_are_read_at_every_call():
    """A scale or renormalise held in a tensor that changes in place counts as it is now; equal numbers of other types
    do not decide what is taken."""
    from moe_grouped_gemm_scales_amd.dg import _routing
    scale, renormalise, groups = torch.tensor(2.5), torch.tensor(True), torch.tensor(2)
    first = _routing("softmax", groups, 1, 1, renormalise, scale)._obj
    assert (first.groups, first.renormalise, first.scale) == (2, 1, 2.5)
    scale.fill_(3.0), renormalise.fill_(False), groups.fill_(4)
    now = _routing("softmax", groups, 1, 1, renormalise, scale)._obj
    assert (now.groups, now.renormalise, now.scale) == (4, 0, 3.0)
    weight = torch.nn.Parameter(torch.tensor(0.5), requires_grad=False)
    assert _routing("sigmoid", 1, 1, 1, True, weight)._obj.scale == 0.5
    weight += 1
    assert _routing("sigmoid", 1, 1, 1, True, weight)._obj.scale == 1.5
    for _ in range(2):                                              # before and after an equal whole number is kept
        with pytest.raises(TypeError):
            _routing("softmax", 1.0, 1, 1, True, 1.0)
        _routing("softmax", 1, 1, 1, True, 1)
