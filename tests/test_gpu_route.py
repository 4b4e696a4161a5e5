"""Routing and its gradient on the GPU against a plain implementation in 64 bits.

The choice is made on 64-bit values, so ids must be equal; weights are rounded once to FP32 (2^-24, and as much
again for the 64-bit exponential's own error, far below).  The gradient is computed in FP32: exponentials of
differences of up to 30 (30 2^-24 of each, 2 ulp of the function), two sums over 64 lanes and five more
operations, below 64 2^-24 = 2^-18 of the terms' magnitudes; BF16 gradients are rounded to 2^-8."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import layer_ref as ref
from tests.test_gpu_norm import Fenced, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _logits(T, E, seed, bf16=False, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    l = 2 * torch.randn((T, E), generator=g)
    if kind == "equal":
        l = torch.ones((T, E))
    if kind == "ties":                       # few distinct values
        l = torch.randint(-2, 3, (T, E), generator=g).float()
    if kind == "close":                      # neighbours in FP32, in a range where a sigmoid's FP32 values run together
        l = torch.full((T, E), 14.0) + torch.randint(0, 8, (T, E), generator=g) * 2.0 ** -20
    return l.to(torch.bfloat16) if bf16 else l


def _route(logits, bias, k, **kw):
    T = logits.shape[0]
    ids, w = Fenced((T, k), torch.int32), Fenced((T, k), torch.float32)
    dg.dg_moe_route(logits.cuda(), None if bias is None else bias.cuda(), ids.t, w.t, **kw)
    return ids.check(), w.check()


def _check(logits, bias, k, **kw):
    ids, w = _route(logits, bias, k, **kw)
    wi, ww = ref.route(logits, bias, k, **kw)
    assert torch.equal(ids, wi)
    _near(w, ww, 2 ** -23 * ww.abs())
    return ids


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (17, 7, 7), (9, 60, 6), (33, 64, 4), (5, 65, 8), (40, 128, 8),
                                   (7, 160, 6), (21, 256, 8), (4, 384, 16), (3, 1000, 64), (2, 1024, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased,renormalise", [(True, True), (False, False)])
def test_route(T, E, k, score, bf16, biased, renormalise):
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(3)) if biased else None
    _check(_logits(T, E, E + k, bf16), bias, k, score=score, renormalise=renormalise, scale=1.75)


@pytest.mark.parametrize("kind", ["equal", "ties", "close"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(96, 1), (256, 8), (1024, 64)])
def test_route_ties(kind, score, E, groups):
    """Equal values go to the lowest index; values that only FP64 tells apart are told apart."""
    _check(_logits(12, E, 5, kind=kind), None, 6, score=score, groups=groups, topk_groups=max(1, groups // 2), group_best=2)


@pytest.mark.parametrize("E,groups,kept", [(8, 2, 1), (12, 3, 2), (60, 5, 2), (64, 64, 8), (256, 8, 4), (160, 8, 3),
                                           (320, 20, 7), (1024, 16, 1), (96, 33 - 1, 9)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, groups, kept, best, score):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(4))
    k = min(8, kept * (E // groups))
    ids = _check(_logits(19, E, E), bias, k, score=score, groups=groups, topk_groups=kept, group_best=best)
    used = torch.zeros((19, groups), dtype=torch.bool).scatter_(1, (ids // (E // groups)).long(), True)
    assert (used.sum(1) <= kept).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_experts_that_are_not_available(score, groups):
    """-inf logits, and biases, are never chosen; too few, or none: id -1 with weight 0."""
    E, k = 16, 4
    l = _logits(6, E, 8)
    l[0] = -float("inf")                       # none
    l[1] = -float("inf")
    l[1, 5] = 0.5                              # one
    l[2, ::2] = -float("inf")
    l[3, :12] = -float("inf")                  # one group
    bias = torch.zeros(E)
    bias[7] = -float("inf")
    for b in (None, bias):
        ids = _check(l, b, k, score=score, groups=groups, topk_groups=2 if groups > 1 else 1, group_best=2)
        assert (ids[0] == -1).all() and ids[1].tolist() == [5, -1, -1, -1]
        assert not bool((ids[2] % 2 == 0).any())
        if b is not None:
            assert not bool((ids == 7).any())


def test_route_nan():
    """A NaN ranks last and shows in the weights where it belongs to the sum; other rows are as ever."""
    l = _logits(3, 8, 9)
    l[1, 2] = float("nan")
    ids, w = _route(l, None, 3, score="sigmoid")
    wi, ww = ref.route(l, None, 3, score="sigmoid")
    assert torch.equal(ids, wi) and not bool((ids[1] == 2).any())
    _near(w, ww, 2 ** -23 * ww)
    ids, w = _route(l, None, 3, score="softmax")
    wi, ww = ref.route(l, None, 3, score="softmax")
    assert torch.equal(ids, wi) and torch.isnan(w[1]).all()
    _near(w[::2], ww[::2], 2 ** -23 * ww[::2])
    ids, w = _route(l[1:2], None, 8, score="sigmoid")
    assert int(ids[0, 7]) == 2 and torch.isnan(w).all()
    l[1, 2] = float("inf")
    ids, w = _route(l, None, 3, score="sigmoid")
    assert int(ids[1, 0]) == 2 and torch.isfinite(w).all()


def test_route_far_logits():
    """Sigmoids far below FP32's range still have their ratios."""
    l = torch.full((2, 5), -200.0)
    l[1] = torch.tensor([-300.0, -299.0, -310.0, -299.0, -298.0])
    _check(l, None, 3, score="sigmoid")
    _check(l, None, 3, score="softmax")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (17, 7, 7), (9, 60, 6), (33, 64, 4), (5, 65, 8), (40, 128, 8),
                                   (21, 256, 8), (4, 384, 16), (3, 1000, 64), (2, 1024, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_backward(T, E, k, score, bf16, renormalise):
    l = _logits(T, E, E + 1, bf16)
    ids, _ = ref.route(l, None, k, score)
    _backward(l, ids, score, renormalise)


def _backward(l, ids, score, renormalise):
    dw = torch.randn(ids.shape, generator=torch.Generator().manual_seed(6))
    out = Fenced(l.shape, l.dtype)
    dg.dg_moe_route_backward(l.cuda(), ids.cuda(), dw.cuda(), out.t, score=score, renormalise=renormalise, scale=1.75)
    want, mag = ref.route_backward(l, ids, dw, score, renormalise, 1.75)
    _near(out.check(), want, 2 ** -18 * mag + (2 ** -8 * want.abs() if l.dtype == torch.bfloat16 else 2 ** -126))
    a = l.cuda()
    dg.dg_moe_route_backward(a, ids.cuda(), dw.cuda(), a, score=score, renormalise=renormalise, scale=1.75)    # in place
    assert torch.equal(a.cpu(), out.t.cpu())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_backward_odd_ids(score, renormalise):
    """Ids outside the experts add nothing, one named twice gets both terms, a token without experts nothing at all."""
    l = _logits(5, 9, 7)
    l[2, 4] = -float("inf")
    l[4] = -float("inf")
    ids = torch.tensor([[0, 3, -1, 8], [5, 5, 2, 5], [4, 1, 9, 100], [-1, -1, -1, -1], [0, 1, -1, 2]], dtype=torch.int32)
    _backward(l, ids, score, renormalise)
    _backward(_logits(2, 70, 8) - 200, torch.tensor([[0, 69], [3, 4]], dtype=torch.int32), score, renormalise)


def test_route_to_combine_and_back():
    """Router, sort, dispatch, combine and their gradients in a row: the gradient of the logits of sum(y * dy)."""
    T, E, k, H = 50, 8, 2, 256
    g = torch.Generator().manual_seed(11)
    l = torch.randn((T, E), generator=g)
    x, dy = (torch.randn((T, H), generator=g).to(torch.bfloat16) for _ in range(2))
    gain = 1 + torch.arange(E)                                   # expert e multiplies by e + 1
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    dg.dg_moe_route(l.cuda(), None, ids, w)
    R = dg.moe_sorted_rows(T, k, E)
    pos, m, ks = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((T, k), (R,), (E,)))
    dg.dg_moe_sort_contiguous(ids, E, pos, m, ks)
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_dispatch_bf16(x.cuda(), pos, m, rows)
    rows = rows * gain.cuda()[m.clamp(min=0).long()][:, None]
    y = dg.dg_moe_combine(rows.contiguous(), pos, w, None, torch.empty((T, H), dtype=torch.bfloat16, device="cuda"))
    d_rows, dw = torch.zeros_like(rows), torch.empty((T, k), device="cuda")
    dg.dg_moe_combine_backward(dy.cuda(), rows.contiguous(), pos, w, m, d_rows, dw)
    dl = dg.dg_moe_route_backward(l.cuda(), ids, dw, torch.empty((T, E), device="cuda"))
    leaf = l.double().requires_grad_()
    p = torch.softmax(leaf, 1)
    chosen = torch.topk(p, k, dim=1)[1]
    cw = torch.gather(p, 1, chosen)
    cw = cw / cw.sum(1, keepdim=True)
    scaled = (x.float()[:, None] * gain[chosen][..., None]).to(torch.bfloat16).double()      # the rows, rounded as above
    want = (cw[..., None] * scaled).sum(1)
    _near(y.cpu(), want.detach(), 2 ** -8 * (1 + 2 ** -8) * want.detach().abs() + 2 ** -20 * scaled.abs().sum(1))
    (want * dy.double()).sum().backward()
    mag = (dy.double()[:, None] * scaled).abs().sum((1, 2)) * 2
    _near(dl.cpu(), leaf.grad, 2 ** -16 * mag[:, None].expand(T, E))


def test_route_replayed():
    """Captured on a side stream, replayed with new logits between eager calls."""
    T, E, k = 64, 256, 8
    stream = torch.cuda.Stream()
    kw = dict(score="sigmoid", groups=8, topk_groups=4, group_best=2)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda()
    l, dw = _logits(T, E, 1).cuda(), torch.randn((T, k)).cuda()
    ids, w, dl = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty_like(l)

    def step():
        dg.dg_moe_route(l, bias, ids, w, **kw)
        dg.dg_moe_route_backward(l, ids, dw, dl, score="sigmoid")

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in range(3):
            l.copy_(_logits(T, E, 20 + seed))
            graph.replay()
            got = [t.clone() for t in (ids, w, dl)]
            step()
            stream.synchronize()
            for a, b in zip(got, (ids, w, dl)):
                assert torch.equal(a, b)


# experts, groups, groups kept: lanes with 1, 2 and 4 experts, groups of whole lanes and others, rows that are not
# read in whole pieces
PROMPTS = [(7, 1, 1), (60, 5, 2), (96, 3, 2), (160, 8, 3), (250, 5, 2), (256, 8, 4)]


@pytest.mark.parametrize("T,E,groups,kept", [(1027, *c) for c in PROMPTS] + [(2049, 256, 8, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_of_prompts(T, E, groups, kept, score, bf16):
    """From 1024 tokens on a workgroup has four, the last one fewer; the gradient in the same sizes."""
    k = min(6, E // groups * kept)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(12))
    l = _logits(T, E, E + T, bf16)
    ids = _check(l, bias, k, score=score, groups=groups, topk_groups=kept, group_best=2 if E // groups > 1 else 1)
    for renormalise in (True, False):
        _backward(l, ids, score, renormalise)


def test_route_group_that_lacks_its_second_expert():
    """What is missing counts 0, so a group with one expert of 0.5 beats one of 0.6 and -0.2; a group without any is
    kept last."""
    inf = float("inf")
    l = torch.zeros((1, 8))                       # sigmoid: 0.5 each
    bias = torch.tensor([0.0, 0, 0.1, -0.7, 0, 0, -0.35, -0.35])
    l[0, 1] = l[0, 4] = l[0, 5] = -inf            # worth 0.5, 0.6 - 0.2, nothing, 0.15 + 0.15
    for kept, want in ((1, [0, -1]), (2, [2, 0, 3, -1]), (3, [2, 0, 6, 7, 3]), (4, [2, 0, 6, 7, 3, -1])):
        ids, _ = _route(l, bias, len(want), score="sigmoid", groups=4, topk_groups=kept, group_best=2)
        assert ids[0].tolist() == want
