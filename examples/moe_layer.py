"""A mixture-of-experts feed-forward layer from this library's operators.

Training, BF16 (forward and backward, contiguous layout):

    sort -> dispatch -> Z1 = rows W1^T + b1, h = act(Z1) -> out = h W2^T + b2 -> y = x + sum_j w_j out

Serving a few tokens, FP8 weights (masked layout): the tokens are quantised on their way to the experts,
the first product is FP8 with its bias and activation in the epilogue, its BF16 result goes through
dg_moe_dispatch_fp8 row by row to become the second product's operand.

A whole block, y = x + experts(norm(x)), with a router that is trained and the first product's pre-activation kept in
8 bits from the forward to the backward pass (MoEBlock):

    norm -> router product -> route -> sort -> dispatch -> Z1 (kept in E4M3), h -> out -> combine with x

`python examples/moe_layer.py` runs them at a small size and prints how far they are from the same layer
in 32-bit torch operations, and the time of a step.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_scales_amd as dg  # noqa: E402

BF16 = torch.bfloat16


def route(x, router, topk):
    """Expert ids [T, topk] (int32) and their normalised weights (float32) from a softmax router."""
    p = torch.softmax(x.float() @ router.float().T, dim=1)
    w, ids = torch.topk(p, topk, dim=1)
    return ids.to(torch.int32).contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


class MoELayer:
    """Training layer for up to `tokens` tokens a step; its row buffers are kept from step to step."""

    def __init__(self, tokens, hidden, inner, experts, topk, activation="silu", device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, scale: (torch.randn(s, generator=g, device=device) * scale).to(BF16)
        self.topk, self.experts, self.act = topk, experts, activation
        self.router = rnd(experts, hidden, scale=hidden ** -0.5)
        self.w1, self.w2 = rnd(experts, inner, hidden, scale=hidden ** -0.5), rnd(experts, hidden, inner, scale=inner ** -0.5)
        self.b1 = torch.randn((experts, inner), generator=g, device=device) * 0.1
        self.b2 = torch.randn((experts, hidden), generator=g, device=device) * 0.1
        rows = dg.moe_sorted_rows(tokens, topk, experts)
        # the products leave rows that they do not compute as they are, so a new buffer is cleared
        buf = lambda width: torch.zeros((rows, width), dtype=BF16, device=device)
        self.rows, self.z1, self.h, self.out = buf(hidden), buf(inner), buf(inner), buf(hidden)
        self.d_out, self.dh, self.d_rows = buf(hidden), buf(inner), buf(hidden)
        self.m_indices = torch.empty(rows, dtype=torch.int32, device=device)
        self.ks = torch.empty(experts, dtype=torch.int32, device=device)
        self.no_tokens = torch.empty((0, inner), dtype=BF16, device=device)
        self.no_places = torch.empty((0, topk), dtype=torch.int32, device=device)

    def forward(self, x, ids, weights):
        self.x, self.weights = x, weights
        self.pos = torch.empty_like(ids)
        dg.dg_moe_sort_contiguous(ids, self.experts, self.pos, self.m_indices, self.ks)
        dg.dg_moe_dispatch_bf16(x, self.pos, self.m_indices, self.rows)
        # a dispatch of no tokens clears the padding rows.  The gradient of w2 multiplies those of h by zeros, and
        # an infinity or NaN that an earlier step left in one would come through that.
        dg.dg_moe_dispatch_bf16(self.no_tokens, self.no_places, self.m_indices, self.h)
        dg.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(self.rows, self.w1, self.m_indices, self.h, bias=self.b1,
                                                         activation=self.act, Z=self.z1)
        dg.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(self.h, self.w2, self.m_indices, self.out, bias=self.b2)
        return dg.dg_moe_combine(self.out, self.pos, weights, x, torch.empty_like(x))

    def backward(self, dy):
        """Gradients of x, the routing weights and the parameters, as a dict."""
        g = dict(dw=torch.empty_like(self.weights), w1=torch.empty_like(self.w1), w2=torch.empty_like(self.w2),
                 b1=torch.empty_like(self.b1), b2=torch.empty_like(self.b2))
        m = self.m_indices
        dg.dg_moe_combine_backward(dy, self.out, self.pos, self.weights, m, self.d_out, g["dw"])
        dg.dg_epilogue_backward(self.d_out, None, "none", None, g["b2"], m)
        dg.dg_m_grouped_bf16_gemm_nn_contiguous(self.d_out, self.w2, m, None, self.dh)
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(self.d_out, self.h, self.ks, None, g["w2"])
        dg.dg_epilogue_backward(self.dh, self.z1, self.act, self.dh, g["b1"], m)            # dZ1, in place
        dg.dg_m_grouped_bf16_gemm_nn_contiguous(self.dh, self.w1, m, None, self.d_rows)
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(self.dh, self.rows, self.ks, None, g["w1"])
        # the dispatch's gradient is the unweighted combine; the residual path adds dy itself
        g["x"] = dg.dg_moe_combine(self.d_rows, self.pos, None, dy, torch.empty_like(dy))
        return g


class MoEBlock(MoELayer):
    """Training block x + experts(norm(x)).  Of Z1 and h only 8 bits of Z1 outlive the forward pass: both buffers can
    be shared by a model's blocks, as here by all blocks that are given the same `shared`."""

    def __init__(self, tokens, hidden, inner, experts, topk, activation="silu", device="cuda", seed=0, shared=None):
        super().__init__(tokens, hidden, inner, experts, topk, activation, device, seed)
        g = torch.Generator(device=device).manual_seed(seed + 100)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(BF16)
        self.eps = 1e-6
        self.codes = torch.zeros((self.rows.shape[0], inner), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((self.rows.shape[0], -(-inner // 128)), dtype=torch.uint8, device=device)
        if shared is not None:
            self.z1, self.h = shared.z1, shared.h

    def forward(self, x):
        self.x = x
        self.xn = dg.dg_rms_norm(x, self.norm, self.eps, Y=torch.empty_like(x))
        self.logits = dg.dg_bf16_gemm_nt(self.xn, self.router, None,
                                         torch.empty((x.shape[0], self.experts), dtype=BF16, device=x.device))
        self.ids = torch.empty((x.shape[0], self.topk), dtype=torch.int32, device=x.device)
        self.weights = torch.empty((x.shape[0], self.topk), device=x.device)
        dg.dg_moe_route(self.logits, None, self.ids, self.weights)
        self.pos, m = torch.empty_like(self.ids), self.m_indices
        dg.dg_moe_sort_contiguous(self.ids, self.experts, self.pos, m, self.ks)
        dg.dg_moe_dispatch_bf16(self.xn, self.pos, m, self.rows)
        dg.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(self.rows, self.w1, m, self.h, bias=self.b1,
                                                         activation=self.act, Z=self.z1)
        dg.dg_checkpoint_fp8(self.z1, self.codes, self.scales, m_indices=m)
        dg.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(self.h, self.w2, m, self.out, bias=self.b2)
        return dg.dg_moe_combine(self.out, self.pos, self.weights, x, torch.empty_like(x))

    def backward(self, dy):
        """Gradients of x and the parameters, as a dict."""
        g = {n: torch.empty_like(getattr(self, n)) for n in ("w1", "w2", "b1", "b2", "router")}
        g["norm"] = torch.empty(self.norm.shape, device=dy.device)
        dw, m = torch.empty_like(self.weights), self.m_indices
        dg.dg_moe_combine_backward(dy, self.out, self.pos, self.weights, m, self.d_out, dw)
        dg.dg_epilogue_backward(self.d_out, None, "none", None, g["b2"], m)
        dg.dg_m_grouped_bf16_gemm_nn_contiguous(self.d_out, self.w2, m, None, self.dh)
        # dZ1 in place of dh, and h again: both with cleared padding rows, as the weight gradients need
        dg.dg_epilogue_backward_fp8(self.dh, self.codes, self.scales, self.act, self.dh, g["b1"], H=self.h, m_indices=m)
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(self.d_out, self.h, self.ks, None, g["w2"])
        dg.dg_m_grouped_bf16_gemm_nn_contiguous(self.dh, self.w1, m, None, self.d_rows)
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(self.dh, self.rows, self.ks, None, g["w1"])
        # the router's share of the norm's gradient, and the dispatch's
        d_logits = dg.dg_moe_route_backward(self.logits, self.ids, dw, torch.empty_like(self.logits))
        dg.dg_bf16_gemm_tn(d_logits, self.xn, None, g["router"])
        d_xn = dg.dg_bf16_gemm_nn(d_logits, self.router, None, torch.empty_like(dy))
        d_xn = dg.dg_moe_combine(self.d_rows, self.pos, None, d_xn, d_xn)
        g["x"] = dg.dg_rms_norm_backward(d_xn, self.x, self.norm, self.eps, d_xn, g["norm"], dS=dy)
        return g


def reference_block(block, x):
    """The block in 32-bit torch operations with the block's choice of experts: (y, its inputs by name)."""
    leaf = lambda t: t.detach().float().requires_grad_()
    v = {n: leaf(getattr(block, n)) for n in ("w1", "w2", "b1", "b2", "router", "norm")} | {"x": leaf(x)}
    acts = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu,
                gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"))
    xn = v["x"] * torch.rsqrt(v["x"].pow(2).mean(1, keepdim=True) + block.eps) * v["norm"]
    w = torch.gather(torch.softmax(xn @ v["router"].T, dim=1), 1, block.ids.long())
    w = w / w.sum(1, keepdim=True)
    y = v["x"]
    for j in range(block.topk):
        for e in range(block.experts):
            t = torch.nonzero(block.ids[:, j] == e)[:, 0]
            if len(t):
                h = acts[block.act](xn[t] @ v["w1"][e].T + v["b1"][e])
                y = y.index_add(0, t, w[t, j, None] * (h @ v["w2"][e].T + v["b2"][e]))
    return y, v


def check_block(tokens=300, hidden=512, inner=384, experts=6, topk=2, activation="gelu", seed=0, device="cuda"):
    """Distances of the outputs of two blocks in a row, forward and backward, from the reference, by name."""
    first = MoEBlock(tokens, hidden, inner, experts, topk, activation, device, seed)
    second = MoEBlock(tokens, hidden, inner, experts, topk, activation, device, seed + 1, shared=first)
    g = torch.Generator(device=device).manual_seed(seed + 2)
    far = {}
    for step in range(2):                      # the second step reuses every buffer with other routes
        x, dy = (torch.randn((tokens, hidden), generator=g, device=device).to(BF16) for _ in range(2))
        between = first.forward(x)
        y = second.forward(between)
        grads = [second.backward(dy)]
        grads.append(first.backward(grads[0]["x"]))
        for block, inp, out, dout, got in ((second, between, y, dy, grads[0]), (first, x, between, grads[0]["x"], grads[1])):
            want, v = reference_block(block, inp)
            want.backward(dout.float())
            name = "first" if block is first else "second"
            far |= {f"{name}.y": distance(out, want.detach())} | {f"{name}.{n}": distance(got[n], v[n].grad) for n in v}
    return far


def quantise_weight(w):
    """E4M3 codes and FP32 128x128 scales of w [G, N, K]."""
    G, N, K = w.shape
    nb = -(-N // 128)
    p = torch.zeros((G, nb * 128, K), device=w.device)
    p[:, :N] = w.float()
    b = p.reshape(G, nb, 128, K // 128, 128)
    s = (b.abs().amax((2, 4)) / 448).clamp(min=2.0 ** -126)
    q = (b / s[:, :, None, :, None]).clamp(-448, 448).reshape(G, nb * 128, K)[:, :N]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


class ServingLayer:
    """FP8 decode: the masked layout, at most m_max tokens an expert."""

    def __init__(self, layer: MoELayer, m_max):
        self.p, self.m_max = layer, m_max
        G, inner, hidden = layer.w1.shape
        dev = layer.w1.device
        self.q1, self.s1 = quantise_weight(layer.w1)
        self.q2, self.s2 = quantise_weight(layer.w2)
        f8 = lambda n: torch.zeros((G, m_max, n), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        sf = lambda n: torch.ones((G, n // 128, m_max), device=dev)
        self.rows, self.rows_sf, self.hq, self.h_sf = f8(hidden), sf(hidden), f8(inner), sf(inner)
        self.h = torch.zeros((G, m_max, inner), dtype=BF16, device=dev)
        self.out = torch.zeros((G, m_max, hidden), dtype=BF16, device=dev)
        self.masked_m = torch.empty(G, dtype=torch.int32, device=dev)
        # every row of the masked layout goes to its own place: the second operand's quantisation
        self.each = torch.arange(G * m_max, dtype=torch.int32, device=dev).reshape(-1, 1)

    def forward(self, x, ids, weights):
        p = self.p
        pos = torch.empty_like(ids)
        dg.dg_moe_sort_masked(ids, p.experts, self.m_max, pos, self.masked_m)
        dg.dg_moe_dispatch_fp8(x, pos, None, self.rows, self.rows_sf)
        dg.dg_m_grouped_fp8_gemm_nt_masked_epilogue(self.rows, self.rows_sf, self.q1, self.s1, self.masked_m, self.h,
                                                    bias=p.b1, activation=p.act)
        dg.dg_moe_dispatch_fp8(self.h.reshape(-1, self.h.shape[-1]), self.each, None, self.hq, self.h_sf)
        dg.dg_m_grouped_fp8_gemm_nt_masked_epilogue(self.hq, self.h_sf, self.q2, self.s2, self.masked_m, self.out,
                                                    bias=p.b2)
        return dg.dg_moe_combine(self.out, pos, weights, x, torch.empty_like(x))


def reference(layer, x, ids, weights):
    """The layer in 32-bit torch operations, with gradients by autograd: (y, its inputs by name)."""
    leaf = lambda t: t.detach().float().requires_grad_()
    v = dict(x=leaf(x), dw=leaf(weights), w1=leaf(layer.w1), w2=leaf(layer.w2), b1=leaf(layer.b1), b2=leaf(layer.b2))
    acts = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu,
                gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"))
    y = v["x"]
    for j in range(ids.shape[1]):
        for e in range(layer.experts):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            if len(t):
                h = acts[layer.act](v["x"][t] @ v["w1"][e].T + v["b1"][e])
                y = y.index_add(0, t, v["dw"][t, j, None] * (h @ v["w2"][e].T + v["b2"][e]))
    return y, v


def distance(a, b):
    """2-norm of the difference over the 2-norm of b."""
    return float((a.float() - b.float()).norm() / b.float().norm())


def check(tokens=300, hidden=512, inner=384, experts=6, topk=2, activation="gelu", seed=0, device="cuda"):
    """Distances of the training step's outputs and of the FP8 forward from the reference, by name."""
    layer = MoELayer(tokens, hidden, inner, experts, topk, activation, device, seed)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    far = {}
    for step in range(2):                      # the second step reuses every buffer with other routes
        x, dy = (torch.randn((tokens, hidden), generator=g, device=device).to(BF16) for _ in range(2))
        ids, weights = route(x, layer.router, topk)
        y = layer.forward(x, ids, weights)
        grads = layer.backward(dy)
        want, v = reference(layer, x, ids, weights)
        want.backward(dy.float())
        far = {"y": distance(y, want.detach())} | {n: distance(grads[n], v[n].grad) for n in v}
    served = ServingLayer(layer, tokens).forward(x, ids, weights)
    far["y_fp8"] = distance(served, want.detach())
    return far


def main():
    for name, d in (check() | check_block()).items():
        print(f"{name:14s} {d:.2e}")
    layer = MoELayer(8192, 4096, 2048, 8, 2)
    x = torch.randn((8192, 4096), device="cuda").to(BF16)
    ids, weights = route(x, layer.router, 2)
    for _ in range(3):
        layer.forward(x, ids, weights)
        layer.backward(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        layer.forward(x, ids, weights)
        layer.backward(x)
    end.record()
    torch.cuda.synchronize()
    print(f"forward and backward of 8192 tokens, 8 experts of 4096 x 2048, top 2: {start.elapsed_time(end) / 10:.2f} ms")


if __name__ == "__main__":
    main()
