"""Measured cases of the operators around the products: norm, router, 8-bit checkpoints, low-rank adapters.

Each case is one pass through one operator, in a plain form (`own = False`: elementary torch operations in 32
bits, or 64 where a choice hangs on the last bits, rounded once) or through this package's entry points
(`own = True`), on the same prepared state.

  norm            residual + x, its root-mean-square norm in BF16 and / or quantised to E4M3 with one FP32 scale
                  per 1x128 block
  norm_backward   gradients of the norm's input (with the residual stream's) and of its weight
  route           the topk experts of each token and their weights from a router's logits
  route_backward  gradient of the logits
  keep            pre-activations kept for the backward pass in E4M3, one power-of-two scale per 1x128 block
  kept_backward   gradients of bias and pre-activation from a kept pre-activation, and the activation's output again
  lora            act(A @ B.T + the row's adapter's low-rank product + bias)
"""
import math

import torch

own = False

ALIGN = 128      # rows every expert's segment starts on a multiple of (contiguous layout)
FP8_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode: the hidden states of a batch, quantised for the first FP8 product of a layer
        dict(name="norm_fp8_decode", op="norm", T=32, H=7168, residual=True, y=False, q=True),
        # a ragged BF16 micro-batch whose width is no multiple of 128
        dict(name="norm_bf16_ragged", op="norm", T=1021, H=1000, residual=True, y=True, q=False),
        # prefill: 8192 tokens; BF16 for the router and the dispatch, E4M3 for a dense FP8 product
        dict(name="norm_both_prefill", op="norm", T=8192, H=7168, residual=True, y=True, q=True),
        # training backward of a large batch, with the gradient that arrives along the residual stream
        dict(name="norm_bwd_large", op="norm_backward", T=8192, H=4096, residual=True),
        # decode: 256 experts in eight groups, sigmoid scores with a bias for balance
        dict(name="route_decode", op="route", T=32, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, best=2,
             renormalise=True, bf16=False),
        # prefill of the same router
        dict(name="route_prefill", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, best=2,
             renormalise=True, bf16=False),
        # training: gradient of a softmax router's BF16 logits, weights as the softmax gives them
        dict(name="route_bwd_softmax", op="route_backward", T=8192, E=64, k=4, score="softmax", renormalise=False,
             bf16=True),
        # training forward at odd sizes: a dense layer's pre-activations are kept
        dict(name="keep_odd", op="keep", M=517, N=2112, G=0),
        # training backward of four experts: dZ, the bias gradient and the second product's operand again
        dict(name="kept_bwd_experts", op="kept_backward", M=8192, N=4096, G=4, act="silu", h=True, bias=True),
        # decode: 32 requests, most with an adapter of their own, beside one projection
        dict(name="lora_decode", op="lora", M=32, N=7168, K=2048, R=16, L=32, act="none", bias=False, mix="rows"),
        # a small batch of short prompts at odd sizes, with bias and activation
        dict(name="lora_odd", op="lora", M=517, N=2112, K=1536, R=24, L=5, act="silu", bias=True, mix="requests"),
        # prefill of several requests with adapters of rank 64
        dict(name="lora_prefill", op="lora", M=4096, N=7168, K=2048, R=64, L=8, act="none", bias=False,
             mix="requests"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "route", "route", "route_backward", "keep", "kept_backward",
                     "lora", "lora"])
    if op == "norm":
        q = rng.random() < 0.6
        H = 128 * rng.randint(2, 56) if q else rng.choice([8 * rng.randint(16, 896), rng.randint(100, 4000)])
        return dict(op=op, T=_log(rng, 1, 8192), H=H, residual=rng.random() < 0.7, y=not q or rng.random() < 0.5, q=q)
    if op == "norm_backward":
        return dict(op=op, T=_log(rng, 16, 8192), H=rng.choice([8 * rng.randint(16, 512), rng.randint(100, 4000)]),
                    residual=rng.random() < 0.6)
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.choice([8, 16, 32]) if groups > 1 else rng.choice([4, 7, 32, 60, 64, 128, 160, 256])
        T = _log(rng, 1, 8192)
        score = rng.choice(["softmax", "sigmoid"])
        case = dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), score=score, renormalise=rng.random() < 0.6,
                    bf16=rng.random() < 0.4)
        if op == "route":
            kept = max(1, groups // 2)
            case.update(bias=rng.random() < 0.6, groups=groups, kept=kept, best=rng.choice([1, 2]))
        return case
    if op in ("keep", "kept_backward"):
        G = rng.choice([0, 0, 2, 5, 8])
        N = rng.choice([8 * rng.randint(16, 512), 64 * rng.randint(2, 64), rng.randint(100, 3000)])
        case = dict(op=op, M=_log(rng, 8, 8192), N=N, G=G)
        if op == "kept_backward":
            case.update(act=rng.choice(["relu", "silu", "gelu", "gelu_tanh"]), h=rng.random() < 0.6,
                        bias=rng.random() < 0.6)
        return case
    M = _log(rng, 1, 4096)
    return dict(op=op, M=M, N=rng.choice([8 * rng.randint(16, 512), 64 * rng.randint(2, 112), rng.randint(100, 3000)]),
                K=64 * rng.randint(4, 32), R=8 * rng.randint(1, 8), L=rng.choice([1, 3, 8, 32]),
                act=rng.choice(["none", "none", "silu", "gelu"]), bias=rng.random() < 0.4,
                mix="rows" if M <= 256 and rng.random() < 0.6 else "requests")


# ------------------------------------------------------------------ state
def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _hidden(T, H, gen):
    """Hidden states with some channels much larger than the others."""
    gain = torch.exp(0.5 * torch.randn((1, H), generator=gen, device="cuda"))
    return (torch.randn((T, H), generator=gen, device="cuda") * gain).to(torch.bfloat16)


def _segments(M, G, seed):
    """Rows of each expert (uneven, M in all) and the row index of the contiguous layout that holds them."""
    share = torch.rand(G, generator=torch.Generator().manual_seed(seed + 7)) + 0.3
    if G > 2:
        share[1] = 0.0
    n = [int(M * float(v)) for v in share / share.sum()]
    n[0] += M - sum(n)
    m = []
    for g, c in enumerate(n):
        m += [g] * c + [-1] * (-c % ALIGN)
    room = -(-(M + G * (ALIGN - 1)) // ALIGN) * ALIGN        # what any counts fit in
    return torch.tensor(m + [-2] * (room - len(m)), dtype=torch.int32, device="cuda")


def _power_scales(x):
    """E8M0 exponents of each 1x128 block of x: the least power of two that brings the block within E4M3's range."""
    M, N = x.shape
    B = -(-N // 128)
    p = torch.zeros((M, B * 128), dtype=torch.float32, device=x.device)
    p[:, :N] = x
    top = p.reshape(M, B, 128).abs().amax(-1)
    # exponent of top / 448, up to the next whole one: top = m 2^e with m in [0.5, 1), 448 = 0.875 2^9
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(top > 0, e.clamp(min=-126) + 127, torch.full_like(e, 127)).to(torch.uint8)


def _codes_of(x, e):
    s = torch.exp2(e.float() - 127).repeat_interleave(128, 1)[:, :x.shape[1]]
    return (x.float() / s).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _kept(st, dtype=torch.float32):
    """The values that the kept codes stand for."""
    z = st["codes"].to(dtype)
    return z * torch.exp2(st["scales"].to(dtype) - 127).repeat_interleave(128, 1)[:, :z.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        st["weight"] = (1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(torch.bfloat16)
        st["x"] = _hidden(T, H, gen)
        res = case["residual"]
        if op == "norm":
            st["residual"] = _hidden(T, H, gen) if res else None
            st["s"] = _empty((T, H), torch.bfloat16) if res else None
            st["y"] = _empty((T, H), torch.bfloat16) if case["y"] else None
            st["q"] = _empty((T, H), torch.uint8).view(torch.float8_e4m3fn) if case["q"] else None
            st["sf"] = _empty((H // 128, T), torch.float32) if case["q"] else None
            return st
        st["dy"] = _normal((T, H), gen)
        st["ds"] = _normal((T, H), gen) if res else None
        st["dx"] = _empty((T, H), torch.bfloat16)
        st["dweight"] = _empty((H,), torch.float32)
        return st
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        dtype = torch.bfloat16 if case["bf16"] else torch.float32
        # a few popular experts
        logits = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn((1, E), generator=gen, device="cuda")
        st["logits"] = (1.5 * logits).to(dtype)
        if op == "route":
            st["bias"] = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
            st["ids"] = _empty((T, k), torch.int32)
            st["weights"] = _empty((T, k), torch.float32)
            return st
        st["ids"] = torch.topk(st["logits"].float(), k, dim=1)[1].to(torch.int32).contiguous()
        st["d_weights"] = torch.randn((T, k), generator=gen, device="cuda")
        st["d_logits"] = _empty((T, E), dtype)
        return st
    if op in ("keep", "kept_backward"):
        M, N, G = case["M"], case["N"], case["G"]
        st["m_indices"] = _segments(M, G, seed) if G else None
        rows = int(st["m_indices"].numel()) if G else M
        z = _normal((rows, N), gen, 1.5)
        if op == "keep":
            st["z"] = z
            st["codes"] = torch.zeros((rows, N), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            st["scales"] = torch.zeros((rows, -(-N // 128)), dtype=torch.uint8, device="cuda")
            return st
        st["scales"] = _power_scales(z.float())
        st["codes"] = _codes_of(z, st["scales"])
        st["dd"] = _normal((rows, N), gen)
        st["dz"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        st["h"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda") if case["h"] else None
        st["dbias"] = _empty((G, N) if G else (N,), torch.float32) if case["bias"] else None
        return st
    M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
    st["a"] = _normal((M, K), gen)
    st["b"] = _normal((N, K), gen, 1.0 / math.sqrt(K))
    st["down"] = _normal((L, R, K), gen, 1.0 / math.sqrt(K))
    st["up"] = _normal((L, N, R), gen, 1.0 / math.sqrt(R))
    st["scale"] = 0.25 + 0.5 * torch.rand(L, generator=gen, device="cuda")
    host = torch.Generator().manual_seed(seed + 3)
    if case["mix"] == "rows":        # one token a request; -1: a request without an adapter
        which = torch.randint(-1, L, (M,), generator=host)
    else:                            # prompts of uneven lengths
        which = torch.empty(M, dtype=torch.long)
        at = 0
        while at < M:
            n = 1 + int(torch.randint(0, max(1, M // 4), (1,), generator=host))
            which[at:at + n] = int(torch.randint(-1, L, (1,), generator=host))
            at += n
    st["adapter"] = which.to(torch.int32).cuda()
    st["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    st["d"] = _empty((M, N), torch.bfloat16)
    return st


# ------------------------------------------------------------------ plain forms
def _plain_norm(st):
    x = st["x"].float()
    out = {}
    if st["residual"] is not None:
        x = x + st["residual"].float()
        out["s"] = x.to(torch.bfloat16)
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * st["weight"].float()
    if st["y"] is not None:
        out["y"] = y.to(torch.bfloat16)
    if st["q"] is not None:
        b = y.reshape(y.shape[0], -1, 128)
        amax = b.abs().amax(-1, keepdim=True)
        s = torch.where(amax == 0, torch.ones_like(amax), (amax / FP8_MAX).clamp(min=TINY))
        out["q"] = (b / s).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).reshape(y.shape)
        out["sf"] = s[..., 0].t().contiguous()
    return out


def _plain_norm_backward(st):
    x, dy, w = st["x"].float(), st["dy"].float(), st["weight"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n = x * r
    g = dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
    return dict(dx=dx.to(torch.bfloat16), dweight=(dy * n).sum(0))


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _first(key, n):
    """Columns of the n largest of each row, largest first, the lowest column among equals."""
    return torch.sort(key, dim=1, descending=True, stable=True)[1][:, :n]


def _plain_route(st):
    c = st["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    s = _scores(st["logits"].double(), c["score"])
    key = s if st["bias"] is None else s + st["bias"].double()
    if G > 1:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True)[0][..., :c["best"]].sum(2)
        keep = torch.zeros((T, G), dtype=torch.bool, device=key.device)
        keep.scatter_(1, _first(best, c["kept"]), True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, torch.full_like(key, -math.inf))
    ids = _first(key, c["k"])
    w = torch.gather(s, 1, ids)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), weights=(2.5 * w).float())


def _plain_route_backward(st):
    c = st["case"]
    s = _scores(st["logits"].float(), c["score"])
    ids = st["ids"].long()
    chosen = torch.gather(s, 1, ids)
    dw = 2.5 * st["d_weights"]
    if c["renormalise"]:
        total = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_add_(1, ids, dw)
    if c["score"] == "sigmoid":
        dl = ds * s * (1 - s)
    else:
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_keep(st):
    z = st["z"]
    if st["m_indices"] is not None:      # padding rows are kept as zeros, rows past the segments not at all
        z = torch.where((st["m_indices"] >= 0)[:, None], z, torch.zeros_like(z))
    e = _power_scales(z.float())
    codes = _codes_of(z, e)
    if st["m_indices"] is not None:
        e = torch.where((st["m_indices"] >= -1)[:, None], e, torch.zeros_like(e))
    return dict(codes=codes, scales=e)


def _plain_kept_backward(st):
    c = st["case"]
    z = _kept(st)
    dz = st["dd"].float() * _act_grad(z, c["act"])
    h = _act(z, c["act"])
    m = st["m_indices"]
    if m is not None:
        real = (m >= 0)[:, None]
        dz, h = torch.where(real, dz, torch.zeros_like(dz)), torch.where(real, h, torch.zeros_like(h))
    out = dict(dz=dz.to(torch.bfloat16))
    if st["h"] is not None:
        out["h"] = h.to(torch.bfloat16)
    if st["dbias"] is not None:
        if m is None:
            out["dbias"] = dz.sum(0)
        else:
            out["dbias"] = torch.stack([dz[m == g].sum(0) for g in range(c["G"])])
    return out


def _plain_lora(st):
    c = st["case"]
    a = st["a"].float()
    z = a @ st["b"].float().t()
    if c["M"] <= 64:                     # every row with its own adapter's matrices
        at = st["adapter"].clamp(min=0).long()
        low = (a[:, None, :] * st["down"][at].float()).sum(2) * st["scale"][at][:, None]
        delta = (low[:, None, :] * st["up"][at].float()).sum(2)
        z = z + torch.where((st["adapter"] >= 0)[:, None], delta, torch.zeros_like(delta))
    for l in range(c["L"] if c["M"] > 64 else 0):        # two products an adapter, over all rows
        mine = (st["adapter"] == l)[:, None] * st["scale"][l]
        z = z + ((a @ st["down"][l].float().t()) * mine) @ st["up"][l].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    return _act(z, c["act"]).to(torch.bfloat16)


# ------------------------------------------------------------------ this package's operators
def _own(st):
    import moe_grouped_gemm_scales_amd as dg
    c = st["case"]
    op = c["op"]
    if op == "norm":
        dg.dg_rms_norm(st["x"], st["weight"], EPS, Y=st["y"], residual=st["residual"], S=st["s"], Q=st["q"], sf=st["sf"])
        return {n: st[n] for n in ("s", "y", "q", "sf") if st[n] is not None}
    if op == "norm_backward":
        dg.dg_rms_norm_backward(st["dy"], st["x"], st["weight"], EPS, st["dx"], st["dweight"], dS=st["ds"])
        return dict(dx=st["dx"], dweight=st["dweight"])
    if op == "route":
        dg.dg_moe_route(st["logits"], st["bias"], st["ids"], st["weights"], score=c["score"], groups=c["groups"],
                        topk_groups=c["kept"], group_best=c["best"], renormalise=c["renormalise"], scale=2.5)
        return dict(ids=st["ids"], weights=st["weights"])
    if op == "route_backward":
        dg.dg_moe_route_backward(st["logits"], st["ids"], st["d_weights"], st["d_logits"], score=c["score"],
                                 renormalise=c["renormalise"], scale=2.5)
        return st["d_logits"]
    if op == "keep":
        dg.dg_checkpoint_fp8(st["z"], st["codes"], st["scales"], m_indices=st["m_indices"])
        return dict(codes=st["codes"], scales=st["scales"])
    if op == "kept_backward":
        dg.dg_epilogue_backward_fp8(st["dd"], st["codes"], st["scales"], c["act"], st["dz"], st["dbias"], H=st["h"],
                                    m_indices=st["m_indices"], num_experts=c["G"] or None)
        return {n: st[n] for n in ("dz", "h", "dbias") if st[n] is not None}
    dg.dg_bf16_gemm_nt_lora(st["a"], st["b"], st["down"], st["up"], st["adapter"], st["d"], scale=st["scale"],
                            bias=st["bias"], activation=c["act"])
    return st["d"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route,
            "route_backward": _plain_route_backward, "keep": _plain_keep, "kept_backward": _plain_kept_backward,
            "lora": _plain_lora}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        each = 2 + 4 * case["residual"] + 2 * case["y"] + (1 + 4 / 128) * case["q"]
        return dict(bytes=T * H * each + 2 * H, flops=5 * T * H)
    if op == "norm_backward":
        T, H = case["T"], case["H"]
        return dict(bytes=T * H * (6 + 2 * case["residual"]) + 6 * H, flops=10 * T * H)
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        wide = 2 if case["bf16"] else 4
        if op == "route":
            return dict(bytes=T * (E * wide + 8 * k) + 4 * E * case["bias"], flops=10 * T * E)
        return dict(bytes=T * (2 * E * wide + 8 * k), flops=10 * T * E)
    if op in ("keep", "kept_backward"):
        M, N, G = case["M"], case["N"], case["G"]
        if op == "keep":
            return dict(bytes=M * N * 3 + M * -(-N // 128), flops=2 * M * N)
        return dict(bytes=M * N * (5 + 2 * case["h"]) + M * -(-N // 128) + 4 * max(1, G) * N * case["bias"],
                    flops=10 * M * N)
    M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
    used = min(L, M)
    return dict(bytes=2 * (M * K + N * K + M * N + used * R * (K + N)) + 4 * M + 4 * N * case["bias"],
                flops=2 * M * N * K + 2 * M * R * (K + N))


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "route": _exact_route,
            "route_backward": _exact_route_backward, "keep": _exact_keep, "kept_backward": _exact_kept_backward,
            "lora": _exact_lora}[case["op"]](st)


def _exact_norm(st):
    x = st["x"].double()
    out = {}
    if st["residual"] is not None:
        x += st["residual"].double()
        out["s"] = x
    length = torch.sqrt(torch.linalg.vecdot(x, x) / x.shape[1] + EPS)
    y = x / length[:, None] * st["weight"].double()
    if st["y"] is not None:
        out["y"] = y
    if st["q"] is not None:
        blocks = y.unflatten(1, (-1, 128))
        top = blocks.abs().max(-1).values
        scale = torch.clamp(top / 448, min=TINY).masked_fill(top == 0, 1.0)
        out["q"] = (blocks / scale.unsqueeze(-1)).flatten(1)
        out["sf"] = scale.T.contiguous()
    return out


def _exact_norm_backward(st):
    x, dy = st["x"].double(), st["dy"].double()
    H = x.shape[1]
    square = torch.linalg.vecdot(x, x) / H + EPS
    root = square.sqrt()[:, None]
    g = dy * st["weight"].double()
    dx = g / root - x * (torch.linalg.vecdot(g, x) / (H * square * square.sqrt()))[:, None]
    if st["ds"] is not None:
        dx += st["ds"].double()
    return dict(dx=dx, dweight=torch.einsum("th,th->h", dy, x / root))


def _exact_score(l, score):
    return torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)


def _exact_route(st):
    """The choice by repeated search for the largest, group by group and expert by expert."""
    c = st["case"]
    s = _exact_score(st["logits"].double(), c["score"])
    value = s.clone() if st["bias"] is None else s + st["bias"].double()
    T, E, G = c["T"], c["E"], c["groups"]
    rows = torch.arange(T, device=s.device)

    def largest(v):
        top = v.max(1, keepdim=True).values
        at = torch.arange(v.shape[1], device=v.device).expand_as(v)
        return torch.where(v == top, at, torch.full_like(at, v.shape[1])).min(1).values

    if G > 1:
        rest = value.view(T, G, -1).clone()
        worth = torch.zeros((T, G), dtype=torch.float64, device=s.device)
        for _ in range(c["best"]):
            top, at = rest.max(2)
            worth += top
            rest.scatter_(2, at.unsqueeze(2), -math.inf)
        allowed = torch.zeros((T, G), dtype=torch.bool, device=s.device)
        for _ in range(c["kept"]):
            g = largest(worth)
            allowed[rows, g] = True
            worth[rows, g] = -math.inf
        value.view(T, G, -1)[~allowed] = -math.inf
    w = []
    for _ in range(c["k"]):
        e = largest(value)
        w.append(s[rows, e])
        value[rows, e] = -math.inf
    w = torch.stack(w, 1)
    if c["renormalise"]:
        w = w / w.sum(1)[:, None]
    return dict(ids=None, weights=2.5 * w)


def _exact_route_backward(st):
    c = st["case"]
    l = st["logits"].double().requires_grad_()
    w = torch.take_along_dim(_exact_score(l, c["score"]), st["ids"].long(), 1)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad(2.5 * w, l, st["d_weights"].double())[0]


def _exact_keep(st):
    z = st["z"].double()
    M, N = z.shape
    if st["m_indices"] is not None:
        z[st["m_indices"] < 0] = 0
    out = torch.empty_like(z)
    for first in range(0, N, 128):
        block = z[:, first:first + 128]
        top = block.abs().max(1).values
        # 2^e with top / 2^e at most 448, e the least
        e = torch.ceil(torch.log2(torch.where(top > 0, top / 448, torch.ones_like(top)))).clamp(min=-126)
        out[:, first:first + 128] = block / torch.exp2(e)[:, None]
    return dict(codes=out, scales=None)


def _phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * _phi(z)
    if act == "gelu_tanh":       # (1 + tanh u) / 2 is the logistic function of 2 u
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return torch.relu(z) if act == "relu" else z


def _exact_slope(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        return _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(u * (z + 0.044715 * z * z * z))
        return s + z * s * (1 - s) * u * (1 + 0.134145 * z * z)
    return (z > 0).double() if act == "relu" else torch.ones_like(z)


def _exact_kept_backward(st):
    c = st["case"]
    M, N = st["codes"].shape
    scale = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), st["scales"].int() - 127)
    z = torch.empty((M, N), dtype=torch.float64, device="cuda")
    for j in range(scale.shape[1]):
        z[:, 128 * j:128 * j + 128] = st["codes"][:, 128 * j:128 * j + 128].double() * scale[:, j, None]
    dz, h = st["dd"].double() * _exact_slope(z, c["act"]), _exact_act(z, c["act"])
    spans = [torch.arange(M, device="cuda")]
    if c["G"]:
        dz[st["m_indices"] < 0] = 0
        h[st["m_indices"] < 0] = 0
        spans = [torch.nonzero(st["m_indices"] == g)[:, 0] for g in range(c["G"])]
    out = dict(dz=dz)
    if st["h"] is not None:
        out["h"] = h
    if st["dbias"] is not None:
        out["dbias"] = torch.stack([dz[r].sum(0) for r in spans]).reshape(st["dbias"].shape)
    return out


def _exact_lora(st):
    c = st["case"]
    a = st["a"].double()
    z = torch.mm(a, st["b"].double().t())
    for l in sorted(set(st["adapter"].tolist()) - {-1}):
        r = torch.nonzero(st["adapter"] == l)[:, 0]
        low = torch.mm(a[r], st["down"][l].double().t())
        z[r] += st["scale"][l].double() * torch.mm(low, st["up"][l].double().t())
    if st["bias"] is not None:
        z += st["bias"].double()
    return _exact_act(z, c["act"])
