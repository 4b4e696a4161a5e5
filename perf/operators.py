"""Measured cases of the mixture-of-experts and fused-product operators.

Each case is one pass through one operator, in a plain form (`own = False`: elementary torch operations in 32
bits, rounded once) or through this package's entry points (`own = True`), on the same prepared state.

  route            sort the top-k assignments by expert, then move the tokens to their expert rows
                   (BF16, or quantised to E4M3 with one FP32 scale per 1x128 block)
  combine          weighted sum of a token's expert rows, plus the residual
  combine_backward gradients of the expert rows and of the weights
  linear           act(A @ B.T + bias) + residual: dense, or one weight matrix per expert
  linear_backward  gradients of A, B and bias
"""
import math

import torch

own = False

ALIGN = 128      # rows every expert's segment starts on a multiple of (contiguous layout)
FP8_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode: a handful of tokens into the masked layout of 32 experts, quantised for the FP8 products
        dict(name="route_fp8_masked_decode", op="route", T=32, k=8, G=32, H=7168, fp8=True, m_max=64, drop=False),
        # a ragged BF16 micro-batch on one rank of several: ids of other ranks' experts are not dispatched
        dict(name="route_bf16_ragged", op="route", T=1021, k=3, G=7, H=1000, fp8=False, m_max=0, drop=True),
        # prefill: 8192 tokens, 32768 expert rows of the 7168-wide hidden state, quantised
        dict(name="route_fp8_prefill", op="route", T=8192, k=4, G=32, H=7168, fp8=True, m_max=0, drop=False),
        # decode: the way back, with the residual stream added
        dict(name="combine_masked_decode", op="combine", T=32, k=8, G=32, H=7168, m_max=64, drop=False, residual=True),
        # prefill: the way back for 32768 expert rows
        dict(name="combine_prefill", op="combine", T=8192, k=4, G=32, H=7168, m_max=0, drop=False, residual=True),
        # training: gradients of a ragged micro-batch whose width is no multiple of 128
        dict(name="combine_bwd_ragged", op="combine_backward", T=1021, k=3, G=7, H=1000, m_max=0, drop=True),
        # training: gradients of a large batch
        dict(name="combine_bwd_large", op="combine_backward", T=8192, k=4, G=32, H=4096, m_max=0, drop=False),
        # decode of one token through a dense layer: bound by reading the weights
        dict(name="linear_bf16_one_token", op="linear", form="dense", fp8=False, M=1, N=7168, K=2048, G=1, act="silu",
             bias=True, residual=False, save=False),
        # training forward at odd sizes: everything the epilogue has, the pre-activation kept
        dict(name="linear_bf16_odd", op="linear", form="dense", fp8=False, M=517, N=2112, K=1536, G=1, act="gelu",
             bias=True, residual=True, save=True),
        # prefill of four experts in FP8
        dict(name="linear_fp8_experts", op="linear", form="contiguous", fp8=True, M=8192, N=4096, K=7168, G=4,
             act="silu", bias=True, residual=False, save=False),
        # training backward of a few experts with ragged row counts
        dict(name="linear_bwd_experts", op="linear_backward", form="contiguous", M=1500, N=2112, K=1536, G=5,
             act="gelu_tanh", bias=True),
        # training backward of a large dense layer
        dict(name="linear_bwd_large", op="linear_backward", form="dense", M=8192, N=4096, K=7168, G=1, act="gelu",
             bias=True),
    ]


def _log(rng, lo, hi):
    return _size(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(n):
    """2112, this repository's odd width, stands in for 3072, which none of its configurations has."""
    return 2112 if n == 3072 else n


def _times(rng, step, lo, hi):
    return _size(step * rng.randint(lo, hi))


def draw(rng):
    op = rng.choice(["route", "combine", "combine_backward", "linear", "linear", "linear_backward"])
    if op in ("route", "combine", "combine_backward"):
        k = rng.randint(1, 8)
        G = rng.choice([3, 4, 7, 16, 32, 64, 128, 256])
        masked = op != "combine_backward" and rng.random() < 0.4
        fp8 = op == "route" and rng.random() < 0.6
        T = _log(rng, 1, 256) if masked else _log(rng, 1, 8192)
        T = max(1, min(T, 32768 // k))
        H = 128 * rng.choice([i for i in range(2, 57) if i != 24]) if fp8 else \
            rng.choice([_times(rng, 64, 2, 112), _times(rng, 8, 8, 500), rng.randint(60, 2000)])
        if masked:
            # the buffer of G x m_max rows stays near a gigabyte at most
            G = min(G, 64)
        case = dict(op=op, T=T, k=k, G=G, H=H, m_max=max(16, min(256, 2 * T)) if masked else 0,
                    drop=rng.random() < 0.5)
        if op == "route":
            case["fp8"] = fp8
        if op == "combine":
            case["residual"] = rng.random() < 0.5
        return case
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    if op == "linear":
        form = rng.choice(["dense", "dense", "contiguous", "masked"])
        fp8 = rng.random() < 0.4
        G = 1 if form == "dense" else rng.choice([2, 4, 5, 8])
        M = _log(rng, 1, 8192) if form == "dense" else _log(rng, G, 8192) if form == "contiguous" else _log(rng, 8, 512)
        K = 128 * rng.choice([i for i in range(2, 57) if i != 24]) if fp8 else _times(rng, 64, 2, 112)
        N = rng.choice([_times(rng, 8, 16, 512), _times(rng, 64, 2, 64), _size(rng.randint(100, 4096))])
        return dict(op=op, form=form, fp8=fp8, M=M, N=N, K=K, G=G, act=act, bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, save=rng.random() < 0.4)
    form = rng.choice(["dense", "contiguous"])
    G = 1 if form == "dense" else rng.choice([2, 4, 5, 8])
    return dict(op=op, form=form, M=_log(rng, G, 8192), N=_times(rng, 64, 2, 64 if G == 1 else 32),
                K=rng.choice([_times(rng, 64, 2, 112), _times(rng, 8, 16, 512)]), G=G, act=act,
                bias=rng.random() < 0.7)


# ------------------------------------------------------------------ state
def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _sorted_rows(T, k, G):
    n = T * k
    return -(-(n + min(G, n) * (ALIGN - 1)) // ALIGN) * ALIGN


def _assignments(case, gen):
    """Top-k ids of random scores with a few popular experts, and their softmax weights."""
    T, k, G = case["T"], case["k"], case["G"]
    kk = min(k, G)
    score = torch.randn((T, G), generator=gen, device="cuda") + 0.7 * torch.randn((1, G), generator=gen, device="cuda")
    top, ids = torch.topk(score, kk, dim=1)
    if kk < k:           # fewer experts than choices: some are chosen again
        top, ids = top.repeat(1, -(-k // kk))[:, :k], ids.repeat(1, -(-k // kk))[:, :k]
    weights = torch.softmax(top, dim=1).contiguous()
    ids = ids.to(torch.int32).contiguous()
    if case["drop"]:     # experts of another rank
        away = torch.rand((T, k), generator=gen, device="cuda") < 0.2
        ids = torch.where(away, torch.full_like(ids, -1), ids)
    return ids, weights


def _place(ids, G, m_max):
    """Stable order by expert: (pos, m_indices, segment rows) or (pos, rows of each expert)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < G), flat, torch.full_like(flat, G))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=G + 1)[:G]
    rank = torch.empty_like(flat)
    starts = torch.cumsum(counts, 0) - counts
    ok = key < G
    at = torch.arange(flat.numel(), device=flat.device)
    rank[order] = at - torch.cat([starts, counts.sum().reshape(1)])[key[order]]
    safe = key.clamp(max=G - 1)
    if m_max:
        pos = torch.where(ok & (rank < m_max), safe * m_max + rank, torch.full_like(rank, -1))
        return pos.to(torch.int32).reshape(ids.shape), counts.clamp(max=m_max).to(torch.int32)
    seg = (counts + ALIGN - 1) // ALIGN * ALIGN
    base = torch.cumsum(seg, 0) - seg
    pos = torch.where(ok, base[safe] + rank, torch.full_like(rank, -1))
    R = _sorted_rows(ids.shape[0], ids.shape[1], G)
    r = torch.arange(R, device=flat.device)
    g = torch.searchsorted(base + seg, r, right=True)
    gs = g.clamp(max=G - 1)
    m_indices = torch.where(g >= G, torch.full_like(r, -2),
                            torch.where(r - base[gs] < counts[gs], gs, torch.full_like(r, -1)))
    return pos.to(torch.int32).reshape(ids.shape), m_indices.to(torch.int32), seg.to(torch.int32)


def _quantise_rows(x):
    """x [rows][K] as E4M3 with one FP32 scale per 1x128 block."""
    b = x.float().reshape(x.shape[0], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax == 0, torch.ones_like(amax), (amax / FP8_MAX).clamp(min=TINY))
    q = (b / s).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.reshape(x.shape), s[..., 0]


def _quantise_weight(w):
    """w [N][K] as E4M3 with one FP32 scale per 128x128 block."""
    N, K = w.shape
    Nb = -(-N // 128)
    p = torch.zeros((Nb * 128, K), device=w.device)
    p[:N] = w
    b = p.reshape(Nb, 128, K // 128, 128)
    s = (b.abs().amax((1, 3)) / FP8_MAX).clamp(min=TINY)
    q = (b / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).reshape(Nb * 128, K)[:N]
    return q.to(torch.float8_e4m3fn), s


def _counts(M, G, seed):
    """Rows of each expert: uneven, M in all, the second expert of three or more empty."""
    share = torch.rand(G, generator=torch.Generator().manual_seed(seed + 7)) + 0.3
    if G > 2:
        share[1] = 0.0
    n = [int(M * float(v)) for v in share / share.sum()]
    n[0] += M - sum(n)
    return n


def _layout(case, seed):
    """Grouped row layout: counts of each expert on the host, and the tensor that the entry points take."""
    M, G, form = case["M"], case["G"], case["form"]
    if form == "contiguous":
        counts = _counts(M, G, seed)
        m = []
        for g, c in enumerate(counts):
            m += [g] * c + [-1] * (-c % ALIGN)
        room = -(-(M + G * (ALIGN - 1)) // ALIGN) * ALIGN       # what any counts fit in
        m += [-2] * (room - len(m))
        return counts, torch.tensor(m, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(seed + 7)
    counts = [int(v) for v in torch.randint(0, M + 1, (G,), generator=gen)]
    return counts, torch.tensor(counts, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("route", "combine", "combine_backward"):
        T, k, G, H, m_max = (case[n] for n in ("T", "k", "G", "H", "m_max"))
        st["ids"], st["weights"] = _assignments(case, gen)
        shape = (G, m_max) if m_max else (_sorted_rows(T, k, G),)
        if op == "route":
            # an activation with some channels much larger than the others
            gain = torch.exp(0.5 * torch.randn((1, H), generator=gen, device="cuda"))
            st["x"] = (torch.randn((T, H), generator=gen, device="cuda") * gain).to(torch.bfloat16)
            st["pos"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            st["groups"] = torch.empty(G if m_max else shape[0], dtype=torch.int32, device="cuda")
            if not m_max:
                st["ks"] = torch.empty(G, dtype=torch.int32, device="cuda")
            st["rows"] = torch.zeros((*shape, H), dtype=torch.uint8 if case["fp8"] else torch.bfloat16, device="cuda")
            if case["fp8"]:
                st["rows"] = st["rows"].view(torch.float8_e4m3fn)
                st["sf"] = torch.zeros((*shape[:-1], H // 128, shape[-1]), dtype=torch.float32, device="cuda")
            return st
        placed = _place(st["ids"], G, m_max)
        st["pos"], st["groups"] = placed[0], placed[1]
        st["rows"] = _normal((*shape, H), gen)
        if op == "combine":
            st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            st["residual"] = _normal((T, H), gen) if case["residual"] else None
        else:
            st["dy"] = _normal((T, H), gen)
            st["d_rows"] = torch.zeros((*shape, H), dtype=torch.bfloat16, device="cuda")
            st["d_weights"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        return st
    M, N, K, G, form = (case[n] for n in ("M", "N", "K", "G", "form"))
    lead = ()
    if form == "dense":
        rows, st["groups"], st["counts"] = M, None, [M]
    else:
        st["counts"], st["groups"] = _layout(case, seed)
        lead = (G,)
        rows = G * M if form == "masked" else int(st["groups"].numel())
    shape = (G, M) if form == "masked" else (rows,)
    a = _normal((rows, K), gen)
    if form == "contiguous":
        a = torch.where((st["groups"] >= 0)[:, None], a, torch.zeros_like(a))   # padding rows are zero, as dispatched
    w = _normal((G * N, K), gen, 1.0 / math.sqrt(K))
    st["bias"] = torch.randn((*lead, N), generator=gen, device="cuda") * 0.1 if case["bias"] else None
    if op == "linear":
        if case["fp8"]:
            q, s = _quantise_rows(a)
            Kb = K // 128
            st["a"] = q.reshape(*shape, K)
            st["sfa"] = s.reshape(*shape, Kb).transpose(-1, -2).contiguous()
            parts = [_quantise_weight(w[g * N:(g + 1) * N].float()) for g in range(G)]
            st["b"] = torch.stack([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn).reshape(*lead, N, K)
            st["sfb"] = torch.stack([p[1] for p in parts]).reshape(*lead, -1, Kb)
        else:
            st["a"], st["b"] = a.reshape(*shape, K), w.reshape(*lead, N, K)
        st["residual"] = _normal((*shape, N), gen) if case["residual"] else None
        st["d"] = torch.zeros((*shape, N), dtype=torch.bfloat16, device="cuda")
        st["z"] = torch.zeros((*shape, N), dtype=torch.bfloat16, device="cuda") if case["save"] else None
        return st
    st["a"], st["b"] = a, w.reshape(*lead, N, K)
    st["dd"] = _normal((rows, N), gen)
    st["z"] = _normal((rows, N), gen)
    if form == "contiguous":
        seg = [-(-c // ALIGN) * ALIGN for c in st["counts"]]
        st["ks"] = torch.tensor(seg, dtype=torch.int32, device="cuda")
    st["dz"] = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    st["da"] = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    st["db"] = torch.empty((*lead, N, K), dtype=torch.bfloat16, device="cuda")
    st["dbias"] = torch.empty((*lead, N), dtype=torch.float32, device="cuda") if case["bias"] else None
    return st


# ------------------------------------------------------------------ plain forms
def _plain_route(st):
    c = st["case"]
    placed = _place(st["ids"], c["G"], c["m_max"])
    pos = placed[0]
    x = st["x"]
    flat = st["rows"].reshape(-1, c["H"])
    token = torch.arange(c["T"], device=x.device).repeat_interleave(c["k"])
    # dropped assignments go to a row past the end, which is cut off again
    to = torch.where(pos.reshape(-1) < 0, torch.full_like(pos.reshape(-1), flat.shape[0]), pos.reshape(-1)).long()
    if not c["fp8"]:
        out = torch.zeros((flat.shape[0] + 1, c["H"]), dtype=x.dtype, device=x.device)
        out[to] = x[token]
        return dict(pos=pos, groups=placed[1], rows=out[:-1].reshape(st["rows"].shape), **_ks(placed))
    q, s = _quantise_rows(x)
    out = torch.zeros((flat.shape[0] + 1, c["H"]), dtype=torch.uint8, device=x.device)
    out[to] = q.view(torch.uint8)[token]
    # a row that holds no token: scale 1 in a padding row of a segment, untouched (0 here) past the layout
    sf = torch.zeros((flat.shape[0] + 1, c["H"] // 128), dtype=torch.float32, device=x.device)
    if not c["m_max"]:
        sf[:-1] = (placed[1] == -1).float()[:, None]
    sf[to] = s[token]
    sf = sf[:-1].reshape(*st["rows"].shape[:-1], -1).transpose(-1, -2).contiguous()
    return dict(pos=pos, groups=placed[1], rows=out[:-1].view(torch.float8_e4m3fn).reshape(st["rows"].shape), sf=sf,
                **_ks(placed))


def _ks(placed):
    return dict(ks=placed[2]) if len(placed) > 2 else {}


def _rows_of(st, rows):
    """A token's rows [T][k][H] in FP32 (zeros where dropped), and the flat positions."""
    flat = rows.reshape(-1, rows.shape[-1])
    pos = st["pos"].long()
    keep = (pos >= 0)[..., None]
    return torch.where(keep, flat[pos.clamp(min=0)].float(), torch.zeros((), device=flat.device)), pos


def _plain_combine(st):
    r, _ = _rows_of(st, st["rows"])
    y = (r * st["weights"][..., None]).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def _plain_combine_backward(st):
    r, pos = _rows_of(st, st["rows"])
    dy = st["dy"].float()
    dw = (r * dy[:, None, :]).sum(-1)
    n = st["rows"].numel() // st["rows"].shape[-1]
    d_rows = torch.zeros((n + 1, st["rows"].shape[-1]), dtype=torch.bfloat16, device=dy.device)
    to = torch.where(pos < 0, torch.full_like(pos, n), pos).reshape(-1)
    d_rows[to] = (st["weights"][..., None] * dy[:, None, :]).to(torch.bfloat16).reshape(-1, dy.shape[-1])
    return dict(d_rows=d_rows[:-1].reshape(st["rows"].shape), d_weights=dw)


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


def _dense_operands(st, dtype):
    """A [rows][K] and B [G][N][K] in `dtype`, with the scales applied."""
    c = st["case"]
    N, K, G = c["N"], c["K"], c["G"]
    a, b = st["a"].to(dtype).reshape(-1, K), st["b"].to(dtype).reshape(G, N, K)
    if c.get("fp8"):
        s = st["sfa"].transpose(-1, -2).reshape(a.shape[0], K // 128, 1).to(dtype)
        a = (a.reshape(a.shape[0], -1, 128) * s).reshape(a.shape)
        sb = st["sfb"].reshape(G, -1, K // 128).to(dtype).repeat_interleave(128, 1)[:, :N]
        b = (b.reshape(G, N, -1, 128) * sb[..., None]).reshape(b.shape)
    return a, b


def _spans(st):
    """(expert, first row, rows) of each expert that has rows."""
    c, at, spans = st["case"], 0, []
    for g, n in enumerate(st["counts"]):
        first = g * c["M"] if c["form"] == "masked" else at
        at += -(-n // ALIGN) * ALIGN
        if n:
            spans.append((g, first, n))
    return spans


def _linear(st, dtype):
    c = st["case"]
    a, b = _dense_operands(st, dtype)
    shape = st["d"].shape
    # rows that no expert computes stay as they are (zero)
    d = torch.zeros((a.shape[0], c["N"]), dtype=dtype, device=a.device)
    z = torch.zeros_like(d) if st["z"] is not None else None
    bias = None if st["bias"] is None else st["bias"].to(dtype).reshape(c["G"], -1)
    res = None if st["residual"] is None else st["residual"].reshape(a.shape[0], -1)
    for g, first, n in _spans(st):          # one library product an expert
        part = slice(first, first + n)
        v = a[part] @ b[g].T
        if bias is not None:
            v = v + bias[g]
        if z is not None:
            z[part] = v
        v = _act(v, c["act"])
        if res is not None:
            v = v + res[part].to(dtype)
        d[part] = v
    return d.reshape(shape), z.reshape(shape) if z is not None else None


def _plain_linear(st):
    d, z = _linear(st, torch.float32)
    out = dict(d=d.to(torch.bfloat16))
    if z is not None:
        out["z"] = z.to(torch.bfloat16)
    return out


def _linear_backward(st, dtype):
    c = st["case"]
    a, b = _dense_operands(st, dtype)
    dz = st["dd"].to(dtype) * _act_grad(st["z"].to(dtype), c["act"])
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    dbias = torch.zeros((c["G"], c["N"]), dtype=dtype, device=a.device)
    for g, first, n in _spans(st):          # two library products an expert
        part = slice(first, first + n)
        da[part] = dz[part] @ b[g]
        db[g] = dz[part].T @ a[part]
        dbias[g] = dz[part].sum(0)
    return da, db.reshape(st["b"].shape), dbias.reshape(st["bias"].shape) if st["bias"] is not None else None


def _plain_linear_backward(st):
    da, db, dbias = _linear_backward(st, torch.float32)
    out = dict(da=da.to(torch.bfloat16), db=db.to(torch.bfloat16))
    if dbias is not None:
        out["dbias"] = dbias
    return out


# ------------------------------------------------------------------ this package's operators
def _own(st):
    import moe_grouped_gemm_scales_amd as dg
    c = st["case"]
    op = c["op"]
    if op == "route":
        masked = bool(c["m_max"])
        if masked:
            dg.dg_moe_sort_masked(st["ids"], c["G"], c["m_max"], st["pos"], st["groups"])
        else:
            dg.dg_moe_sort_contiguous(st["ids"], c["G"], st["pos"], st["groups"], st["ks"])
        m_indices = None if masked else st["groups"]
        out = dict(pos=st["pos"], groups=st["groups"], rows=st["rows"])
        if c["fp8"]:
            dg.dg_moe_dispatch_fp8(st["x"], st["pos"], m_indices, st["rows"], st["sf"])
            out["sf"] = st["sf"]
        else:
            dg.dg_moe_dispatch_bf16(st["x"], st["pos"], m_indices, st["rows"])
        if not masked:
            out["ks"] = st["ks"]
        return out
    if op == "combine":
        dg.dg_moe_combine(st["rows"], st["pos"], st["weights"], st["residual"], st["y"])
        return st["y"]
    if op == "combine_backward":
        dg.dg_moe_combine_backward(st["dy"], st["rows"], st["pos"], st["weights"], st["groups"], st["d_rows"],
                                   st["d_weights"])
        return dict(d_rows=st["d_rows"], d_weights=st["d_weights"])
    form = c["form"]
    if op == "linear":
        extra = dict(bias=st["bias"], activation=c["act"], residual=st["residual"], Z=st["z"])
        operands = (st["a"], st["sfa"], st["b"], st["sfb"]) if c["fp8"] else (st["a"], st["b"])
        kind = "fp8" if c["fp8"] else "bf16"
        if form == "dense":
            getattr(dg, f"dg_{kind}_gemm_nt_epilogue")(*operands, st["d"], **extra)
        else:
            getattr(dg, f"dg_m_grouped_{kind}_gemm_nt_{form}_epilogue")(*operands, st["groups"], st["d"], **extra)
        out = dict(d=st["d"])
        if st["z"] is not None:
            out["z"] = st["z"]
        return out
    dg.dg_epilogue_backward(st["dd"], st["z"], c["act"], st["dz"], st["dbias"], st["groups"])
    if form == "dense":
        dg.dg_bf16_gemm_nn(st["dz"], st["b"], None, st["da"])
        dg.dg_bf16_gemm_tn(st["dz"], st["a"], None, st["db"])
    else:
        dg.dg_m_grouped_bf16_gemm_nn_contiguous(st["dz"], st["b"], st["groups"], None, st["da"])
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(st["dz"], st["a"], st["ks"], None, st["db"])
    out = dict(da=st["da"], db=st["db"])
    if st["dbias"] is not None:
        out["dbias"] = st["dbias"]
    return out


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "combine": _plain_combine, "combine_backward": _plain_combine_backward,
            "linear": _plain_linear, "linear_backward": _plain_linear_backward}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("route", "combine", "combine_backward"):
        T, k, G, H = case["T"], case["k"], case["G"], case["H"]
        n = T * k * (0.8 if case["drop"] else 1.0)        # assignments that reach an expert here
        if op == "route":
            groups = G if case["m_max"] else _sorted_rows(T, k, G) + G
            row = H + H // 128 * 4 if case["fp8"] else 2 * H
            return dict(bytes=2 * T * H + n * row + 8 * T * k + 4 * groups, flops=0)
        if op == "combine":
            return dict(bytes=2 * n * H + (4 if case["residual"] else 2) * T * H + 8 * T * k, flops=2 * n * H)
        return dict(bytes=4 * n * H + 2 * T * H + 12 * T * k, flops=3 * n * H)
    M, N, K, G = case["M"], case["N"], case["K"], case["G"]
    # masked: about half of each expert's M rows are taken
    rows = M * G / 2 if case["form"] == "masked" else M
    wide = 1 if case.get("fp8") else 2
    if op == "linear":
        out = 2 * (1 + bool(case["residual"]) + bool(case["save"]))
        return dict(bytes=rows * K * wide + G * N * K * wide + rows * N * out + 4 * G * N * bool(case["bias"]),
                    flops=2 * rows * N * K)
    return dict(bytes=4 * rows * N + 4 * rows * K + 4 * G * N * K + 4 * G * N * bool(case["bias"]),
                flops=4 * rows * N * K)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        placed = _host_place(st["ids"], case)
        rows = torch.zeros((placed["slots"] + 1, case["H"]), dtype=torch.float64, device="cuda")
        where = torch.tensor(placed["where"], device="cuda", dtype=torch.long)
        x = st["x"].double()[torch.tensor(placed["token"], device="cuda", dtype=torch.long)]
        if not case["fp8"]:
            rows[where] = x
            return dict(pos=None, groups=None, rows=rows[:-1].reshape(st["rows"].shape), ks=None)
        top = x.reshape(len(where), -1, 128).abs().amax(-1)
        scale = torch.where(top > 0, torch.clamp(top / 448, min=TINY), torch.ones_like(top))
        rows[where] = (x.reshape(len(where), -1, 128) / scale[..., None]).reshape(x.shape)
        sf = torch.zeros((placed["slots"] + 1, case["H"] // 128), dtype=torch.float64, device="cuda")
        sf[torch.tensor(placed["padding"], device="cuda", dtype=torch.long)] = 1.0
        sf[where] = scale
        sf = sf[:-1].reshape(*st["rows"].shape[:-1], -1).movedim(-1, -2).contiguous()
        return dict(pos=None, groups=None, rows=rows[:-1].reshape(st["rows"].shape), sf=sf, ks=None)
    if op in ("combine", "combine_backward"):
        T, H = case["T"], case["H"]
        flat = st["rows"].reshape(-1, H)
        grad = op == "combine_backward"
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        d_rows = torch.zeros(flat.shape if grad else (0, H), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, case["k"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            here = torch.nonzero(st["pos"][:, j] >= 0)[:, 0]
            at = st["pos"][here, j].long()
            w = st["weights"][here, j].double()[:, None]
            if grad:
                d = st["dy"][here].double()
                d_rows[at] = w * d
                dw[here, j] = torch.linalg.vecdot(d, flat[at].double())
            else:
                y[here] += w * flat[at].double()
        if grad:
            return dict(d_rows=d_rows.reshape(st["rows"].shape), d_weights=dw)
        return y if st["residual"] is None else y + st["residual"].double()
    return _exact_linear(st) if op == "linear" else _exact_linear_backward(st)


def _host_place(ids, case):
    """Where each assignment goes, by walking the experts' lists on the host."""
    G, m_max, k = case["G"], case["m_max"], case["k"]
    lists = [[] for _ in range(G)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < G:
            lists[e].append(i)
    where, token, padding, at = [], [], [], 0
    for g, mine in enumerate(lists):
        if m_max:
            mine, at = mine[:m_max], g * m_max
        where += range(at, at + len(mine))
        token += [i // k for i in mine]
        if not m_max:
            end = at + -(-len(mine) // ALIGN) * ALIGN
            padding += range(at + len(mine), end)
            at = end
    slots = G * m_max if m_max else _sorted_rows(case["T"], k, G)
    return dict(where=where, token=token, padding=padding, slots=slots)


def _values(st):
    """Row and weight values in 64 bits."""
    c = st["case"]
    a, b = st["a"].double(), st["b"].double()
    if c.get("fp8"):
        a = a * st["sfa"].double().movedim(-2, -1).repeat_interleave(128, -1)
        b = b * st["sfb"].double().repeat_interleave(128, -2)[..., :c["N"], :].repeat_interleave(128, -1)
    return a.reshape(-1, c["K"]), b.reshape(c["G"], c["N"], c["K"])


def _expert_of_rows(st):
    c = st["case"]
    if c["form"] == "dense":
        return torch.zeros(c["M"], dtype=torch.long, device="cuda")
    if c["form"] == "contiguous":
        return st["groups"].long()
    r = torch.arange(c["M"], device="cuda")
    g = torch.arange(c["G"], device="cuda")[:, None]
    return torch.where(r[None] < st["groups"][:, None], g, torch.full_like(g, -1)).reshape(-1)


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


def _exact_linear(st):
    c = st["case"]
    a, b = _values(st)
    expert = _expert_of_rows(st)
    z = torch.zeros((a.shape[0], c["N"]), dtype=torch.float64, device="cuda")
    d = torch.zeros_like(z)
    for g in range(c["G"]):
        r = torch.nonzero(expert == g)[:, 0]
        v = torch.matmul(a[r], b[g].t())
        if st["bias"] is not None:
            v += st["bias"].double().reshape(c["G"], -1)[g]
        z[r] = v
        d[r] = _exact_act(v, c["act"])
        if st["residual"] is not None:
            d[r] += st["residual"].double().reshape(a.shape[0], -1)[r]
    out = dict(d=d.reshape(st["d"].shape))
    if st["z"] is not None:
        out["z"] = z.reshape(st["d"].shape)
    return out


def _exact_linear_backward(st):
    c = st["case"]
    a, b = _values(st)
    expert = _expert_of_rows(st)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    dbias = torch.zeros((c["G"], c["N"]), dtype=torch.float64, device="cuda")
    for g in range(c["G"]):
        r = torch.nonzero(expert == g)[:, 0]
        dz = st["dd"][r].double() * _exact_slope(st["z"][r].double(), c["act"])
        da[r] = torch.matmul(dz, b[g])
        db[g] = torch.matmul(dz.t(), a[r])
        dbias[g] = dz.sum(0)
    out = dict(da=da, db=db.reshape(st["b"].shape))
    if st["bias"] is not None:
        out["dbias"] = dbias.reshape(st["bias"].shape)
    return out
