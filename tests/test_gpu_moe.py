"""Sorting, dispatch, combine and their gradients on the GPU against plain CPU implementations.

Places are whole numbers and copies are copies, so both must match exactly, quantised codes and scales
too (the definition uses correctly rounded FP32 operations only).  Sums: a BF16 result is rounded once
(at most 2^-8 relative, 2^-9 of it the rounding) after FP32 additions of k terms (k 2^-23 of the sum of
the terms' magnitudes); a dot product of N terms in FP32 is within (N + 16) 2^-24 of that sum."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import moe_ref as ref

pytestmark = pytest.mark.gpu
SENTINEL = 0x5a


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _ids(T, k, G, seed, kind="uniform"):
    rng = np.random.default_rng(seed)
    if kind == "one":                     # every assignment to the last expert
        return np.full((T, k), G - 1, np.int32)
    if kind == "none":                    # nothing for this rank
        return np.where(rng.random((T, k)) < 0.5, -1, G).astype(np.int32)
    ids = rng.integers(0, G, (T, k))
    if kind == "away":                    # some outside [0, G), on both sides
        ids = rng.choice([-2 ** 31, -1, G, 2 ** 31 - 1, 0], (T, k), p=[.1, .1, .1, .1, .6]) + 0 * ids
        ids = np.where(ids == 0, rng.integers(0, G, (T, k)), ids)
    if kind == "skew":                    # a few experts take nearly everything
        ids = np.minimum((rng.random((T, k)) ** 4 * G).astype(np.int64), G - 1)
    return ids.astype(np.int32)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(n, value=77):
    return torch.full(n if isinstance(n, tuple) else (n,), value, dtype=torch.int32, device="cuda")


def _bf(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


SORTS = [(0, 3, 4, "uniform"), (1, 1, 1, "uniform"), (1, 8, 32, "uniform"), (7, 3, 5, "away"), (64, 8, 256, "uniform"),
         (1021, 3, 7, "away"), (2048, 1, 1, "one"), (2049, 1, 63, "skew"), (700, 4, 65, "one"), (513, 4, 1024, "uniform"),
         (4096, 8, 128, "skew"), (1500, 2, 9, "none"), (40000, 8, 33, "uniform")]


@pytest.mark.parametrize("T,k,G,kind", SORTS)
def test_sort_contiguous(T, k, G, kind):
    ids = _ids(T, k, G, T + k + G, kind)
    R = dg.moe_sorted_rows(T, k, G)
    assert R == ref.sorted_rows(T, k, G)
    pos, m, ks = _i32((T, k)), _i32(R), _i32(G)
    dg.dg_moe_sort_contiguous(_cuda(ids), G, pos, m, ks)
    want = ref.sort_contiguous(ids, G, R)
    for got, w, name in zip((pos, m, ks), want, ("pos", "m_indices", "ks")):
        assert np.array_equal(got.cpu().numpy(), w), name


@pytest.mark.parametrize("T,k,G,kind", [(300, 4, 6, "uniform"), (3000, 2, 5, "skew")])
@pytest.mark.parametrize("short", [128, 640])
def test_sort_contiguous_into_too_few_rows(T, k, G, kind, short):
    """Assignments past the capacity are dropped, the segments cut there."""
    ids = _ids(T, k, G, 5, kind)
    pos, m, ks = _i32((T, k)), _i32(short), _i32(G)
    dg.dg_moe_sort_contiguous(_cuda(ids), G, pos, m, ks)
    wp, wm, wk = ref.sort_contiguous(ids, G, 1 << 16)
    wp = np.where(wp < short, wp, -1)
    start = np.cumsum(wk) - wk
    assert np.array_equal(pos.cpu().numpy(), wp) and np.array_equal(m.cpu().numpy(), wm[:short])
    assert np.array_equal(ks.cpu().numpy(), np.clip(short - start, 0, wk))


@pytest.mark.parametrize("T,k,G,kind", SORTS)
@pytest.mark.parametrize("m_max", [1, 100, 4096])
def test_sort_masked(T, k, G, kind, m_max):
    ids = _ids(T, k, G, T + k, kind)
    pos, counts = _i32((T, k)), _i32(G)
    dg.dg_moe_sort_masked(_cuda(ids), G, m_max, pos, counts)
    wp, wc = ref.sort_masked(ids, G, m_max)
    assert np.array_equal(pos.cpu().numpy(), wp) and np.array_equal(counts.cpu().numpy(), wc)


def _placed(T, k, G, seed, kind, m_max=0):
    ids = _ids(T, k, G, seed, kind)
    if m_max:
        pos, _ = ref.sort_masked(ids, G, m_max)
        return pos, None, G * m_max
    R = ref.sorted_rows(T, k, G)
    pos, m, _ = ref.sort_contiguous(ids, G, R)
    return pos, m, R


WIDTHS = [1, 7, 8, 136, 1000, 1023, 1032, 2056]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T,k,G,kind,m_max", [(1, 1, 1, "uniform", 0), (37, 3, 5, "away", 0), (300, 2, 4, "skew", 0),
                                              (37, 9, 5, "uniform", 20), (5, 2, 3, "none", 0)])
def test_dispatch_bf16(H, T, k, G, kind, m_max):
    pos, m, R = _placed(T, k, G, H + T, kind, m_max)
    x = _bf((T, H), 3)
    out = torch.full((R, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_dispatch_bf16(x.cuda(), _cuda(pos), None if m is None else _cuda(m), out)
    want = torch.full((R, H), float("nan"), dtype=torch.bfloat16)
    if m is not None:
        want[torch.from_numpy(m == -1)] = 0
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = x[t]
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("H", [128, 384, 1024, 1152, 7168])
@pytest.mark.parametrize("T,k,G,kind,m_max", [(1, 1, 1, "uniform", 0), (37, 3, 5, "away", 0), (200, 2, 4, "skew", 0),
                                              (37, 9, 5, "uniform", 20)])
def test_dispatch_fp8(ue8m0, H, T, k, G, kind, m_max):
    pos, m, R = _placed(T, k, G, H + T, kind, m_max)
    x = _bf((T, H), 4, 3.0)
    # blocks of every kind: zeros, subnormal and tiny values, large ones, one outlier, ties
    x[0, :128] = 0
    if H > 128:
        x[0, 128:256] = torch.tensor([1e-40, -1e-39, 3e-38, 0.0] * 32).to(torch.bfloat16)
        x[T - 1, 256:384] = torch.tensor([3e38, -1e30, 1.0, 448.0] * 32).to(torch.bfloat16)
    if H >= 1024:
        x[T // 2, 512:640] = torch.arange(128).to(torch.bfloat16) / 16      # many ties of the E4M3 grid
        x[T // 2, 640] = 1e6
    group = m_max or R
    lead = (G, m_max) if m_max else (R,)
    codes = torch.full((*lead, H), SENTINEL, dtype=torch.uint8, device="cuda")
    entries = (H + 511) // 512 if ue8m0 else H // 128
    sf_shape = (*lead[:-1], entries, lead[-1])
    sf = torch.full(sf_shape, SENTINEL, dtype=torch.int32, device="cuda") if ue8m0 else \
        torch.full(sf_shape, 0.25, device="cuda")
    dg.dg_moe_dispatch_fp8(x.cuda(), _cuda(pos), None if m is None else _cuda(m), codes, sf)
    qc, qs, qe = ref.quantise(x.float().numpy(), ue8m0)
    want_c = np.full((R, H), SENTINEL, np.uint8)
    if ue8m0:
        pad = np.full((T, 4 * entries - H // 128), 127, np.int64)
        b = np.concatenate([qe, pad], 1).reshape(T, entries, 4)
        rows_sf = (b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24).astype(np.uint32).view(np.int32)
        want_s, clear = np.full((R, entries), SENTINEL, np.int32), 0x7f7f7f7f
    else:
        rows_sf, want_s, clear = qs, np.full((R, entries), 0.25, np.float32), 1.0
    if m is not None:
        want_c[m == -1], want_s[m == -1] = 0, clear
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want_c[pos[t, j]], want_s[pos[t, j]] = qc[t], rows_sf[t]
    got_s = sf.cpu().numpy().reshape(-1, entries, group).transpose(0, 2, 1).reshape(R, entries)
    assert np.array_equal(codes.cpu().numpy().reshape(R, H), want_c)
    assert np.array_equal(got_s.view(np.int32), want_s.view(np.int32))


@pytest.mark.parametrize("ue8m0", [False, True])
def test_dispatch_fp8_marks_blocks_that_are_not_finite(ue8m0):
    """A block with a NaN or an infinity is not finite after dequantising, its neighbours are untouched by it."""
    x = _bf((2, 512), 6)
    x[0, 130], x[1, 300] = float("nan"), float("-inf")
    codes = torch.zeros((128, 512), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((1, 128), dtype=torch.int32, device="cuda") if ue8m0 else torch.zeros((4, 128), device="cuda")
    dg.dg_moe_dispatch_fp8(x.cuda(), _cuda(np.array([[5], [9]], np.int32)), None, codes, sf)
    if ue8m0:
        e = (sf.cpu().numpy().view(np.uint32)[0][:, None] >> np.array([0, 8, 16, 24])) & 255
        s = np.where(e == 255, np.nan, np.ldexp(1.0, e.astype(int) - 127))
    else:
        s = sf.cpu().numpy().T.astype(np.float64)
    v = codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(128, 4, 128)
    with np.errstate(all="ignore"):
        v = v * s[:, :, None]
    bad = ~np.isfinite(v)
    assert bad[5, 1].any() and bad[9, 2].any()
    assert bad[5, 1, 2] and bad[9, 2, 44]                     # the elements themselves
    bad[5, 1] = bad[9, 2] = False
    assert not bad.any()


def _poisoned(R, N, pos, seed):
    """Rows of which only those some token reads are finite."""
    rows = torch.full((R, N), float("nan"), dtype=torch.bfloat16)
    used = torch.from_numpy(np.unique(pos[pos >= 0]).astype(np.int64))
    rows[used] = _bf((len(used), N), seed)
    return rows


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("T,k,G,kind,m_max", [(1, 1, 1, "uniform", 0), (37, 3, 5, "away", 0), (130, 8, 4, "skew", 0),
                                              (37, 9, 5, "uniform", 20), (5, 2, 3, "none", 0)])
def test_combine(N, weighted, residual, T, k, G, kind, m_max):
    pos, _, R = _placed(T, k, G, N + T, kind, m_max)
    rows = _poisoned(R, N, pos, 7)
    w = np.random.default_rng(8).random((T, k)).astype(np.float32) - 0.3 if weighted else None
    res = _bf((T, N), 9) if residual else None
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    shaped = rows.reshape(G, m_max, N) if m_max else rows
    dg.dg_moe_combine(shaped.cuda(), _cuda(pos), None if w is None else _cuda(w), None if res is None else res.cuda(), y)
    want, mag = ref.combine(rows.float().numpy(), pos, w, None if res is None else res.float().numpy())
    err = np.abs(y.cpu().double().numpy() - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -23 * mag)


def test_combine_skips_places_outside_the_rows():
    rows = _bf((128, 64), 1)
    pos = np.array([[0, 128, -1], [2 ** 31 - 1, -2 ** 31, 127]], np.int32)
    y = torch.empty((2, 64), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(rows.cuda(), _cuda(pos), None, None, y)
    assert torch.equal(y.cpu(), rows[[0, 127]])
    out = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_dispatch_bf16(rows[:2].cuda(), _cuda(pos), None, out)
    want = torch.zeros((128, 64), dtype=torch.bfloat16)
    want[0], want[127] = rows[0], rows[1]
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("N", WIDTHS + [4104])
@pytest.mark.parametrize("T,k,G,kind,m_max", [(1, 1, 1, "uniform", 0), (37, 3, 5, "away", 0), (130, 8, 4, "skew", 0),
                                              (37, 9, 5, "uniform", 20), (5, 2, 3, "none", 0)])
def test_combine_backward(N, T, k, G, kind, m_max):
    pos, m, R = _placed(T, k, G, N + T, kind, m_max)
    rows = _poisoned(R, N, pos, 10)
    w = np.random.default_rng(11).random((T, k)).astype(np.float32) - 0.3
    dy = _bf((T, N), 12)
    d_rows = torch.full((R, N), float("inf"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    dg.dg_moe_combine_backward(dy.cuda(), rows.cuda(), _cuda(pos), _cuda(w), None if m is None else _cuda(m), d_rows, dw)
    want, want_w, mag = ref.combine_backward(dy.float().numpy(), rows.float().numpy(), pos, w)
    got = d_rows.cpu().double().numpy()
    for r in range(R):
        if r in want:
            assert np.all(np.abs(got[r] - want[r]) <= 2.0 ** -8 * np.abs(want[r]) + 2.0 ** -130), r
        elif m is not None and m[r] == -1:
            assert np.all(got[r] == 0), r
        else:
            assert np.all(np.isposinf(got[r])), r                       # untouched
    assert np.all(np.abs(dw.cpu().numpy() - want_w) <= (N + 16) * 2.0 ** -24 * mag)
    # without the weights' gradient (and without rows) the row gradients are the same
    again = torch.full((R, N), float("inf"), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine_backward(dy.cuda(), None, _cuda(pos), _cuda(w), None if m is None else _cuda(m), again, None)
    assert torch.equal(again.view(torch.int16), d_rows.view(torch.int16))


def test_gradients_against_differences():
    """Small whole numbers keep every value exact in BF16, so differences of <dY, combine> are the gradients."""
    T, k, G, N = 6, 3, 4, 16
    pos, m, R = _placed(T, k, G, 2, "away")
    rng = np.random.default_rng(3)
    rows = torch.from_numpy(rng.integers(-2, 3, (R, N)).astype(np.float32)).to(torch.bfloat16)
    dy = torch.from_numpy(rng.integers(-2, 3, (T, N)).astype(np.float32)).to(torch.bfloat16)
    w = rng.choice([0.5, 1.0, 2.0], (T, k)).astype(np.float32)

    def loss(rows, w):
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        dg.dg_moe_combine(rows.cuda(), _cuda(pos), _cuda(w), None, y)
        return float((y.cpu().double() * dy.double()).sum())

    d_rows = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((T, k), device="cuda")
    dg.dg_moe_combine_backward(dy.cuda(), rows.cuda(), _cuda(pos), _cuda(w), _cuda(m), d_rows, dw)
    at = loss(rows, w)
    for r in sorted(set(pos[pos >= 0]))[:8]:
        for c in (0, 5, N - 1):
            moved = rows.clone()
            moved[r, c] += 1
            assert loss(moved, w) - at == float(d_rows[r, c]), (r, c)
    for t in range(T):
        for j in range(k):
            moved = w.copy()
            moved[t, j] += 1
            assert loss(rows, moved) - at == float(dw[t, j]), (t, j)


def test_dispatch_gradient_is_the_unweighted_combine():
    """<dRows, dispatch(X)> = <combine(dRows), X>, exactly, for small whole numbers."""
    T, k, G, H = 20, 4, 5, 40
    pos, m, R = _placed(T, k, G, 4, "away")
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(-3, 4, (T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    dr = torch.from_numpy(rng.integers(-3, 4, (R, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_dispatch_bf16(x, _cuda(pos), _cuda(m), rows)
    dx = torch.empty_like(x)
    dg.dg_moe_combine(dr, _cuda(pos), None, None, dx)
    assert float((rows.double() * dr.double()).sum()) == float((dx.double() * x.double()).sum())


def test_another_stream_and_graph_replays():
    """Sort, dispatch and combine captured once on a side stream: every replay matches the eager calls on
    new contents, with eager work between the replays."""
    T, k, G, H = 900, 4, 16, 264
    R = dg.moe_sorted_rows(T, k, G)
    x, w = _bf((T, H), 1).cuda(), torch.rand((T, k), device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")

    def buffers():
        return [_i32((T, k)), _i32(R), _i32(G), torch.zeros((R, H), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")]

    def calls(b):
        dg.dg_moe_sort_contiguous(ids, G, b[0], b[1], b[2])
        dg.dg_moe_dispatch_bf16(x, b[0], b[1], b[3])
        dg.dg_moe_combine(b[3], b[0], w, x, b[4])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured = buffers()
    with torch.cuda.stream(side):
        calls(captured)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(captured)
    for seed in range(4):
        ids.copy_(_cuda(_ids(T, k, G, seed, "skew")))
        torch.cuda.synchronize()
        eager = buffers()
        calls(eager)
        torch.cuda.synchronize()
        captured[3].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), seed


def test_rows_past_four_gigabytes():
    """Row and scale offsets past 32 bits: the last rows of a buffer of over 4 GiB (BF16, E4M3) are reached."""
    H = 7168
    R = ((1 << 32) // (2 * H) // 128 + 3) * 128
    x = _bf((3, H), 1).cuda()
    pos = torch.tensor([[R - 1], [R - 130], [0]], dtype=torch.int32, device="cuda")
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_dispatch_bf16(x, pos, None, rows)
    at = pos[:, 0].long()
    assert torch.equal(rows[at], x) and not rows[R - 129:R - 1].any() and not rows[1:100].any()
    y = torch.empty_like(x)
    dg.dg_moe_combine(rows, pos, None, None, y)
    assert torch.equal(y, x)
    d_rows, dw = torch.zeros_like(rows), torch.empty((3, 1), device="cuda")
    dg.dg_moe_combine_backward(x, rows, pos, None, None, d_rows, dw)
    assert torch.equal(d_rows[at], x)
    want = x.double().square().sum(1, keepdim=True)
    assert torch.all((dw.double() - want).abs() <= (H + 16) * 2.0 ** -24 * want)
    del rows, d_rows
    R *= 2
    pos = torch.tensor([[R - 1], [R - 130], [0]], dtype=torch.int32, device="cuda")
    codes = torch.zeros((R, H), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((H // 128, R), device="cuda")
    dg.dg_moe_dispatch_fp8(x, pos, None, codes, sf)
    qc, qs, _ = ref.quantise(x.float().cpu().numpy())
    at = pos[:, 0].long()
    assert np.array_equal(codes[at].cpu().numpy(), qc) and np.array_equal(sf[:, at].cpu().numpy().T, qs)


def test_an_earlier_error_is_not_this_calls():
    """An error that another call of the thread left in the runtime is neither reported nor cleared."""
    from moe_grouped_gemm_scales_amd.dg import lib     # its symbols include the HIP runtime it is linked to
    ids = _cuda(_ids(9, 2, 4, 1))
    pos, m, ks = _i32((9, 2)), _i32(1024), _i32(4)
    x = _bf((9, 64), 2).cuda()
    rows = torch.zeros((1024, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros((9, 2), device="cuda")
    db = torch.zeros(64, device="cuda")
    torch.cuda.synchronize()
    assert lib.hipSetDevice(99) != 0                    # no such device: refused by the runtime
    try:
        dg.dg_moe_sort_contiguous(ids, 4, pos, m, ks)
        dg.dg_moe_dispatch_bf16(x, pos, m, rows)
        dg.dg_moe_combine_backward(x, rows, pos, None, m, rows, dw)
        dg.dg_epilogue_backward(x, x, "silu", x, db)
    finally:
        left = lib.hipGetLastError()
    torch.cuda.synchronize()
    assert left != 0
