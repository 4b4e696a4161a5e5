"""The norm and its gradient on the GPU against plain implementations in 64 bits.

A BF16 result is off by its rounding, 2^-8 relative, an E4M3 code by 2^-4 (subnormal codes by half their step,
2^-10 of the scale).  In front of those stand FP32 sums: at most 64 additions in a lane, 4 within 16 lanes, 2
more in the wave, 16 over the waves, so 86 2^-24 of the sum of squares and half of that of its root: below 2^-18
relative.  Sums of products (the mean of g n, the weight's gradient over rows) are within 128 2^-24 = 2^-17 of the
sum of their terms' magnitudes for the rows tested here; 2^-16 holds the terms' own roundings too."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _bf(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def _weight(H, kind, seed):
    if kind == "none":
        return None
    w = 1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(seed))
    return w.to(torch.bfloat16) if kind == "bf16" else w


def _cuda(t):
    return None if t is None else t.cuda()


class Fenced:
    """A [T,H] output between two fences that a kernel must not touch (16-byte aligned, any H)."""

    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        self.fill = 0x5a
        size = torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((256 + n * size + 256,), self.fill, dtype=torch.uint8, device="cuda")
        self.t = self.raw[256:256 + n * size].view(dtype).reshape(shape)
        self.n = n * size

    def check(self):
        raw = self.raw.cpu()
        assert (raw[:256] == self.fill).all() and (raw[256 + self.n:] == self.fill).all()
        return self.t.cpu()


def _near(got, want, tol):
    """|got - want| <= tol; NaN nowhere."""
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"off by {float((off - tol).max())} more than allowed"


SHAPES = [(1, 1), (3, 7), (1, 8), (9, 127), (8, 128), (17, 500), (300, 511), (5, 512), (33, 520), (2, 1000), (7, 2048),
          (4, 2056), (130, 2303), (32, 7168), (3, 8192), (2, 8200), (2, 16384), (2, 20001), (1, 32765), (2, 32768)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("weight,residual", [("bf16", True), ("f32", True), ("none", False)])
def test_norm_bf16(T, H, weight, residual):
    x, r, w = _bf((T, H), 1, 2.0), _bf((T, H), 2) if residual else None, _weight(H, weight, 3)
    y, s = Fenced((T, H), torch.bfloat16), Fenced((T, H), torch.bfloat16)
    assert dg.dg_rms_norm(x.cuda(), _cuda(w), EPS, Y=y.t, residual=_cuda(r), S=s.t) is y.t
    ws, wy = ref.rms_norm(x, r, w, EPS)
    _near(s.check(), ws, 2 ** -8 * ws.abs())
    _near(y.check(), wy, 2 ** -8 * (1 + 2 ** -8) * wy.abs())


@pytest.mark.parametrize("T,H", [(1, 128), (9, 384), (33, 512), (64, 640), (7, 1664), (32, 7168), (1021, 1024), (3, 8320),
                                 (2, 32768)])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("both", [False, True])
def test_norm_e4m3(T, H, ue8m0, both):
    x, r, w = _bf((T, H), 4, 3.0), _bf((T, H), 5), _weight(H, "bf16", 6)
    if H > 128:
        w[128:256] = 0                                     # a block of zeros: scale 1
    q = Fenced((T, H), torch.uint8)
    words = -(-H // 512) if ue8m0 else H // 128
    sf = Fenced((words, T), torch.int32 if ue8m0 else torch.float32)
    y = Fenced((T, H), torch.bfloat16) if both else None
    dg.dg_rms_norm(x.cuda(), w.cuda(), EPS, Y=y.t if both else None, residual=r.cuda(), Q=q.t, sf=sf.t)
    _, wy = ref.rms_norm(x, r, w, EPS)
    top = wy.reshape(T, -1, 128).abs().amax(-1)
    scale = sf.check()
    if ue8m0:
        if H % 512:
            last = (scale[-1].long() & 0xffffffff) >> (8 * (H % 512 // 128))
            assert (last == 0x7f7f7f7f >> (8 * (H % 512 // 128))).all()     # blocks past H count as scale 1
        scale = ref.unpack_words(scale, H)
        full = scale[top > 0]
        least = top[top > 0] / 448
        assert (full >= least * (1 - 1e-5)).all() and (full <= 2 * least * (1 + 1e-5)).all()
    else:
        scale = scale.t().double()
        _near(scale, torch.where(top > 0, top / 448, torch.ones_like(top)), 2 ** -17 * scale)
    assert (scale[top == 0] == 1).all()
    _near(ref.e4m3_values(q.check(), scale), wy,
          2 ** -4 * (1 + 2 ** -8) * wy.abs() + 2 ** -10 * scale.repeat_interleave(128, 1))
    if both:
        _near(y.check(), wy, 2 ** -8 * (1 + 2 ** -8) * wy.abs())


def test_norm_e4m3_feeds_the_fp8_product():
    """Q and sf are A and sfa of dg_fp8_gemm_nt: the product of the kept values."""
    T, H, N = 37, 512, 256
    x = _bf((T, H), 7).cuda()
    w = (torch.randn((N, H), generator=torch.Generator().manual_seed(8)) * 2).to(torch.float8_e4m3fn)
    for ue8m0 in (False, True):
        q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        sf = torch.empty((1, T), dtype=torch.int32, device="cuda") if ue8m0 else torch.empty((4, T), device="cuda")
        sfb = torch.full((2, 1), 0x7f7f7f7f, dtype=torch.int32, device="cuda") if ue8m0 else torch.ones((2, 4), device="cuda")
        dg.dg_rms_norm(x, None, EPS, Q=q, sf=sf)
        D = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        (dg.dg_fp8_gemm_nt_ue8m0 if ue8m0 else dg.dg_fp8_gemm_nt)(q, sf, w.cuda(), sfb, None, D)
        scale = ref.unpack_words(sf.cpu(), H) if ue8m0 else sf.cpu().t()
        a = ref.e4m3_values(q.cpu(), scale)
        want, mag = a @ w.double().t(), a.abs() @ w.double().abs().t()
        _near(D.cpu(), want, 2 ** -8 * want.abs() + 2 ** -14 * mag)


def test_norm_in_place():
    """S over the residual, Y over X; S over X."""
    T, H = 65, 1000
    x, r = _bf((T, H), 9), _bf((T, H), 10)
    ws, wy = ref.rms_norm(x, r, None, EPS)
    a, b = x.cuda(), r.cuda()
    dg.dg_rms_norm(a, None, EPS, Y=a, residual=b, S=b)
    _near(b.cpu(), ws, 2 ** -8 * ws.abs())
    _near(a.cpu(), wy, 2 ** -8 * (1 + 2 ** -8) * wy.abs())
    a, b = x.cuda(), r.cuda()
    dg.dg_rms_norm(a, None, EPS, Y=b, residual=b, S=a)
    _near(a.cpu(), ws, 2 ** -8 * ws.abs())
    _near(b.cpu(), wy, 2 ** -8 * (1 + 2 ** -8) * wy.abs())


def test_norm_rows_that_are_not_finite():
    """A NaN or an infinity stays in its row; a row of zeros gives zeros."""
    T, H = 5, 256
    x = _bf((T, H), 11)
    x[1, 3], x[2, 200], x[3] = float("nan"), float("inf"), 0
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q, sf = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((2, T), device="cuda")
    dg.dg_rms_norm(x.cuda(), None, EPS, Y=y, Q=q, sf=sf)
    got, kept = y.cpu(), ref.e4m3_values(q.cpu(), sf.cpu().t())
    _, wy = ref.rms_norm(x, None, None, EPS)
    for t in (0, 4):
        _near(got[t], wy[t], 2 ** -8 * (1 + 2 ** -8) * wy[t].abs())
        assert torch.isfinite(kept[t]).all()
    assert torch.isnan(got[1]).all() and torch.isnan(kept[1]).all()
    assert torch.isnan(got[2, 200]) and not torch.isfinite(kept[2, 200])
    assert (got[3] == 0).all() and (kept[3] == 0).all()


@pytest.mark.parametrize("T,H", SHAPES + [(1025, 640), (3000, 131)])
@pytest.mark.parametrize("weight,past", [("bf16", True), ("f32", False), ("none", True)])
def test_norm_backward(T, H, weight, past):
    dy, s, w = _bf((T, H), 12), _bf((T, H), 13, 1.5), _weight(H, weight, 14)
    ds = _bf((T, H), 15) if past else None
    dx, dw = Fenced((T, H), torch.bfloat16), Fenced((H,), torch.float32)
    dg.dg_rms_norm_backward(dy.cuda(), s.cuda(), _cuda(w), EPS, dx.t, dw.t, dS=_cuda(ds))
    wx, ww, mx, mw = ref.rms_norm_backward(dy, s, w, EPS, ds)
    _near(dx.check(), wx, 2 ** -8 * wx.abs() + 2 ** -16 * mx)
    _near(dw.check(), ww, 2 ** -16 * mw)


@pytest.mark.parametrize("over", ["dy", "ds"])
def test_norm_backward_in_place(over):
    T, H = 70, 1536
    dy, s, ds = _bf((T, H), 16), _bf((T, H), 17), _bf((T, H), 18)
    a, b = dy.cuda(), ds.cuda()
    dx = a if over == "dy" else b
    dg.dg_rms_norm_backward(a, s.cuda(), None, EPS, dx, None, dS=b)
    wx, _, mx, _ = ref.rms_norm_backward(dy, s, None, EPS, ds)
    _near(dx.cpu(), wx, 2 ** -8 * wx.abs() + 2 ** -16 * mx)


def test_norm_backward_parts():
    """dX or dweight alone; no rows: the weight's gradient is zero."""
    T, H = 40, 300
    dy, s = _bf((T, H), 19).cuda(), _bf((T, H), 20).cuda()
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    dg.dg_rms_norm_backward(dy, s, None, EPS, dx, dw)
    x2, w2 = torch.empty_like(dy), torch.empty(H, device="cuda")
    dg.dg_rms_norm_backward(dy, s, None, EPS, x2, None)
    dg.dg_rms_norm_backward(dy, s, None, EPS, None, w2)
    assert torch.equal(dx, x2) and torch.equal(dw, w2)
    none = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    dg.dg_rms_norm_backward(none, none, None, EPS, none, dw)
    assert (dw == 0).all()
    assert dg.dg_rms_norm(none, None, EPS, Y=none) is none


def test_norm_replayed():
    """Captured on a side stream, replayed with new inputs between eager calls: each replay is the eager result."""
    T, H = 100, 768
    stream = torch.cuda.Stream()
    x, dy = _bf((T, H), 21).cuda(), _bf((T, H), 22).cuda()
    w = _weight(H, "bf16", 23).cuda()
    out = {n: torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for n in ("y", "dx")}
    q, sf = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((H // 128, T), device="cuda")
    dw = torch.empty(H, device="cuda")

    def step():
        dg.dg_rms_norm(x, w, EPS, Y=out["y"], Q=q, sf=sf)
        dg.dg_rms_norm_backward(dy, x, w, EPS, out["dx"], dw)

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in range(4):
            x.copy_(_bf((T, H), 30 + seed))
            dy.copy_(_bf((T, H), 40 + seed))
            for t in (*out.values(), q, sf, dw):
                t.zero_()
            graph.replay()
            stream.synchronize()
            got = [t.clone() for t in (*out.values(), q, sf, dw)]
            step()
            stream.synchronize()
            for a, b in zip(got, (*out.values(), q, sf, dw)):
                assert torch.equal(a, b)


def test_norm_same_bits_every_time():
    T, H = 2500, 1000
    dy, s = _bf((T, H), 24).cuda(), _bf((T, H), 25).cuda()
    runs = []
    for _ in range(3):
        dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
        dg.dg_rms_norm_backward(dy, s, None, EPS, dx, dw)
        runs.append((dx, dw))
    for dx, dw in runs[1:]:
        assert torch.equal(dx, runs[0][0]) and torch.equal(dw, runs[0][1])


def test_norm_backward_of_the_most_rows():
    """2^31 - 1 rows of one element: s = 1 and dY = 1 give dX = 0 and a sum of ones (at most 512 partial sums, each
    exact, so 512 roundings of 2^-24)."""
    T = 2 ** 31 - 1
    ones = torch.ones((T, 1), dtype=torch.bfloat16, device="cuda")
    dx, dw = torch.full_like(ones, float("nan")), torch.empty(1, device="cuda")
    dg.dg_rms_norm_backward(ones, ones, None, 0.0, dx, dw)
    assert bool((dx == 0).all())
    assert abs(float(dw) - T) <= 2 ** -15 * T


@pytest.mark.parametrize("T,H", [(600, 2303), (600, 4096), (600, 2432), (513, 2049), (2100, 1025)])
def test_norm_of_prompts(T, H):
    """More than 512 rows of 1025 to 4096 elements: two chunks a lane; E4M3 where the width has whole blocks."""
    x, r, w = _bf((T, H), 51, 2.0), _bf((T, H), 52), _weight(H, "f32", 53)
    y = Fenced((T, H), torch.bfloat16)
    out = dict(Y=y.t)
    e4m3 = H % 128 == 0
    if e4m3:
        q, sf = Fenced((T, H), torch.uint8), Fenced((H // 128, T), torch.float32)
        out |= dict(Q=q.t, sf=sf.t)
    dg.dg_rms_norm(x.cuda(), w.cuda(), EPS, residual=r.cuda(), **out)
    _, wy = ref.rms_norm(x, r, w, EPS)
    _near(y.check(), wy, 2 ** -8 * (1 + 2 ** -8) * wy.abs())
    if e4m3:
        scale = sf.check().t().double()
        top = wy.reshape(T, -1, 128).abs().amax(-1)
        _near(scale, top / 448, 2 ** -17 * scale)
        _near(ref.e4m3_values(q.check(), scale), wy,
              2 ** -4 * (1 + 2 ** -8) * wy.abs() + 2 ** -10 * scale.repeat_interleave(128, 1))


@pytest.mark.parametrize("T,H", [(600, 2303), (2100, 4096), (700, 7168), (600, 8200), (300, 20001), (520, 32768), (2100, 1025)])
@pytest.mark.parametrize("past", [True, False])
def test_norm_backward_of_prompts(T, H, past):
    """Teams of 512 lanes and of 1024 over several turns, and the weight's gradient kept in LDS from turn to turn."""
    dy, s, w = _bf((T, H), 54), _bf((T, H), 55, 1.5), _weight(H, "bf16", 56)
    ds = _bf((T, H), 57) if past else None
    dx, dw = Fenced((T, H), torch.bfloat16), Fenced((H,), torch.float32)
    dg.dg_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), EPS, dx.t, dw.t, dS=_cuda(ds))
    wx, ww, mx, mw = ref.rms_norm_backward(dy, s, w, EPS, ds)
    _near(dx.check(), wx, 2 ** -8 * wx.abs() + 2 ** -16 * mx)
    _near(dw.check(), ww, 2 ** -16 * mw)
