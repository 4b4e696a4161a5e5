"""8-bit checkpoints and the backward pass that reads them, on the GPU against plain implementations in 64 bits.

Dividing by a power of two is exact, so codes and scales must be equal, and restored values too (BF16 holds a
code times a power of two).  Backward: BF16 results are rounded to 2^-8; the slopes and activations are FP32
with hardware exponentials and reciprocals (1 ulp each, arguments rounded to 2^-24: below 2^-19 of a slope's terms, which
are below 1.2, and 2^-15 relative of an activation for |z| up to 12); sums over at most 512 rows are within 2^-17
of the sum of their terms' magnitudes."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import layer_ref as ref
from tests.test_gpu_norm import Fenced, _bf, _cuda, _near

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _special(M, N, seed):
    """Blocks of every kind: zeros, tiny, huge, at the edges of a scale, ties of the code's grid."""
    x = _bf((M, N), seed, 2.0)
    x[0] = 0
    if M > 2 and N >= 100:
        x[1, :8] = torch.tensor([448.0, -448, 17, 1.0625, 1.1875, -1.3125, 2.0 ** -9, 2.0 ** -10]).to(torch.bfloat16)
        x[1, 8:100] = 0
        x[2, :100] = torch.tensor([450.0] + [0.0] * 99).to(torch.bfloat16)
    if M > 6 and N >= 300:
        x[3, :128] = torch.arange(128).to(torch.bfloat16) / 16
        x[3, 128:256] = torch.tensor([3.3e38, -1e30, 1.0, 0.0] * 32).to(torch.bfloat16)
        x[4, :128] = torch.tensor([1e-40, -9e-41, 3e-38, 0.0] * 32).to(torch.bfloat16)
        x[4, 128:256] = torch.tensor([4.6e-41, 0.0] * 64).to(torch.bfloat16)
        x[5, :128] = torch.tensor([1.2e-36, 5e-39] * 64).to(torch.bfloat16)
    return x


def _indices(M, seed):
    """Rows of two experts, padding (-1) and rows past the segments (-2)."""
    g = torch.Generator().manual_seed(seed)
    m = torch.randint(-2, 2, (M,), generator=g).to(torch.int32)
    m[0] = 0
    return m


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 100), (4, 127), (7, 128), (9, 129), (8, 300), (33, 520), (64, 1000), (17, 2112), (3, 4100)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("grouped", [False, True])
def test_keep_and_restore(M, N, grouped):
    x, m = _special(M, N, M + N), _indices(M, N) if grouped else None
    codes, scales = Fenced((M, N), torch.uint8), Fenced((M, -(-N // 128)), torch.uint8)
    assert dg.dg_checkpoint_fp8(x.cuda(), codes.t, scales.t, _cuda(m)) is codes.t
    v, e = ref.keep(x, m)
    want = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    if m is not None:
        e[m < -1], want[m < -1] = 0x5a, 0x5a                      # untouched
    assert torch.equal(scales.check(), e) and torch.equal(codes.check(), want)
    back = Fenced((M, N), torch.bfloat16)
    dg.dg_checkpoint_restore(codes.t, scales.t, back.t, _cuda(m))
    values = ref.kept_values(want, e)
    kept = back.check()
    if m is not None:
        assert (kept[m < -1].contiguous().view(torch.uint8) == 0x5a).all() and (kept[m == -1] == 0).all()
        values, kept = values[m >= 0], kept[m >= 0]
    normal = values.abs() >= 2.0 ** -126
    assert torch.equal(kept.double()[normal], values[normal])
    _near(kept.double()[~normal], values[~normal], torch.full((), 2.0 ** -134, dtype=torch.float64))


def test_keep_marks_blocks_that_are_not_finite():
    x = _bf((3, 384), 1)
    x[0, 130], x[1, 300] = float("nan"), float("-inf")
    codes, scales = torch.zeros((3, 384), dtype=torch.uint8, device="cuda"), torch.zeros((3, 3), dtype=torch.uint8, device="cuda")
    dg.dg_checkpoint_fp8(x.cuda(), codes, scales)
    assert scales.cpu()[0, 1] == 255 and scales.cpu()[1, 2] == 255 and int((scales.cpu() == 255).sum()) == 2
    back = dg.dg_checkpoint_restore(codes, scales, torch.empty((3, 384), dtype=torch.bfloat16, device="cuda")).cpu()
    bad = torch.isnan(back)
    assert bad[0, 128:256].all() and bad[1, 256:].all() and int(bad.sum()) == 256


def _kept(M, N, seed):
    z = _special(M, N, seed)
    z = torch.where(z.abs() < 12, z, torch.zeros_like(z))
    v, e = ref.keep(z)
    codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, e, ref.kept_values(codes, e)


@pytest.mark.parametrize("M,N", SHAPES + [(300, 515), (512, 128)])
@pytest.mark.parametrize("act", ACTS)
def test_backward_dense(M, N, act):
    codes, e, z = _kept(M, N, M)
    dd = _bf((M, N), 3)
    dz, h, db = Fenced((M, N), torch.bfloat16), Fenced((M, N), torch.bfloat16), Fenced((N,), torch.float32)
    dg.dg_epilogue_backward_fp8(dd.cuda(), codes.cuda(), e.cuda(), act, dz.t, db.t, H=h.t)
    value, slope = ref.activation(z, act)
    want = dd.double() * slope
    _near(dz.check(), want, 2 ** -8 * want.abs() + 2 ** -18 * dd.double().abs())
    _near(h.check(), value, (2 ** -8 + 2 ** -15) * value.abs() + 2 ** -134)
    _near(db.check(), want.sum(0), 2 ** -17 * want.abs().sum(0) + 2 ** -18 * dd.double().abs().sum(0))


@pytest.mark.parametrize("N", [8, 130, 515, 1024])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_backward_contiguous(N, act):
    """Three experts, one without rows; segments with padding, rows past them left alone, whatever stands there."""
    counts, G, M = [130, 0, 77], 3, 512
    m = torch.full((M,), -2, dtype=torch.int32)
    m[:130], m[130:256], m[256:333], m[333:384] = 0, -1, 2, -1
    codes, e, z = _kept(M, N, 5)
    dd = _bf((M, N), 6)
    dd[m < 0] = float("nan")
    codes[m < 0] = 0x7f
    dz, h, db = Fenced((M, N), torch.bfloat16), Fenced((M, N), torch.bfloat16), Fenced((G, N), torch.float32)
    dg.dg_epilogue_backward_fp8(dd.cuda(), codes.cuda(), e.cuda(), act, dz.t, db.t, H=h.t, m_indices=m.cuda())
    value, slope = ref.activation(z, act)
    want = torch.where((m >= 0)[:, None], dd.double(), torch.zeros((), dtype=torch.float64)) * slope
    got_z, got_h, got_b, real = dz.check(), h.check(), db.check(), m >= 0
    _near(got_z[real], want[real], 2 ** -8 * want[real].abs() + 2 ** -18 * dd.double()[real].abs())
    _near(got_h[real], value[real], (2 ** -8 + 2 ** -15) * value[real].abs() + 2 ** -134)
    assert (got_z[m == -1] == 0).all() and (got_h[m == -1] == 0).all()
    for t in (got_z, got_h):
        assert (t[m == -2].contiguous().view(torch.uint8) == 0x5a).all()
    for g in range(G):
        mine = want[m == g]
        _near(got_b[g], mine.sum(0), 2 ** -17 * mine.abs().sum(0) + 2 ** -18 * dd.double()[m == g].abs().sum(0))
    assert sum(counts) == int(real.sum())


def test_backward_parts_and_in_place():
    M, N = 70, 300
    codes, e, _ = (t.cuda() if t.dtype == torch.uint8 else t for t in _kept(M, N, 7))
    dd = _bf((M, N), 8).cuda()
    dz, h, db = torch.empty_like(dd), torch.empty_like(dd), torch.empty(N, device="cuda")
    dg.dg_epilogue_backward_fp8(dd, codes, e, "gelu", dz, db, H=h)
    z2, h2, b2 = torch.empty_like(dd), torch.empty_like(dd), torch.empty(N, device="cuda")
    dg.dg_epilogue_backward_fp8(dd, codes, e, "gelu", z2, None)
    dg.dg_epilogue_backward_fp8(dd, codes, e, "gelu", None, None, H=h2)
    dg.dg_epilogue_backward_fp8(dd, codes, e, "gelu", None, b2)
    assert torch.equal(dz, z2) and torch.equal(h, h2) and torch.equal(db, b2)
    dg.dg_epilogue_backward_fp8(dd, codes, e, "gelu", dd, None)                     # dZ over dD
    assert torch.equal(dd, dz)
    none = dd[:0]
    dg.dg_epilogue_backward_fp8(none, codes[:0], e[:0], "gelu", none, db)
    assert (db == 0).all()
    dg.dg_checkpoint_fp8(none, codes[:0], e[:0])


@pytest.mark.parametrize("act", ACTS)
def test_backward_is_that_of_the_restored_values(act):
    """dg_epilogue_backward on the restored Z: the same dZ and bias gradient, bit for bit."""
    M, N = 384, 640
    z = _bf((M, N), 9, 2.0).cuda()
    codes, e = torch.empty((M, N), dtype=torch.uint8, device="cuda"), torch.empty((M, 5), dtype=torch.uint8, device="cuda")
    dg.dg_checkpoint_fp8(z, codes, e)
    back = dg.dg_checkpoint_restore(codes, e, torch.empty_like(z))
    dd = _bf((M, N), 10).cuda()
    a, b, db1, db2 = torch.empty_like(z), torch.empty_like(z), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dg.dg_epilogue_backward_fp8(dd, codes, e, act, a, db1)
    dg.dg_epilogue_backward(dd, back, act, b, db2)
    assert torch.equal(a, b) and torch.equal(db1, db2)


def test_checkpoint_replayed():
    M, N = 256, 520
    stream = torch.cuda.Stream()
    z, dd = _bf((M, N), 11).cuda(), _bf((M, N), 12).cuda()
    codes, e = torch.empty((M, N), dtype=torch.uint8, device="cuda"), torch.empty((M, 5), dtype=torch.uint8, device="cuda")
    dz, h, db = torch.empty_like(z), torch.empty_like(z), torch.empty(N, device="cuda")

    def step():
        dg.dg_checkpoint_fp8(z, codes, e)
        dg.dg_epilogue_backward_fp8(dd, codes, e, "silu", dz, db, H=h)

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in range(3):
            z.copy_(_bf((M, N), 20 + seed))
            graph.replay()
            got = [t.clone() for t in (codes, e, dz, h, db)]
            step()
            stream.synchronize()
            for a, b in zip(got, (codes, e, dz, h, db)):
                assert torch.equal(a, b)
