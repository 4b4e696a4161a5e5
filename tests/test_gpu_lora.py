"""Low-rank adapters beside a shared product on the GPU against a plain implementation in 64 bits.

D is rounded to BF16 (2^-8).  FP32 sums of K terms are within K 2^-24 of the sum of their magnitudes, those of the
adapters within (K + rank) 2^-24 and 2^-17 for low as two BF16; an activation has slopes up to 1.2 and an error
of its own below 2^-18 of its argument and 1."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import layer_ref as ref
from tests.test_gpu_norm import Fenced, _bf, _cuda, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _adapters(M, L, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "rows":                        # any, some without (also far outside)
        a = torch.randint(-1, L + 1, (M,), generator=g)
        a[a == L] = 2 ** 31 - 1
        return a.to(torch.int32)
    if kind == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    a = torch.empty(M, dtype=torch.int32)     # prompts of uneven lengths
    at = 0
    while at < M:
        n = int(torch.randint(1, max(2, M // 3), (1,), generator=g))
        a[at:at + n] = int(torch.randint(-1, L, (1,), generator=g))
        at += n
    return a


def _case(M, N, K, R, L, kind, seed=1):
    return dict(a=_bf((M, K), seed), b=_bf((N, K), seed + 1, K ** -0.5), down=_bf((L, R, K), seed + 2, K ** -0.5),
                up=_bf((L, N, R), seed + 3, R ** -0.5), adapter=_adapters(M, L, kind, seed + 4),
                scale=0.5 + torch.rand(L, generator=torch.Generator().manual_seed(seed + 5)))


def _run(c, D, scale=True, **extra):
    return dg.dg_bf16_gemm_nt_lora(*(c[n].cuda() for n in ("a", "b", "down", "up", "adapter")), D,
                                   scale=c["scale"].cuda() if scale else None, **extra)


def _tolerance(c, base, low):
    K, R = c["a"].shape[1], c["down"].shape[1]
    return K * 2 ** -24 * base + ((K + R) * 2 ** -24 + 2 ** -16) * low


CASES = [(1, 8, 64, 8, 1, "one"), (1, 1000, 256, 16, 4, "one"), (5, 33, 64, 8, 2, "rows"), (16, 640, 128, 16, 16, "rows"),
         (32, 1024, 512, 16, 32, "rows"), (33, 515, 192, 24, 3, "rows"), (64, 2112, 256, 64, 64, "rows"),
         (130, 640, 192, 256, 3, "rows"), (200, 1000, 320, 40, 2, "prompts"), (300, 515, 128, 24, 5, "prompts"),
         (512, 256, 1024, 96, 7, "rows"), (517, 2112, 512, 32, 9, "prompts"), (700, 1024, 512, 64, 8, "prompts"),
         (1030, 2048, 256, 8, 100, "rows"), (2100, 1536, 448, 128, 6, "prompts"), (2048, 4096, 128, 16, 4, "rows"),
         (40, 512, 256, 16, 3, "none")]


@pytest.mark.parametrize("M,N,K,R,L,kind", CASES)
def test_lora(M, N, K, R, L, kind):
    c = _case(M, N, K, R, L, kind, M)
    D = Fenced((M, N), torch.bfloat16)
    assert _run(c, D.t) is D.t
    want, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], c["scale"], None)
    _near(D.check(), want, 2 ** -8 * want.abs() + _tolerance(c, base, low))


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K,R,L,kind", [(17, 136, 128, 16, 5, "rows"), (300, 515, 128, 24, 5, "prompts")])
def test_lora_epilogue(act, M, N, K, R, L, kind):
    c = _case(M, N, K, R, L, kind, 3)
    bias, res = 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(9)), _bf((M, N), 10)
    D, Z = Fenced((M, N), torch.bfloat16), Fenced((M, N), torch.bfloat16)
    _run(c, D.t, scale=False, bias=bias.cuda(), activation=act, residual=res.cuda(), Z=Z.t)
    z, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], None, bias)
    tol = _tolerance(c, base, low)
    _near(Z.check(), z, 2 ** -8 * z.abs() + tol)
    want = ref.activation(z, act)[0] + res.double()
    _near(D.check(), want, 2 ** -8 * want.abs() + 1.2 * tol + 2 ** -18 * (1 + z.abs()))


@pytest.mark.parametrize("M,L,kind", [(48, 4, "rows"), (300, 3, "prompts"), (600, 40, "rows"), (600, 3, "prompts")])
def test_lora_keeps_requests_apart(M, L, kind):
    """An adapter, or a row, that is not finite shows in its own rows only."""
    N, K, R = 640, 128, 16
    c = _case(M, N, K, R, L, kind, 5)
    c["adapter"][:3] = torch.tensor([1, 0, 2])
    sound = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    _run(c, sound)
    bad = {k: v.clone() for k, v in c.items()}
    bad["down"][1, 2, 5], bad["up"][2, 7, 3] = float("inf"), float("nan")
    got = torch.empty_like(sound)
    _run(bad, got)
    others = (c["adapter"] != 1) & (c["adapter"] != 2)
    got, sound = got.cpu(), sound.cpu()
    assert torch.equal(got[others], sound[others])
    two = c["adapter"] == 2
    assert torch.isnan(got[two][:, 7]).all()
    keep = torch.arange(N) != 7
    assert torch.equal(got[two][:, keep], sound[two][:, keep])
    assert not torch.isfinite(got[c["adapter"] == 1]).all(1).any()
    bad = {k: v.clone() for k, v in c.items()}
    bad["a"][1, 4] = float("nan")
    got = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    _run(bad, got)
    rest = torch.arange(M) != 1
    assert torch.isnan(got[1]).all() and torch.equal(got.cpu()[rest], sound[rest])


def test_lora_without_adapters_is_the_plain_product():
    M, N, K = 100, 640, 256
    c = _case(M, N, K, 16, 2, "none", 6)
    D, P = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _run(c, D)
    want, base, _ = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], None, None)
    dg.dg_bf16_gemm_nt(c["a"].cuda(), c["b"].cuda(), None, P)
    for t in (D, P):
        _near(t.cpu(), want, 2 ** -8 * want.abs() + K * 2 ** -24 * base)
    none = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_gemm_nt_lora(none, c["b"].cuda(), c["down"].cuda(), c["up"].cuda(), c["adapter"][:0].cuda(), D[:0])


@pytest.mark.parametrize("M,N,K", [(24, 1024, 1024), (600, 768, 256)])
def test_lora_replayed(M, N, K):
    """Captured on a side stream, replayed with other rows and adapters between eager calls."""
    R, L = 16, 6
    stream = torch.cuda.Stream()
    c = {k: v.cuda() for k, v in _case(M, N, K, R, L, "rows", 7).items()}
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")

    def step():
        dg.dg_bf16_gemm_nt_lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], D, scale=c["scale"])

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for seed in range(4):
            c["a"].copy_(_bf((M, K), 20 + seed))
            c["adapter"].copy_(_adapters(M, L, "rows" if seed % 2 else "prompts", seed))
            D.zero_()
            graph.replay()
            got = D.clone()
            step()
            stream.synchronize()
            assert torch.equal(got, D)


def test_lora_on_two_streams():
    """Each stream has its own workspace: calls in turn on two streams do not disturb each other."""
    cs = [{k: v.cuda() for k, v in _case(200, 512, 256, 32, 5, "prompts", s).items()} for s in (11, 12)]
    alone = [torch.empty((200, 512), dtype=torch.bfloat16, device="cuda") for _ in cs]
    for c, D in zip(cs, alone):
        dg.dg_bf16_gemm_nt_lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], D, scale=c["scale"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    out = [[torch.empty_like(D) for _ in range(20)] for D in alone]
    for i in range(20):
        for c, s, o in zip(cs, streams, out):
            dg.dg_bf16_gemm_nt_lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], o[i], scale=c["scale"], stream=s)
    torch.cuda.synchronize()
    for D, o in zip(alone, out):
        for t in o:
            assert torch.equal(t, D)


@pytest.mark.parametrize("M,L,R", [(40, 3, 128), (40, 40, 8)])          # adapter after adapter, and gathered
def test_lora_low_past_bf16(M, L, R):
    """Where low is infinite D is what the formula gives; where it is finite, but past BF16's numbers (3.39e38), D is as
    near as elsewhere.  An infinity in up stays in its column of its adapter's rows."""
    N, K = 136, 64
    c = _case(M, N, K, R, L, "rows", 21)
    c["adapter"] = (torch.arange(M) % L).to(torch.int32)
    sound = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    _run(c, sound)
    c["a"] = c["a"].abs() + 2 ** -6                              # (no zero meets an infinity)
    c["down"][0, 3, 5] = float("inf")
    c["a"][:, 0] = 1
    c["down"][1] = 0
    c["down"][1, :, 0] = torch.tensor([1, -1, 1, -1, 1, 1, -1, -1]).repeat(R // 8)     # low: +-scale
    c["scale"][1] = 3.4e38
    c["up"][1] *= 2.0 ** -100
    D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    _run(c, D)
    want, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], c["scale"], None)
    got, first = D.cpu(), c["adapter"] == 0
    assert torch.equal(got[first].double(), want[first]) and torch.isinf(want[first]).all()
    _near(got[~first], want[~first], (2 ** -8 * want.abs() + _tolerance(c, base, low))[~first])
    c = _case(M, N, K, R, L, "rows", 21)
    c["adapter"] = (torch.arange(M) % L).to(torch.int32)
    c["up"][2, 7, 3] = float("inf")
    _run(c, D)
    got, mine = D.cpu(), c["adapter"] == 2
    assert not torch.isfinite(got[mine][:, 7]).any()
    got[mine, 7] = sound.cpu()[mine, 7]
    assert torch.equal(got, sound.cpu())


# tiles of the planner, and whether a wave's rows are gathered (many adapters, up to 16 sub-tiles of 16 x 16) or go
# adapter after adapter
STRUCTURES = [("256n256", 2560, 5120, 256, 24, 6, "prompts"), ("256n256", 2500, 5001, 256, 64, 40, "rows"),
              ("128n256", 3000, 2111, 1024, 64, 5, "prompts"), ("128n256", 3000, 2111, 1024, 24, 50, "rows"),
              ("128n128", 2049, 2111, 64, 8, 100, "rows"), ("128n128", 2049, 2111, 64, 136, 9, "prompts")]


@pytest.mark.parametrize("tile,M,N,K,R,L,kind", STRUCTURES)
@pytest.mark.parametrize("full", [False, True])
def test_lora_on_large_tiles(tile, M, N, K, R, L, kind, full):
    flags = dg.EPI_BIAS_F32 | dg.EPI_RESIDUAL | dg.EPI_Z | dg.ACTIVATIONS["silu"] << 12 if full else 0
    assert f"_m{tile}_" in dg.describe_config(dg.KIND_BF16 | dg.EPI_LORA | flags, M, N, K, 1, 0, 256)
    c = _case(M, N, K, R, L, kind, 31)
    D = Fenced((M, N), torch.bfloat16)
    if not full:
        _run(c, D.t)
        z, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], c["scale"], None)
        _near(D.check(), z, 2 ** -8 * z.abs() + _tolerance(c, base, low))
        return
    bias, res = 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(9)), _bf((M, N), 10)
    Z = Fenced((M, N), torch.bfloat16)
    _run(c, D.t, bias=bias.cuda(), activation="silu", residual=res.cuda(), Z=Z.t)
    z, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], c["scale"], bias)
    tol = _tolerance(c, base, low)
    _near(Z.check(), z, 2 ** -8 * z.abs() + tol)
    want = ref.activation(z, "silu")[0] + res.double()
    _near(D.check(), want, 2 ** -8 * want.abs() + 1.2 * tol + 2 ** -18 * (1 + z.abs()))


def _adapters_by_block(M, L, counts):
    """Block b of 16 rows has counts[b mod len(counts)] adapters, in turn over its rows; some of the rows have none."""
    row = torch.arange(M)
    n = torch.tensor(counts)[(row // 16) % len(counts)]
    a = (3 * (row // 16) + (row % 16) % n) % L
    a[row % 29 == 7] = -1
    return a.to(torch.int32)


@pytest.mark.parametrize("M,R", [(2048, 64), (2049, 16), (2100, 64), (4117, 136)])
@pytest.mark.parametrize("counts", [(2,), (1, 3, 2), (16, 1, 5)])
def test_lora_blocks_of_many_adapters(M, R, counts):
    """Blocks of 16 rows with 1 to 16 adapters on both sides of the row count from which a block has two workgroups,
    the second of which does every adapter but the first in turn."""
    N, K, L = 264, 192, 37
    c = _case(M, N, K, R, L, "none", 41)
    c["adapter"] = _adapters_by_block(M, L, counts)
    D = Fenced((M, N), torch.bfloat16)
    _run(c, D.t)
    want, base, low = ref.lora(c["a"], c["b"], c["down"], c["up"], c["adapter"], c["scale"], None)
    _near(D.check(), want, 2 ** -8 * want.abs() + _tolerance(c, base, low))
