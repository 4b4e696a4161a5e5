// Tile selection for the block-scaled FP8 GEMM kernels on MI355X.
//
// DeepGEMM picks block sizes per shape so that the grid fills the machine,
// including non-power-of-two widths such as 112 (launch article, section 2.2
// "non-standard block partitioning", and section 7).  The same idea is used
// here with a small cost model of gfx950: 256 CUs, 8 XCDs, 160 KB LDS per CU,
// 8192 dense FP8 FLOP/clk/CU at 2.4 GHz and ~8 TB/s of HBM.  Candidates are
// (tile, wave grid, LDS stages, split-K) tuples; the model charges each
// candidate its wave-quantised MFMA time, its operand traffic and a fixed
// per-tile cost, and the cheapest one wins.  DG_FORCE_CONFIG
// ("bm,bn,wm,wn,stages,splitk[,kstep[,variant[,nb,ne]]]", launches separated
// by ';') overrides the choice for tuning sweeps.
#include <algorithm>
#include <iterator>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "dg_internal.h"

namespace dg {
namespace {

constexpr double kClockHz = 2.4e9;
constexpr double kMfmaFlopPerClkCu = 8192.0;
constexpr double kHbmBytesPerS = 8.0e12;
constexpr double kCuLoadBytesPerS = 64.0 * kClockHz;   // one CU's share of L2 fabric
constexpr int kLdsBytes = 160 * 1024;

int round_up(int x, int m) { return (x + m - 1) / m * m; }

int vgpr_estimate(int tm, int tn) {
    // accumulators + A fragments + two B fragments + products + addressing
    return tm * tn * 4 + tm * 8 + 16 + tm * tn / 2 + 48;
}

int occupancy(const KernelConfig& c) {
    int lds = c.lds_bytes();
    int by_lds = kLdsBytes / std::max(lds, 1);
    int tm = c.bm / c.wm / 16, tn = c.bn / c.wn / 16;
    int v = round_up(vgpr_estimate(tm, tn), 8);
    int waves_per_simd = std::min(8, 512 / std::max(v, 8));
    int by_regs = waves_per_simd * 4 / (c.wm * c.wn);
    return std::max(1, std::min(by_lds, by_regs));
}

struct Estimate {
    double seconds;
    KernelConfig cfg;
};

double estimate(const Problem& p, const KernelConfig& c, int num_cus, double valid_rows) {
    const int mt = (p.kind == kMasked) ? (int)std::ceil(valid_rows / std::max(p.g, 1) / c.bm) * p.g
                                       : (p.rows + c.bm - 1) / c.bm * (p.kind == kKGrouped ? p.g : 1);
    const int nt = (p.n + c.bn - 1) / c.bn;
    const double tiles = (double)mt * nt * c.splitk;
    const int occ = occupancy(c);
    const double slots = (double)num_cus * occ;
    const double waves = std::ceil(tiles / slots);
    // K-grouped: a tile covers one group's share of K (taken as an even split)
    const double kspan = (double)p.k / c.splitk / (p.kind == kKGrouped ? std::max(p.g, 1) : 1);
    const double kblocks = kspan / 128.0;
    const int nw = c.wm * c.wn;
    const double waves_per_simd = std::max(1.0, occ * nw / 4.0);
    // Per-CU cycle counts of one tile (measured shape of the kernel on gfx950):
    //  * MFMA: 32 cycles per 16x16x128 step on each of 4 SIMDs, shared by the
    //    occ resident workgroups;
    //  * VALU: one FMA per output element per K block plus a scale product per
    //    sub-tile, 4 cycles per wave64 instruction; only part of it hides under
    //    the MFMAs of the same SIMD;
    //  * a fixed cost per LDS stage (barrier, first LDS reads) that a second
    //    wave per SIMD mostly hides.
    const double mfma_cyc = (double)c.bm * c.bn * kspan * 2.0 / kMfmaFlopPerClkCu * occ /
                            std::min(1.0, nw * occ / 4.0);
    const double valu_cyc = (double)c.bm * c.bn / 64.0 * kblocks * 1.3 * 4.0 / 4.0 * occ;
    const double compute_cyc = std::max(mfma_cyc, valu_cyc) + 0.35 * std::min(mfma_cyc, valu_cyc);
    const double stage_cyc = 900.0 / waves_per_simd * (kblocks / c.kstep);
    const double t_compute = (compute_cyc + stage_cyc) / kClockHz;
    // operand tiles mostly come from L2/MALL (they are shared between tiles);
    // the HBM bound of the whole launch is applied below
    const double t_load = ((c.sf == 4 ? 0.5 : 1.0) * c.bm + (c.sf == 2 || c.sf == 4 ? 0.5 : 1.0) * c.bn) * kspan /
                          (kCuLoadBytesPerS / occ);
    // pipeline fill, epilogue and scheduling per tile; split-K adds a round trip
    double t_fixed = 1.2e-6 + (c.splitk > 1 ? 1.0e-6 * c.splitk + c.bm * c.bn * 8.0 * c.splitk / kCuLoadBytesPerS : 0.0);
    double t = waves * (std::max(t_compute, t_load) + t_fixed);
    // whole-device floor: HBM traffic.  Row blocks that share a B column block
    // re-read it; they only hit in L2 when they run close together, which the
    // grouped tile order gives for large M (8 row blocks per sweep) but not for
    // a handful of row blocks spread over the whole grid.
    const double groups_b = (p.kind == kDense) ? 1.0 : p.g;
    const double rows_per_group = valid_rows / groups_b;
    const double b_reads = rows_per_group <= 512 ? std::ceil(rows_per_group / c.bm)
                                                 : std::max(1.0, std::ceil(rows_per_group / c.bm) / 8.0);
    const double b_row_bytes = (p.sf == 2 || p.sf == 4) ? p.k / 2.0 : (double)p.k;
    const double bytes = valid_rows * p.k + b_reads * groups_b * p.n * b_row_bytes +
                         valid_rows * p.n * (2.0 + 4.0 * p.has_c);
    t = std::max(t, bytes / kHbmBytesPerS);
    return t;
}

int dma_per_wave(const KernelConfig& c) {
    const int nw = c.wm * c.wn;
    const int rpi = 8 / c.kstep;
    const int na = c.sf == 4 ? c.bm / 16 : c.bm / rpi, nb = (c.sf == 2 || c.sf == 4) ? c.bn / 16 : c.bn / rpi;
    const int ns = c.sf == 3 ? 0 : (c.bm + 63) / 64 * c.kstep;
    const int nt = c.sf == 3 ? 0 : (c.sf == 2 || c.sf == 4 || c.kind == kKGrouped) ? (c.bn + 63) / 64 : c.kstep;
    return (na + nw - 1) / nw + (nb + nw - 1) / nw + (ns + nw - 1) / nw + (nt + nw - 1) / nw;
}

// Vector-memory instructions per wave per K block of variant 1 (A/sfa DMA
// share, one sfb DMA, two 16-byte B loads per 16-row sub-tile).
int unit_per_wave_v1(const KernelConfig& c) {
    const int nw = c.wm * c.wn;
    return (c.bm / 8 + nw - 1) / nw + ((c.bm + 63) / 64 + nw - 1) / nw + 1 + 2 * (c.bn / c.wn / 16);
}

// Mirrors the kernel's static_asserts, so a selected config always compiles.
bool valid(const KernelConfig& c, const Problem& p) {
    if (c.bm % (16 * c.wm) || c.bn % (16 * c.wn)) return false;
    if (c.ne > 0 && (c.nb < 0 || c.nb % 16 || c.nb >= c.ne || c.ne > p.n)) return false;
    // operands read K-outermost: power-of-two tiles through LDS, aligned rows
    auto kout_tile = [](int t, int w) { return (t == 64 || t == 128 || t == 256) && ((t / w) & (t / w - 1)) == 0; };
    if (c.b_kout && (!kout_tile(c.bn, c.wn) || p.n % 8 || (c.variant != 0 && c.variant != 6) || c.kstep != 1)) return false;
    if (c.a_kout && (!kout_tile(c.bm, c.wm) || p.rows % 8)) return false;
    // split-K: not where a row block makes two passes, K-grouped in BF16 only, and of the grouped
    // forms in variants 0 and 6 only
    if (c.splitk < 1 || (c.splitk > 1 && ((p.kind == kContiguous && c.bm > 128) || (p.kind == kKGrouped && p.sf != 3) ||
                                          (p.kind != kDense && c.variant != 0 && c.variant != 6))))
        return false;
    if (c.sf != p.sf) return false;
    // variant 4: variant 0 with A requested a K block ahead of B (two B slots, three A
    // slots), for FP8 operands with FP32 or UE8M0 scales and the M forms
    if (c.variant == 4 && (c.kstep != 1 || c.stages != 2 || c.sf == 2 || c.sf == 4 || p.kind == kKGrouped))
        return false;
    // variant 6: variant 0 with the split refill (FP8 operands with FP32 or UE8M0 scales,
    // or BF16; one K block a stage, an even number of n sub-tiles per wave)
    if (c.variant == 6 && (c.kstep != 1 || c.sf == 2 || c.sf == 4 ||
                           (c.bn / c.wn / 16) % 2 || c.bn / c.wn / 16 < 4))
        return false;
    if (c.sf && ((c.variant != 0 && c.variant != 4 && c.variant != 6) || c.kstep != 1)) return false;   // UE8M0, FP4: variant 0, one K block a stage
    if (p.kind == kKGrouped && ((c.sf && c.sf != 3) || (c.variant != 0 && c.variant != 6) || c.kstep != 1)) return false;   // K-grouped: the same
    if (c.variant < 0 || c.variant > 6) return false;
    int tm = c.bm / c.wm / 16, tn = c.bn / c.wn / 16;
    if (c.lds_bytes() > kLdsBytes) return false;
    if (c.bn > 256) return false;
    if (c.variant == 5) {
        // B in VGPRs (each wave its own columns), A through a ring of `stages` slots;
        // FP32 scales, one K block a slot, no split-K, the M forms
        const int nw = c.wm * c.wn;
        if (c.sf || c.kstep != 1 || c.splitk != 1 || c.wm != 1 || p.kind == kKGrouped) return false;
        if (c.bm % 64 || (c.bm / 8) % nw || c.bm / 64 + 1 > nw || c.stages < 3) return false;
        if (128 % (c.bn / nw) || tm % 4 || tm * tn > 32 || tn < 1) return false;
        if (p.kind == kContiguous && c.bm > 128) return false;   // one expert per row block
        return (c.bm / 8 / nw + 1 + 2 * tn) * 2 <= 63;           // vmcnt field (two K blocks of B ahead)
    }
    if (p.kind == kContiguous && 128 % c.bm != 0 && c.bm % 128 != 0) return false;
    // one expert per row block; 256-row blocks (both operands through LDS) make one
    // pass per expert of their two 128-row blocks
    if (p.kind == kContiguous && c.bm > 128 && !(c.bm == 256 && (c.variant == 0 || c.variant == 4 || c.variant == 6)))
        return false;
    if (c.variant != 0 && c.variant != 4 && c.variant != 6) {
        // waves along n only, one K block at a time, the whole K range of a
        // work item unrolled, B registers of stages - 1 blocks in flight
        if (c.wm != 1 || c.kstep != 1 || c.stages < 2) return false;
        if ((p.k / 128) % c.splitk || p.k / 128 / c.splitk > 64) return false;
        const int ub = 2 * (c.bn / c.wn / 16);
        const int nkb = p.k / 128 / c.splitk, pre = std::min(c.stages - 1, nkb);
        if (c.variant == 1 && unit_per_wave_v1(c) * (c.stages - 2) > 63) return false;
        if (c.variant == 2 && (ub * (c.stages - 2) > 63 || ub * pre > 63)) return false;
        if (c.variant == 3 && (ub * pre > 63 || c.bm * 128 + 256 > 78 * 1024)) return false;
        if (tm < 1 || tn < 1 || tm > 16 || tn > 4 || tm * tn > 32) return false;
        if (c.bm % 8) return false;
        return true;
    }
    if (c.kstep != 1 && c.kstep != 2) return false;
    if (c.bm % (8 / c.kstep) || c.bn % (8 / c.kstep) || c.stages < 2) return false;
    if (dma_per_wave(c) * (c.stages - 1) > 63) return false;   // vmcnt field
    if (c.variant == 6 && (dma_per_wave(c) + 1) * (c.stages - 1) > 63) return false;   // split groups round up
    // more than 32 sub-tiles per wave: only 4-wave groups without promotion (accumulators in AGPRs)
    const bool agpr_acc = (c.sf == 1 || c.sf == 3 || c.sf == 5) && c.wm * c.wn == 4;
    if (tm < 1 || tn < 1 || tm > 8 || tn > 8 || tm * tn > (agpr_acc ? 64 : 32)) return false;
    // uneven splits: one K block a stage, variants 0 and 6
    if (p.kind != kKGrouped && (c.kstep != 1 || c.variant == 4) && (p.k / 128) % (c.splitk * c.kstep)) return false;
    return p.kind == kKGrouped || p.k / 128 >= c.splitk;
}

// Configurations measured fastest on an MI355X (graph-replayed back-to-back
// launches, tile/wave/stage/split sweeps) for the shapes of the DeepGEMM
// launch article's benchmark tables; other shapes go through the model.
// Consecutive rows of one shape with column ranges [nb, ne) are launched in
// turn (none at present: 4096 x 7168 as 256 x 256 tiles over [0, 4096) then
// 256 x 192 over [4096, 7168) fills two whole rounds of 256 CUs instead of
// 1.75, yet measured the same as 448 tiles of 256 x 256, 459 us each: the
// part runs at its power limit there, so idle CUs in a partial round are not
// lost time).
struct Tuned {
    int kind, rows, n, k, g, has_c;
    int bm, bn, wm, wn, stages, splitk, kstep, variant;
    int nb, ne;
};
const Tuned kTuned[] = {
    {kDense, 64, 2112, 7168, 1, 0, 64, 64, 1, 4, 4, 7, 1, 2, 0, 0},
    {kDense, 128, 24576, 1536, 1, 0, 128, 96, 1, 6, 3, 1, 1, 3, 0, 0},
    {kDense, 128, 24576, 1536, 1, 1, 128, 96, 4, 2, 2, 1, 2, 0, 0, 0},
    // the large shapes: 256 x 256 with the split refill (variant 6): 426-434 us against
    // 449 us for the one-part refill and 447-465 us for 256 x 224 (512 tiles, two full
    // rounds); contiguous: 808 us against 862 us for the one-part refill (one box)
    {kDense, 4096, 7168, 16384, 1, 0, 256, 256, 4, 2, 2, 1, 1, 6, 0, 0},
    {kContiguous, -1, 4096, 7168, 4, 0, 256, 256, 4, 2, 2, 1, 1, 6, 0, 0},
    // the masked decode shape, B streamed: 128 x 128 on variant 0 with three stages
    // 17.47-17.58 us against 17.97-18.10 us for the producer variant with 128 x 112
    // (one box; before B was streamed the producer variant led, 20.6 against 20.4-21.7)
    {kMasked, 256, 7168, 2048, 4, 0, 128, 128, 4, 2, 3, 1, 1, 0, 0, 0},
    // K-grouped weight gradient of the contiguous workload (K: the row pitch of the
    // K-contiguous operands, 4 x 8192 tokens): 192 x 256 with two stages measured 2-4 %
    // under 128 x 256 with three (22 row tiles, the last one a third full); with the split
    // refill 1274-1280 us against 1310-1344 us
    {kKGrouped, 4096, 7168, 32768, 4, 0, 192, 256, 4, 2, 2, 1, 1, 6, 0, 0},
};

// Packed UE8M0 scales (one K block a stage; no promotion in the K loop).  The
// large shapes use 256 x 256 with the split refill (variant 6): 399-404 us against
// 411 us for four waves of 128 x 128 with accumulators in AGPRs; contiguous 739-746 us
// against 790 us for the four-wave tile and 845 us for it without the split (one box)
const Tuned kTunedE8[] = {
    {kDense, 64, 2112, 7168, 1, 0, 64, 64, 2, 2, 4, 7, 1, 0, 0, 0},
    {kDense, 128, 24576, 1536, 1, 0, 128, 96, 4, 2, 3, 1, 1, 0, 0, 0},
    // with C: 15.8 us against 16.7-16.8 us for the model's 128 x 128 with 2 x 4 waves (one box)
    {kDense, 128, 24576, 1536, 1, 1, 128, 96, 4, 2, 4, 1, 1, 0, 0, 0},
    {kDense, 4096, 7168, 16384, 1, 0, 256, 256, 4, 2, 2, 1, 1, 6, 0, 0},
    {kContiguous, -1, 4096, 7168, 4, 0, 256, 256, 4, 2, 2, 1, 1, 6, 0, 0},
    {kMasked, 256, 7168, 2048, 4, 0, 128, 128, 4, 2, 3, 1, 1, 0, 0, 0},
};

// FP8 x FP4 and FP4 x FP4 (variant 0; B, and for FP4 x FP4 also A, tiles are half
// the bytes of the FP8 ones, so 256 x 256 fits three LDS stages: measured 429 us
// (FP8 x FP4) and 403 us (FP4 x FP4) against 485 and 465 us with two, the K loop
// of the large tile being bound by how far ahead its loads are issued)
const Tuned kTunedF4[] = {
    {kDense, 64, 2112, 7168, 1, 0, 64, 64, 2, 2, 4, 7, 1, 0, 0, 0},
    {kDense, 128, 24576, 1536, 1, 0, 128, 96, 4, 2, 3, 1, 1, 0, 0, 0},
    {kDense, 4096, 7168, 16384, 1, 0, 256, 256, 4, 2, 3, 1, 1, 0, 0, 0},
    // contiguous: 256-row blocks with three stages, 849-854 us against 1100-1111 us
    // for 128 x 224 with four (one box)
    {kContiguous, -1, 4096, 7168, 4, 0, 256, 256, 4, 2, 3, 1, 1, 0, 0, 0},
    {kMasked, 256, 7168, 2048, 4, 0, 128, 128, 4, 2, 3, 1, 1, 0, 0, 0},
};

// FP4 x FP4: the FP8 x FP4 choices (contiguous: 724-728 us against 917-924 us for
// 128 x 256 with three stages)
const Tuned kTunedF4F4[] = {
    {kDense, 64, 2112, 7168, 1, 0, 64, 64, 2, 2, 4, 7, 1, 0, 0, 0},
    {kDense, 128, 24576, 1536, 1, 0, 128, 96, 4, 2, 3, 1, 1, 0, 0, 0},
    {kDense, 4096, 7168, 16384, 1, 0, 256, 256, 4, 2, 3, 1, 1, 0, 0, 0},
    {kContiguous, -1, 4096, 7168, 4, 0, 256, 256, 4, 2, 3, 1, 1, 0, 0, 0},
    {kMasked, 256, 7168, 2048, 4, 0, 128, 128, 4, 2, 3, 1, 1, 0, 0, 0},
};

// BF16 x BF16 (k here is the row length in bytes, 2 x K).  A 128-byte K block is
// 64 elements, half the MFMA time of an FP8 one, so the loads' lead matters more:
// variant 4 (A one K block further ahead) 794 us against 865 us for variant 0; the split
// refill with 256 x 256 812-816 us against 819-839 us for variant 4 with 256 x 224
const Tuned kTunedBF16[] = {
    {kDense, 4096, 7168, 32768, 1, 0, 256, 256, 4, 2, 2, 1, 1, 6, 0, 0},
};

std::vector<KernelConfig> tuned(const Problem& p, int num_cus, const KernelConfig& base) {
    std::vector<KernelConfig> out;
    if (num_cus != 256) return out;       // measured on the full 256-CU part
    // FP4 x FP4 starts from the FP8 x FP4 table (same structure, A half the bytes)
    const Tuned* first = p.sf == 3 ? std::begin(kTunedBF16) : p.sf == 4 ? std::begin(kTunedF4F4)
                       : p.sf == 2 ? std::begin(kTunedF4) : p.sf ? std::begin(kTunedE8) : std::begin(kTuned);
    const Tuned* last = p.sf == 3 ? std::end(kTunedBF16) : p.sf == 4 ? std::end(kTunedF4F4)
                      : p.sf == 2 ? std::end(kTunedF4) : p.sf ? std::end(kTunedE8) : std::end(kTuned);
    for (const Tuned* it = first; it != last; ++it) {
        const Tuned& t = *it;
        if (t.kind != p.kind || t.n != p.n || t.k != p.k || t.g != p.g || t.has_c != p.has_c) continue;
        if (t.rows >= 0 && t.rows != p.rows) continue;
        if (t.rows < 0 && p.rows < 4096) continue;   // contiguous: any large token count
        KernelConfig c = base;
        c.bm = t.bm; c.bn = t.bn; c.wm = t.wm; c.wn = t.wn;
        c.stages = t.stages; c.splitk = t.splitk; c.kstep = t.kstep; c.variant = t.variant;
        c.nb = t.nb; c.ne = t.ne;
        out.push_back(c);
    }
    return out;
}

// The products with a fused epilogue and the BF16 NN and TN products choose among
// these structures by the time that a sum of measured parts gives them.  A CU
// that gets t tiles (splits of K included) in b batches of at most per_cu takes
//
//   one tile at a time:   b * (start + K blocks * us)
//   several at a time:    start * (1 + 1.5 (b - 1)) + K blocks * max(b * us, t * us_full)
//
// with us the time of one 128-byte K block while a tile has the CU to itself, us_full
// that per tile with the CU full, and start = 1.1 + 2.3 * (tile area / 128^2) us for
// the first loads and the epilogue.  A split of K adds its hand-off, 0.6 us, and 2.7 us
// per 10^6 FP32 partials.  The figures are fitted to 1420 launches of 59 shapes (1 to
// 17408 rows, BF16 and FP8, every form) on an MI355X; over these and 11 more the choice takes
// 2.0 % longer than the fastest structure in the geometric mean (a sum without start,
// without split-K for the grouped and TN forms and with one tile a CU: 7.7 %).  What decides,
// measured (the general model's choice in brackets): 64 x 4096 x 7168 BF16 16.8 us
// (28.6); 1024 x 4096 x 4096 39.7 (48.2); masked 8 x 256 x 2048 x 4096 FP8 33.0 (53.5);
// 4 experts' 8704 x 4096 x 7168 FP8 267 as 128 x 128, whose 2176 tiles leave 6 % of the last
// round idle, against 343 as 256 x 256 (544 tiles, 29 % idle), where 8192 x 4096 x 7168
// BF16 (512 tiles) runs 348 as 256 x 256 and over 430 as 128 x 128.  Split against
// unsplit: TN 512 x 512 over K 16384 21 us against 65, TN 1600 x 1408 over 6721 45 against
// 56, masked 4 x 64 x 2048 x 7168 FP8 17.0 against 25.5, masked 2 x 447 x 1152 x 6528 BF16
// 17.4 against 24.9, contiguous 2 experts' 256 x 1600 x 4352 FP8 11.7 against 13.9.
//
// Contiguous rows in 256-row tiles: an expert that ends inside a tile (every second one does, of
// random lengths) has it computed twice, which lengthens that CU's round.  It adds 0.25 + 0.065
// (experts - 1) rounds, whatever the rows and columns: measured over 40 shapes of 8192 to 65536
// rows in 4 to 32 experts of random lengths, where a choice with it takes 0.3 % longer than the best of
// 256 x 256, 128 x 256 and 128 x 128 (half a row block an expert, rounded up to whole rounds: 1.1 %).
// us, 256 x 256 and 128 x 256: FP8 32768 x 4096 x 7168 in 4 experts 862 and 977 (ending at
// multiples of 256 rows 823 and 996), in 8 891 and 987, in 32 1060 and 1022; 8192 rows in 4
// 241 and 226; BF16 32768 x 4096 x 4096 in 8 877 and 929, in 32 1058 and 974.
struct Structure {
    int bm, bn, wm, wn, stages, variant;
    int per_cu;                    // tiles a CU works on at a time
    double us_bf16, us_fp8;        // (FP8: a block is 128 K values, and its scales are applied)
    double us_full_bf16, us_full_fp8;
};
const Structure kStructures[] = {
    {256, 256, 4, 2, 2, 6, 1, 1.37, 1.64, 0, 0},       {128, 256, 2, 4, 3, 0, 1, 0.80, 0.92, 0, 0},
    {128, 192, 2, 4, 3, 0, 1, 0.75, 0.82, 0, 0},       {192, 128, 4, 2, 3, 0, 1, 0.64, 0.74, 0, 0},
    {128, 128, 4, 2, 4, 0, 1, 0.51, 0.54, 0, 0},       {128, 128, 2, 2, 2, 6, 2, 0.64, 0.64, 0.49, 0.49},
    {128, 64, 4, 2, 4, 0, 1, 0.33, 0.41, 0, 0},        {64, 128, 2, 4, 4, 0, 1, 0.34, 0.41, 0, 0},
    {64, 128, 2, 2, 3, 0, 2, 0.45, 0.43, 0.38, 0.33},  {64, 64, 2, 2, 4, 0, 2, 0.23, 0.32, 0.23, 0.18},
    {32, 64, 1, 4, 4, 0, 2, 0.20, 0.29, 0.15, 0.21},   {16, 64, 1, 4, 4, 0, 4, 0.13, 0.22, 0.11, 0.20},
    {16, 32, 1, 2, 6, 0, 4, 0.16, 0.17, 0.11, 0.12},
};

bool uses_structures(const Problem& p) {
    return p.ep.any() || p.direct || (p.sf == 3 && (p.kind == kKGrouped || p.b_k_outer));
}

std::vector<KernelConfig> choose_structure(const Problem& p, int num_cus, const KernelConfig& base) {
    // row blocks, with this share of a masked group's rows valid (the last block part full)
    auto row_blocks = [&](int bm, double valid_rows) {
        if (p.kind == kMasked)
            return std::min((double)((p.rows + bm - 1) / bm), valid_rows * p.rows / bm + 0.5) * p.g;
        return (double)((p.rows + bm - 1) / bm) * (p.kind == kKGrouped ? p.g : 1);
    };
    // rows of the output, for a split's partials
    const double out_rows = p.kind == kMasked ? 0.5 * p.rows * p.g : p.kind == kKGrouped ? (double)p.rows * p.g : p.rows;
    // K blocks of a tile; K-grouped: of a group on average, from the plan's share of K
    const double kb = p.kind == kKGrouped ? std::max(1.0, (double)k_share_blocks(k_share(p.kt)) / p.g) : p.k / 128;
    double best = 1e30;
    std::vector<KernelConfig> out;
    for (const Structure& st : kStructures) {
        // (TN reads 128 x 64 tiles slowly: 512 x 512 over K 16384 28.8 us against 21.0 as 64 x 128)
        if (p.kind == kKGrouped && st.bm > st.bn) continue;
        // (many blocks of few rows read B again and again: 97 x 2616 x 448 NN 6.6 us as 16 x 64, 5.4 as
        // 32 x 64; and blocks of many more rows than there are were not among the launches)
        if (p.rows > (st.bm == 16 ? 64 : st.bm == 32 ? 1024 : p.rows)) continue;
        if (p.kind != kKGrouped && p.rows <= (st.bm > 64 ? 64 : st.bm > 16 ? 16 : 0)) continue;
        const int columns = (p.n + st.bn - 1) / st.bn;
        const double tiles = row_blocks(st.bm, 0.5) * columns;
        const double us = p.sf == 3 ? st.us_bf16 : st.us_fp8;
        const double us_full = p.sf == 3 ? st.us_full_bf16 : st.us_full_fp8;
        const double start = 1.1 + 2.3 * st.bm * st.bn / 16384.0;
        for (int sk = 1; sk <= 16; ++sk) {
            if (sk > 1 && kb / sk < 4) continue;
            if (sk > 1 && tiles * sk > 2 * num_cus) break;     // (the tiles alone fill the device)
            const double blocks = std::ceil(kb / sk);
            auto time_of = [&](double items) {
                double per_cu = std::max(1.0, std::ceil(items / num_cus - 1e-9));
                double batches = std::ceil(per_cu / st.per_cu);
                if (p.kind == kContiguous && st.bm > 128 && p.g > 1) batches += 0.25 + 0.065 * (p.g - 1);
                if (st.per_cu == 1) return batches * (start + blocks * us);
                return start * (1 + 1.5 * (batches - 1)) + blocks * std::max(batches * us, per_cu * us_full);
            };
            double t = time_of(tiles * sk);
            // (half the rows, a quarter fewer and a quarter more: a choice must not need luck)
            if (p.kind == kMasked)
                t = (t + time_of(row_blocks(st.bm, 0.375) * columns * sk) + time_of(row_blocks(st.bm, 0.625) * columns * sk)) / 3;
            if (sk > 1) t += 0.6 + 2.7e-6 * out_rows * p.n * sk;
            KernelConfig c = base;
            c.bm = st.bm; c.bn = st.bn; c.wm = st.wm; c.wn = st.wn;
            c.stages = st.stages; c.variant = st.variant; c.splitk = sk; c.kstep = 1;
            if (t < best && valid(c, p)) {
                best = t;
                out = {c};
            }
        }
    }
    return out;
}

// Dense products of few rows with low-rank adapters: the epilogue waits for the adapters' factors, so more and
// smaller tiles win, several to a CU.  The times are as above, start + K blocks, with a start of each structure's
// own, fitted to 1150 launches of 50 shapes (1 to 256 rows, 1024 to 7168 columns, K 512 to 4096, 32 adapters of rank 16,
// a different one each row); over these the choice takes 2.6 % longer than the fastest of twelve structures, kStructures'
// 8.6 %.  us: 32 x 7168 x 2048 14.8 against 17.8, 96 x 2112 x 1536 13.0 against 14.7, 256 x 1024 x 1024 10.9 against
// 12.7.  (From 256 rows on kStructures' tiles win: 517 x 2112 x 1536 20.4 as 128 x 64, 24.0 as 64 x 64.)
// Rank and mix of the adapters are not among its inputs.  Over eleven settings of other ranks (16 to 256) and mixes (a
// different adapter each row, prompts, one adapter for all) the choice takes 2 % longer than the fastest of these
// structures, at most 10 % (256 x 4096 x 2048, rank 32, each row its own: 29.6 as 32 x 64, 26.9 as 64 x 64).
constexpr int kLoraRows = 256;
struct LoraStructure {
    int bm, bn, wm, wn, stages, per_cu;
    double start, us, us_full;
};
const LoraStructure kLoraStructures[] = {
    {32, 32, 2, 2, 6, 3, 1.52, 0.074, 0.087},
    {32, 64, 1, 4, 4, 3, 2.24, 0.186, 0.129},
    {16, 32, 1, 2, 6, 4, 1.51, 0.045, 0.059},
    {64, 64, 2, 2, 4, 2, 4.01, 0.195, 0.225},
};
std::vector<KernelConfig> choose_lora_structure(const Problem& p, int num_cus, const KernelConfig& base) {
    const int kb = p.k / 128;
    double best = 1e30;
    std::vector<KernelConfig> out;
    for (const LoraStructure& st : kLoraStructures) {
        if (st.bm > std::max(16, 2 * p.rows)) continue;      // (not among the launches)
        const int tiles = (p.rows + st.bm - 1) / st.bm * ((p.n + st.bn - 1) / st.bn);
        for (int sk = 1; sk <= 4; sk *= 2) {
            if (sk > 1 && (kb / sk < 4 || tiles * sk > 2 * num_cus)) continue;
            const double each = std::ceil((double)tiles * sk / num_cus), batches = std::ceil(each / st.per_cu);
            const double blocks = std::ceil((double)kb / sk);
            double t = st.start * (1 + 1.5 * (batches - 1)) + blocks * std::max(batches * st.us, each * st.us_full);
            if (sk > 1) t += 2.8e-6 * p.rows * p.n * sk;
            KernelConfig c = base;
            c.bm = st.bm; c.bn = st.bn; c.wm = st.wm; c.wn = st.wn;
            c.stages = st.stages; c.variant = 0; c.splitk = sk; c.kstep = 1;
            if (t < best && valid(c, p)) {
                best = t;
                out = {c};
            }
        }
    }
    return out;
}

// DG_FORCE_CONFIG="bm,bn,wm,wn,stages,splitk[,kstep[,variant[,nb,ne]]]", or
// several such launches over column ranges [nb, ne) separated by ';'.
std::vector<KernelConfig> parse_forced(const KernelConfig& base) {
    const char* env = std::getenv("DG_FORCE_CONFIG");
    if (!env || !*env) return {};
    std::vector<KernelConfig> out;
    std::string all(env);
    size_t pos = 0;
    while (pos <= all.size()) {
        size_t end = all.find(';', pos);
        if (end == std::string::npos) end = all.size();
        const std::string one = all.substr(pos, end - pos);
        pos = end + 1;
        int bm, bn, wm, wn, st, sk, ks = 1, var = 0, nb = 0, ne = 0;
        int got = std::sscanf(one.c_str(), "%d,%d,%d,%d,%d,%d,%d,%d,%d,%d", &bm, &bn, &wm, &wn, &st, &sk, &ks, &var,
                              &nb, &ne);
        if (got < 6 || got == 9) return {};
        KernelConfig c = base;
        c.bm = bm; c.bn = bn; c.wm = wm; c.wn = wn; c.stages = st; c.splitk = sk; c.kstep = ks;
        c.variant = var;
        c.nb = nb; c.ne = ne;
        out.push_back(c);
    }
    return out;
}

// A B block that at most two row blocks of the launch read (dense or masked
// with few rows) is streamed: its loads carry the non-temporal hint.  Measured
// (one box, alternating): 128x24576x1536 15.1 against 15.5 us, with C 16.0
// against 18.8, UE8M0 14.6 against 15.4, the masked decode shape 18.3 against
// 19.7; where four row blocks share each B block through L2 (the large
// shapes) the hint cost 1-9 %.
std::vector<KernelConfig> with_b_streams(std::vector<KernelConfig> plan, const Problem& p) {
    for (KernelConfig& c : plan)
        c.bstream = (p.kind == kDense || p.kind == kMasked) && p.rows <= 2 * c.bm ? 1 : 0;
    return plan;
}

// The launches cover [0, N) in order, each valid.
bool valid_plan(const std::vector<KernelConfig>& plan, const Problem& p) {
    if (plan.empty()) return false;
    int next = 0;
    for (const KernelConfig& c : plan) {
        if (!valid(c, p) || c.n_begin() != next) return false;
        next = c.n_end();
    }
    return next == p.n;
}

}  // namespace

int64_t num_work_items(const KernelConfig& c, int rows) {
    const int64_t mt = (rows + c.bm - 1) / c.bm;
    const int64_t nt = (c.n_end() - c.n_begin() + c.bn - 1) / c.bn;
    return mt * nt * c.splitk * (c.kind == kMasked || c.kind == kKGrouped ? c.g : 1);
}

std::vector<KernelConfig> select_plan(const Problem& p, int num_cus) {
    KernelConfig base;
    base.kind = p.kind;
    base.has_c = p.has_c;
    base.sf = p.sf;
    base.n = p.n;
    base.k = p.k;
    base.g = (p.kind == kDense) ? 1 : p.g;
    base.ep = p.ep;
    // operands read as stored keep that through every choice below
    base.a_kout = p.direct && p.kind == kKGrouped;
    base.b_kout = p.direct;

    std::vector<KernelConfig> forced = parse_forced(base);
    if (valid_plan(forced, p)) return with_b_streams(forced, p);
    std::vector<KernelConfig> table;
    // (the contiguous entries are for any large row count; the structures weigh its rounds)
    if (!uses_structures(p) || p.kind == kDense || p.kind == kMasked) table = tuned(p, num_cus, base);
    if (p.direct) table.clear();
    if (table.empty() && p.ep.lora && p.rows <= kLoraRows) table = choose_lora_structure(p, num_cus, base);
    if (table.empty() && uses_structures(p)) table = choose_structure(p, num_cus, base);
    table = with_b_streams(table, p);
    if (valid_plan(table, p)) {
        if (env_flag("DG_PRINT_CONFIGS"))
            for (const KernelConfig& c : table)
                std::fprintf(stderr, "[dg] kind=%d rows=%d N=%d K=%d G=%d -> %s (measured)\n", p.kind, p.rows, p.n,
                             p.k, p.g, c.key().c_str());
        return table;
    }

    // masked: the host cannot see masked_m; plan for half the rows being valid
    const double valid_rows = (p.kind == kMasked) ? 0.5 * p.rows * p.g : (double)p.rows;
    const int kb = p.k / 128;
    static const int bms[] = {16, 32, 64, 128, 256};
    static const int bns[] = {16, 32, 48, 64, 96, 112, 128, 160, 192, 224, 256};
    static const int wgs[][2] = {{1, 4}, {2, 2}, {4, 1}, {2, 4}, {4, 2}, {1, 8}, {8, 1}, {1, 1}, {1, 2}, {2, 1}};
    const int max_bm = round_up(std::max(p.rows, 16), 16);
    // Skinny row counts: one row block covers every row (of a group), so each B
    // tile is fetched from HBM once instead of once per row block.
    // (masked groups are not: their row blocks past masked_m[g] are skipped)
    const bool one_row_block = p.kind == kDense && p.rows <= 256;

    // Structure the measurements favour on gfx950: two waves per SIMD (8-wave
    // workgroups) for large tiles, four waves otherwise, wave grids no more
    // than 4:1, row blocks of 64+ rows unless the problem has fewer rows, and
    // split-K only when the output tiles alone cannot fill the device.
    const int out_tiles_128 = ((p.rows + 127) / 128) * ((p.n + 127) / 128);
    Estimate best{1e30, base};
    for (int bm : bms) {
        if (bm > max_bm && bm > 16 && bm / 2 >= max_bm) continue;   // no tile twice the rows
        if (one_row_block && bm < max_bm) continue;
        if (bm < 64 && max_bm >= 64) continue;
        for (int bn : bns) {
            if (bn > round_up(p.n, 16) && bn / 2 >= round_up(p.n, 16)) continue;
            for (auto& w : wgs) {
                const int nw = w[0] * w[1];
                const bool tiny = bm * bn < 64 * 64;
                if (!tiny && nw < 4) continue;
                if (bm * bn >= 128 * 96 && nw < 8) continue;
                if (bm * bn < 128 * 96 && nw > 4) continue;
                if (w[0] > 2 * w[1] || w[1] > 2 * w[0]) {
                    if (!tiny) continue;
                }
                for (int sk = 1; sk <= 16; ++sk) {
                  for (int ks = 1; ks <= (p.sf ? 1 : 2); ++ks) {
                    if (sk > 1 && (p.kind != kDense || kb % sk || kb / sk < 2)) continue;
                    if (sk > 1 && out_tiles_128 * 2 >= num_cus) continue;
                    if (sk > 1 && bm * bn < 64 * 128) continue;   // small split tiles measured slow
                    KernelConfig c = base;
                    c.bm = bm; c.bn = bn; c.wm = w[0]; c.wn = w[1]; c.splitk = sk; c.kstep = ks;
                    c.stages = std::min(4, kLdsBytes / c.stage_bytes());
                    while (c.stages > 2 && dma_per_wave(c) * (c.stages - 1) > 63) --c.stages;
                    if (c.stages < 2) continue;
                    if (!valid(c, p)) continue;
                    double t = estimate(p, c, num_cus, valid_rows);
                    // prefer bigger wave tiles on ties (fewer LDS reads per MFMA)
                    t *= 1.0 + 0.01 / (c.bm / c.wm / 16 * (c.bn / c.wn / 16));
                    if (t < best.seconds) best = {t, c};
                  }
                }
            }
        }
    }
    std::vector<KernelConfig> plan = with_b_streams({best.cfg}, p);
    if (env_flag("DG_PRINT_CONFIGS"))
        std::fprintf(stderr, "[dg] kind=%d rows=%d N=%d K=%d G=%d -> %s (model %.2f us)\n", p.kind, p.rows, p.n,
                     p.k, p.g, plan[0].key().c_str(), best.seconds * 1e6);
    return plan;
}

}  // namespace dg
