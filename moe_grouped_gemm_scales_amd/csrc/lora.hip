// Low-rank adapters of many requests beside a shared product (hipcc, gfx950): the
// first of their two products, low = scale (A down[adapter]^T).  The second is
// added in the shared product's epilogue (kernels/fp8_gemm.hip).  The operation
// is specified in include/dg.h.
//
// One workgroup takes 16 rows of A and up to 64 ranks; its eight waves take an
// eighth of K each, on the matrix cores straight from global memory (an operand's 16
// rows are 128 bytes each a step), and their sums meet in LDS.  It reads A once, and from
// L2 an adapter once for each 16 rows that use it; a few dependent round trips bound it.
// us (sixteen waves in brackets): 32 x 2048, 32 adapters of rank 16 4.1 (4.1), of which a launch is 2; 4096 x 2048,
// eight of rank 64 11 (13), one alone 7.8 (10.0), 8192 x 7168 rank 64 60 (85).  With 32 rows a workgroup, which
// reads an adapter half as often, the last takes 55, but 4096 x 2048 17.6 and 16384 x 2048 25.8 against 23.6.
#include <cmath>

#include "row_kernels.h"

namespace dg {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;
constexpr int kWaves = 8;

// 16 rows of 64 bytes, lane 4 r + c with 16-byte piece c of row r, as an operand of the matrix instruction: piece c of
// row r to lane 16 c + r.  Loaded that way round, four lanes side by side read one piece of 64 bytes; a lane a row apart
// from its neighbour each, as the operand lies, is a request of its own for each lane, which was what bounded the
// pass (32 rows of K = 2048 with 32 adapters of rank 16 6.1 us).
__device__ __forceinline__ bf16x8 operand(u32x4 w, int from) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (u32)__builtin_amdgcn_ds_bpermute(from, (int)w[i]);
    return __builtin_bit_cast(bf16x8, v);
}

struct DownArgs {
    const u16* A;
    const u16* down;
    const int* adapter;
    const float* scale;
    u16* low;
    int M, K, adapters, rank, pitch;
};

// SUBS: 16-rank pieces of a workgroup (1, 2 or 4; a workgroup has 16 SUBS ranks).  Grid z of 16: a row, whose adapter the
// workgroup does if no earlier row has the same.  Of fewer: a place in the list of the 16 rows' adapters, the last place
// doing all that are left, in turn.
template <int SUBS>
__global__ void __launch_bounds__(64 * kWaves) dg_lora_down_kernel(const DownArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const int m = (int)blockIdx.x * kRows + l16;
    const int r0 = (int)blockIdx.y * (16 * SUBS);
    int ad = m < a.M ? a.adapter[m] : -1;
    if ((u32)ad >= (u32)a.adapters) ad = -1;
    // rows whose adapter is not done by an earlier place
    u32 todo = (u32)__ballot(ad >= 0) & 0xffffu;
    auto next_of = [&]() { return __builtin_amdgcn_readlane(ad, __builtin_ctz(todo)); };
    if (gridDim.z == kRows) {
        const int of_z = __builtin_amdgcn_readlane(ad, (int)blockIdx.z);
        todo = of_z < 0 ? 0u : (u32)__ballot(ad == of_z) & 0xffffu;
        if (todo == 0u || (u32)__builtin_ctz(todo) != blockIdx.z) return;
    } else {
        for (u32 z = 0; z < blockIdx.z && todo; ++z) todo &= ~(u32)__ballot(ad == next_of());
        if (todo == 0u) return;
        if (blockIdx.z + 1 < gridDim.z) todo &= (u32)__ballot(ad == next_of());
    }
    f32x4 sum[SUBS];
#pragma unroll
    for (int s = 0; s < SUBS; ++s) sum[s] = f32x4{0.f, 0.f, 0.f, 0.f};
    bool done = false;                               // this lane's row
    // a wave's share of K, in steps of 64: waves an eighth of a row apart read different memory channels,
    // where neighbouring steps of all rows (4 KB apart at K = 2048) would meet in a few
    const int steps = a.K / 64;
    const int k_begin = steps * wave / kWaves * 64, k_end = steps * (wave + 1) / kWaves * 64;
    // loads: lane 4 r + c takes piece c of row r
    const int lr = lane >> 2, lc = 8 * (lane & 3), from = 4 * (4 * l16 + q);
    const int mr = (int)blockIdx.x * kRows + lr;
    const u16* rows = a.A + (u64)(mr < a.M ? mr : a.M - 1) * (u64)a.K + lc;
    while (todo) {
        const int mine = next_of();
        todo &= ~(u32)__ballot(ad == mine);
        const u16* down[SUBS];
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
            // ranks past the last read the last one; their results are not kept
            const int r = r0 + 16 * s + lr;
            down[s] = a.down + ((u64)mine * (u64)a.rank + (u32)(r < a.rank ? r : a.rank - 1)) * (u64)a.K + lc;
        }
        f32x4 acc[SUBS];
#pragma unroll
        for (int s = 0; s < SUBS; ++s) acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int k = k_begin; k < k_end; k += 64) {
            u32x4 x[2], d[SUBS][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[h] = *(const u32x4*)(rows + k + 32 * h);
#pragma unroll
                for (int s = 0; s < SUBS; ++s) d[s][h] = *(const u32x4*)(down[s] + k + 32 * h);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bf16x8 row = operand(x[h], from);
#pragma unroll
                for (int s = 0; s < SUBS; ++s)
                    acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(d[s][h], from), row, acc[s], 0, 0, 0);
            }
        }
        // (a select: another adapter's rows keep their own sums, whatever this one made of them)
        if (ad == mine) {
            done = true;
#pragma unroll
            for (int s = 0; s < SUBS; ++s) sum[s] = acc[s];
        }
    }
    __shared__ f32x4 parts[kWaves][SUBS][64];
#pragma unroll
    for (int s = 0; s < SUBS; ++s) parts[wave][s][lane] = sum[s];
    __syncthreads();
    // wave s adds piece s in wave order: lane (row l16, ranks 4 q ..); one piece of 16 clears the 16 behind it
    if (wave >= SUBS || !done) return;
    f32x4 t = parts[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += parts[w][wave][lane];
    const int r = r0 + 16 * wave + 4 * q;
    const float scale = a.scale ? a.scale[ad] : 1.f;
    // the layout of the other product's operand: of 16 rows and 32 ranks, 1 KB of the values and 1 KB of what BF16
    // leaves of them, each with ranks 8 c .. 8 c + 7 of row r at piece 16 c + r
    auto store = [&](int r, u64 hi, u64 lo) {
        u16* to = a.low + ((u64)blockIdx.x * (u32)(a.pitch / 32) + (u32)(r / 32)) * 1024 +
                  ((r % 32) / 8 * 16 + l16) * 8 + r % 8;
        *(u64*)to = hi;
        *(u64*)(to + 512) = lo;
    };
    if (r < a.pitch) {
        u64 hi = 0, lo = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = r + e < a.rank ? scale * t[e] : 0.f;
            u16 h = to_bf16(v);
            // a number past BF16's range keeps what of it BF16 holds and the rest; an infinity or NaN has no rest
            if ((h & 0x7fffu) == 0x7f80u && __builtin_fabsf(v) < INFINITY) h -= 1;
            const float rest = (h & 0x7fffu) < 0x7f80u ? v - bf16_lo(h) : 0.f;
            hi |= (u64)h << (16 * e);
            lo |= (u64)to_bf16(rest) << (16 * e);
        }
        store(r, hi, lo);
    }
    if constexpr (SUBS == 1) {
        if (r + 16 < a.pitch) store(r + 16, 0, 0);
    }
}

}  // namespace

dg_status lora_down(const LoraArgs& l, const void* A, void* low, int M, int K, void* stream) {
    const int pitch = lora_pitch(l.rank);
    const DownArgs args{static_cast<const u16*>(A), static_cast<const u16*>(l.down), l.adapter, l.scale, static_cast<u16*>(low), M, K,
                        l.adapters, l.rank, pitch};
    // Up to 2048 rows every row is a place (decode: 16 adapters side by side), for more there are two (prompts, where a
    // block that ends one and begins the next would take twice as long); most of them find nothing to do and end.  us with
    // one place, two and 16: 600 rows of 32 adapters 28.3, 26.6, 8.6; prompts, 517 x 1536 5.5, 4.2, 4.2, 2048 x 2048
    // 6.3, 4.9, 5.0; 4096 x 2048, rank 64, 11.6 each, with one adapter 8.0, 8.0, 9.3.  The rule sees the number of rows
    // alone: where more than 2048 rows have an adapter each, the second place does fifteen in turn (with the product, 2048 x
    // 2112 x 2048 of rank 16 61 us, 2064 rows 76).
    const int subs = l.rank <= 16 ? 1 : l.rank <= 32 ? 2 : 4;
    const dim3 grid((M + kRows - 1) / kRows, (l.rank + 16 * subs - 1) / (16 * subs), M <= 2048 ? kRows : 2);
    auto* kernel = subs == 1 ? dg_lora_down_kernel<1> : subs == 2 ? dg_lora_down_kernel<2> : dg_lora_down_kernel<4>;
    return launch_rows("lora (down)", kernel, grid, 64 * kWaves, stream, args);
}

}  // namespace dg
