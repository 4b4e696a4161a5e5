// Tokens to experts and back (hipcc, gfx950): the steps between a router's
// top-k choice and the grouped products, and from their rows back to the
// tokens.  The operations and their layouts are specified in include/dg.h.
//
//   sort      a counting sort of T * k expert ids: stable, so that a token's
//             place depends on the ids alone and every run gives the same rows
//   dispatch  rows[pos[t][j]] = X[t] (BF16 copies, or quantised to E4M3)
//   combine   Y[t] = residual[t] + sum_j w[t][j] rows[pos[t][j]]
//   combine backward   dRows[pos[t][j]] = w[t][j] dY[t],  dw[t][j] = <dY[t], rows[pos[t][j]]>
//
// All of it moves data: nothing here has more than a few operations a byte, so
// each kernel is built to read and write every byte once, 16 bytes a lane.
// Work is cut by token, not by row: a token's hidden state is then read (and
// quantised) once for its k copies, and a token's k rows meet in one wave's
// registers, where the sum over j has a fixed order.
#include <climits>

#include "row_kernels.h"

namespace dg {
namespace {

constexpr int kAlign = 128;            // rows an expert's segment starts on a multiple of
constexpr int kMaxExperts = 1024;      // the sort's per-wave counters live in LDS
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortRounds = 4;
constexpr int kSortStep = kSortRounds * kSortThreads;
constexpr int kSortBlocks = 256;       // at most, so that one pass over their counts stays short
constexpr int kUnused = -2;            // ... of a row past the last segment

// 16 bytes a lane.  STREAM: with the non-temporal hint, for calls that read and
// write more than the caches keep until the next pass (kStreamBytes).  Measured
// (two sets of buffers in turn, top 4 of 32, width 7168; plain against streamed,
// us): combine of 1024 tokens (88 MB) 14.4 / 15.4, 2048 (176 MB) 33.6 / 29.7, 8192
// 132 / 118.5; its gradient 512 (66 MB) 21.1 / 28.2, 1024 (132 MB) 39.9 / 39.4, 4096
// 118.5 / 111.9; dispatch in BF16 1024 (73 MB) 17.7 / 19.3, 2048 (147 MB) 34.0 / 29.2,
// in FP8 2048 (88 MB) 21.4 / 20.9, 4096 (176 MB) 44.3 / 36.3.  (The FP8 dispatch streams its stores only: with
// its loads too it gives half of that back.)
template <bool STREAM>
__device__ __forceinline__ u32x4 load16(const void* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const u32x4*>(p));
    else return *static_cast<const u32x4*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, u32x4 v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
    else *static_cast<u32x4*>(p) = v;
}

// ---------------------------------------------------------------- sort
// Block b counts the experts of its chunk of the ids.
struct CountArgs {
    const int* ids;
    u32* hist;
    int n, G, chunk;
};
__global__ void __launch_bounds__(kSortThreads) dg_moe_count_kernel(const CountArgs a) {
    const int* __restrict__ ids = a.ids;
    u32* __restrict__ hist = a.hist;
    const int n = a.n, G = a.G, chunk = a.chunk;
    __shared__ u32 h[kMaxExperts];
    for (int g = threadIdx.x; g < G; g += kSortThreads) h[g] = 0u;
    __syncthreads();
    const int first = (int)blockIdx.x * chunk;
    const int last = n - first < chunk ? n : first + chunk;
    for (int i = first + (int)threadIdx.x; i < last; i += kSortThreads) {
        const u32 e = (u32)ids[i];
        if (e < (u32)G) atomicAdd(&h[e], 1u);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += kSortThreads) hist[(u64)blockIdx.x * G + g] = h[g];
}

// Block b places its chunk.  Rank of an id = ids of the same expert in earlier
// blocks (summed here from every block's counts) + in earlier waves of the
// block (an LDS table [wave][expert]) + earlier in the wave.  A wave takes
// consecutive ids, 64 a round and up to four rounds: the lanes that hold the same
// expert are found by one ballot per bit of the id, and their lowest adds their
// number to the wave's counter and hands the others the count before it, so the
// rounds need no barrier.  hist == nullptr: the only block, whose one step also
// counts.  masked_rows > 0: masked layout, expert g's rows start at g *
// masked_rows; 0: contiguous layout, segments of whole 128-row blocks, and every
// block writes its share of m_indices.
struct SortArgs {
    const int* ids;
    const u32* hist;
    int* pos;
    int* m_indices;
    int* group_rows;
    int n, G, bits, chunk, masked_rows, rows;
};
__global__ void __launch_bounds__(kSortThreads)
dg_moe_place_kernel(const SortArgs a) {
    const int* __restrict__ ids = a.ids;
    const u32* __restrict__ hist = a.hist;
    int* __restrict__ pos = a.pos;
    int* __restrict__ m_indices = a.m_indices;
    int* __restrict__ group_rows = a.group_rows;
    const int n = a.n, G = a.G, bits = a.bits, chunk = a.chunk, masked_rows = a.masked_rows, rows = a.rows;
    __shared__ u32 total[kMaxExperts];      // rows of each expert
    __shared__ u32 before[kMaxExperts];     // ... placed so far: by earlier blocks, then by earlier steps
    __shared__ u32 base[kMaxExperts];       // first row of the expert's segment
    __shared__ u32 wcnt[kSortWaves * kMaxExperts];
    __shared__ u32 wave_sum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.x, blocks = gridDim.x;

    const int first = b * chunk;
    const int last = n - first < chunk ? n : first + chunk;
    // the ids of the step at i0, asked for before the work in front of their first use
    u32 e[kSortRounds];
    auto read_ids = [&](int i0) {
        const int len = last - i0 < kSortStep ? last - i0 : kSortStep;
        const int rounds = (len + kSortThreads - 1) / kSortThreads;
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) {
            const int at = (wave * rounds + q) * 64 + lane;
            e[q] = q < rounds && at < len ? (u32)ids[i0 + at] : 0xffffffffu;
        }
    };
    read_ids(first);
    for (int g = tid; g < G; g += kSortThreads) total[g] = before[g] = 0u;
    for (int w = tid; w < kSortWaves * G; w += kSortThreads) wcnt[w] = 0u;
    __syncthreads();
    if (hist) {
        // thread (part, g): the counts of every parts-th block (g fastest: coalesced)
        int wide = 64;
        while (wide < G) wide *= 2;
        const int parts = kSortThreads / wide, g = tid & (wide - 1);
        if (g < G) {
            u32 all = 0, mine = 0;
            for (int o = tid / wide; o < blocks; o += parts) {
                const u32 c = hist[(u64)o * G + g];
                all += c;
                if (o < b) mine += c;
            }
            if (all) atomicAdd(&total[g], all);
            if (mine) atomicAdd(&before[g], mine);
        }
        __syncthreads();
    }

    // first rows: exclusive sum of the segments (one expert a thread: G <= 1024)
    auto place_segments = [&]() {
        const u32 cnt = tid < G ? total[tid] : 0u;
        u32 seg = 0;
        if (tid < G) seg = masked_rows > 0 ? (u32)masked_rows : (cnt + kAlign - 1) / kAlign * kAlign;
        u32 x = seg;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const u32 y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        if (lane == 63) wave_sum[wave] = x;
        __syncthreads();
        u32 sums = lane < wave ? wave_sum[lane] : 0u;       // of the waves before this one (at most 15)
#pragma unroll
        for (int d = 8; d > 0; d /= 2) sums += __shfl_xor(sums, d);
        const u32 start = __shfl(sums, 0) + x - seg;
        if (tid < G) {
            base[tid] = start;
            if (b == 0) {
                if (masked_rows > 0) {
                    group_rows[tid] = (int)(cnt < (u32)masked_rows ? cnt : (u32)masked_rows);
                } else {
                    const u32 room = start < (u32)rows ? (u32)rows - start : 0u;
                    group_rows[tid] = (int)(seg < room ? seg : room);
                }
            }
        }
    };
    if (hist) place_segments();

    for (int i0 = first;;) {
        const int len = last - i0 < kSortStep ? last - i0 : kSortStep;     // 0: no ids at all
        const int rounds = (len + kSortThreads - 1) / kSortThreads;
        u32 rank[kSortRounds];
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) {
            if (q >= rounds) break;
            const bool ok = e[q] < (u32)G;
            u64 peers = __ballot(ok);
            for (int bit = 0; bit < bits; ++bit) {
                const bool one = (e[q] >> bit) & 1u;
                const u64 m = __ballot(one);
                peers &= one ? m : ~m;
            }
            // (a lane without an id has no peers: it is its own, and adds nothing)
            const u32 below = __popcll(peers & ((1ull << lane) - 1ull));
            const int lowest = ok ? __builtin_ctzll(peers) : lane;
            u32 old = 0;
            if (ok && below == 0) old = atomicAdd(&wcnt[wave * G + e[q]], (u32)__popcll(peers));
            rank[q] = __shfl(old, lowest) + below;
        }
        __syncthreads();
        u32 step_total = 0;                       // of expert tid
        if (tid < G) {
            u32 c[kSortWaves];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) c[w] = wcnt[w * G + tid];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                wcnt[w * G + tid] = step_total;
                step_total += c[w];
            }
            if (!hist) total[tid] = step_total;
        }
        __syncthreads();
        if (!hist) {
            place_segments();
            __syncthreads();
        }
#pragma unroll
        for (int q = 0; q < kSortRounds; ++q) {
            const int at = (wave * rounds + q) * 64 + lane;
            if (q >= rounds || at >= len) continue;
            int row = -1;
            if (e[q] < (u32)G) {
                const u32 r = before[e[q]] + wcnt[wave * G + e[q]] + rank[q];
                const u32 to = base[e[q]] + r;
                if (masked_rows > 0 ? r < (u32)masked_rows : to < (u32)rows) row = (int)to;
            }
            pos[i0 + at] = row;
        }
        i0 += kSortStep;
        if (i0 >= last) break;
        read_ids(i0);
        __syncthreads();
        if (tid < G) before[tid] += step_total;
        for (int w = tid; w < kSortWaves * G; w += kSortThreads) wcnt[w] = 0u;
        __syncthreads();
    }

    if (masked_rows > 0) return;
    // this block's share of m_indices: the expert whose segment holds the row is
    // the last one that starts at or before it (empty segments start where the
    // next one does, and the last of equals is the one that holds rows)
    __syncthreads();
    const int share = rows / blocks + 1;
    const int r0 = b * share < rows ? b * share : rows;
    const int r1 = rows - r0 < share ? rows : r0 + share;
    // (unsigned: rows may be up to 2^31 - 128, and a thread's last step passes 2^31)
    for (u32 r = (u32)r0 + (u32)tid; r < (u32)r1; r += kSortThreads) {
        int lo = 0;
        for (int half = 1 << bits >> 1; half > 0; half >>= 1)
            if (lo + half < G && base[lo + half] <= r) lo += half;
        const u32 in = r - base[lo], cnt = total[lo];
        m_indices[r] = in < cnt ? lo : in < (cnt + kAlign - 1) / kAlign * kAlign ? kPadding : kUnused;
    }
}

// ---------------------------------------------------------------- padding rows
// `fill(row)` for each row of the kPadRows-row block `blk` whose index is -1.
// Rows past the last segment (-2) are left alone.  16 rows a wave: with 128 the
// waves that clear a nearly empty segment outlive all others (1021 tokens x 3
// to 7 experts, width 1000: 8.0 us; with 16 3.7).
constexpr int kPadRows = 16;
template <typename F>
__device__ __forceinline__ void for_padding_rows(const int* __restrict__ m_indices, int blk, int rows, F&& fill) {
    const int r0 = blk * kPadRows, r = r0 + (int)(threadIdx.x & (kPadRows - 1));
    u32 pad = (u32)__ballot(r < rows && m_indices[r] == kPadding) & ((1u << kPadRows) - 1u);
    while (pad) {
        const int at = __builtin_ctz(pad);
        pad &= pad - 1;
        fill(r0 + at);
    }
}
__host__ __device__ constexpr int pad_blocks(int rows) { return rows / kPadRows + (rows % kPadRows != 0); }

// Rows of assignments j0 .. j0 + 7 of a token, -1 where there is none: eight
// independent scalar loads.  (A load in front of each store made the decode
// dispatch wait eight times: 5.4 us against 4.6, 32 tokens to 8 experts each.)
constexpr int kAhead = 8;
__device__ __forceinline__ void read_places(const int* __restrict__ pos, int j0, int k, int rows, int (&r)[kAhead]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int at = j0 + i < k ? pos[j0 + i] : -1;
        r[i] = (u32)at < (u32)rows ? at : -1;
    }
}

// ---------------------------------------------------------------- dispatch
// One wave a (token, piece of 1024 elements); pieces of a token are
// neighbours.  Waves past them clear the padding rows, one a (16-row block, piece).
constexpr int kPiece = 1024;

// Every kernel below takes one by-value struct: the HIP runtime prepares each
// launch argument on the host, about 0.15 us apiece.
struct DispatchArgs {
    const u16* X;
    const int* pos;
    const int* m_indices;
    void* out;
    u32* sf;
    int T, k, rows, group_rows, H, pieces;
};

// BF16.  VEC: rows are 16-byte aligned (H % 8 == 0), a lane moves two groups of
// 8 elements; otherwise 16 single elements, 64 apart.
template <bool VEC, bool STREAM>
__global__ void __launch_bounds__(256)
dg_moe_dispatch_bf16_kernel(const DispatchArgs a) {
    const u16* __restrict__ X = a.X;
    const int* __restrict__ pos = a.pos;
    const int* __restrict__ m_indices = a.m_indices;
    u16* __restrict__ out = static_cast<u16*>(a.out);
    const int T = a.T, k = a.k, rows = a.rows, H = a.H, pieces = a.pieces;
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = unit / pieces, c0 = unit % pieces * kPiece;
    if (t < T) {
        const u16* src = X + (u64)t * H;
        if constexpr (VEC) {
            const int ca = c0 + lane * 8, cb = ca + 512;
            u32x4 va = {0u, 0u, 0u, 0u}, vb = va;
            if (ca < H) va = *(const u32x4*)(src + ca);
            if (cb < H) vb = *(const u32x4*)(src + cb);
            for (int j0 = 0; j0 < k; j0 += kAhead) {
                int r[kAhead];
                read_places(pos + (u64)t * k, j0, k, rows, r);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (r[i] < 0) continue;
                    u16* dst = out + (u64)r[i] * H;
                    if (ca < H) store16<STREAM>(dst + ca, va);
                    if (cb < H) store16<STREAM>(dst + cb, vb);
                }
            }
        } else {
            u16 v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = src[c0 + lane + 64 * i < H ? c0 + lane + 64 * i : H - 1];   // (dropped past H)
            for (int j = 0; j < k; ++j) {
                const int r = pos[(u64)t * k + j];
                if ((u32)r >= (u32)rows) continue;
                u16* dst = out + (u64)r * H;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c0 + lane + 64 * i < H) dst[c0 + lane + 64 * i] = v[i];
            }
        }
        return;
    }
    const int blk = t - T;
    if (!m_indices || blk >= pad_blocks(rows)) return;
    for_padding_rows(m_indices, blk, rows, [&](int r) {
        u16* dst = out + (u64)r * H;
        if constexpr (VEC) {
            const int ca = c0 + lane * 8, cb = ca + 512;
            if (ca < H) *(u32x4*)(dst + ca) = u32x4{0u, 0u, 0u, 0u};
            if (cb < H) *(u32x4*)(dst + cb) = u32x4{0u, 0u, 0u, 0u};
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c0 + lane + 64 * i < H) dst[c0 + lane + 64 * i] = 0;
        }
    });
}

// E4M3 with one scale per 1x128 block, each token quantised once for its k
// rows.  A lane holds 16 consecutive elements, eight lanes a block, so a row
// takes 16-byte stores of 1 KB a wave.  The quotient x / s is the correctly
// rounded FP32 one (not x times a rounded 1 / s), so the codes are those of the
// definition.  The largest magnitude is taken over the bit patterns: as unsigned
// integers the magnitudes order with infinities and NaN on top, so a block that
// holds one gets a scale that says so.
// UE8M0: scales are powers of two, four K blocks to a word (sf int32 [H/512][rows]).
template <bool UE8M0, bool STREAM>
__global__ void __launch_bounds__(256)
dg_moe_dispatch_fp8_kernel(const DispatchArgs args) {
    const u16* __restrict__ X = args.X;
    const int* __restrict__ pos = args.pos;
    const int* __restrict__ m_indices = args.m_indices;
    u8* __restrict__ out = static_cast<u8*>(args.out);
    u32* __restrict__ sf = args.sf;
    const int T = args.T, k = args.k, rows = args.rows, group_rows = args.group_rows, H = args.H, pieces = args.pieces;
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = unit / pieces, c0 = unit % pieces * kPiece;
    const int c = c0 + lane * 16;
    const int kb = c >> 7;                              // this lane's 128-wide block
    const int sf_rows = UE8M0 ? (H + 511) / 512 : H / 128;   // scale entries along K
    // lanes that write a scale entry, and its index along K
    const bool scale_lane = (UE8M0 ? (lane & 31) : (lane & 7)) == 0 && c < H;
    const int sk = UE8M0 ? c >> 9 : kb;
    // row r's entry sk: sf [group][sk][row in the group]
    auto sf_at = [&](int r) {
        const int g = r / group_rows;
        return ((u64)g * sf_rows + sk) * group_rows + (r - g * group_rows);
    };
    if (t < T) {
        int r[kAhead];
        read_places(pos + (u64)t * k, 0, k, rows, r);
        float x[16];
        u32 top = 0;
        if (c < H) {
            const u16* src = X + (u64)t * H + c;
            const u32x4 a = *(const u32x4*)src, b = *(const u32x4*)(src + 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(a[i]);
                x[2 * i + 1] = bf16_hi(a[i]);
                x[8 + 2 * i] = bf16_lo(b[i]);
                x[9 + 2 * i] = bf16_hi(b[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const u32 m = __builtin_bit_cast(u32, x[i]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
#pragma unroll
        for (int d = 1; d < 8; d *= 2) {
            const u32 y = __shfl_xor(top, d);
            top = y > top ? y : top;
        }
        const float amax = __builtin_bit_cast(float, top);
        float s = amax / 448.f;
        if (s < 0x1p-126f) s = 0x1p-126f;               // a subnormal scale would lose bits of the quotient
        if (top == 0u) s = 1.f;
        u32 entry;
        if constexpr (UE8M0) {
            // the next power of two: exponent field, one more when any mantissa bit is set
            const u32 sb = __builtin_bit_cast(u32, s);
            u32 e = (sb >> 23) + ((sb & 0x7fffffu) ? 1u : 0u);
            if (e > 255u) e = 255u;
            s = __builtin_bit_cast(float, e == 255u ? 0x7fc00000u : e << 23);
            // four neighbouring blocks' bytes (8 lanes apart) meet in the lowest lane of 32;
            // blocks past H count as scale 1
            if (c >= H) e = 127u;
            entry = e | (__shfl_down(e, 8) << 8) | (__shfl_down(e, 16) << 16) | (__shfl_down(e, 24) << 24);
        } else {
            entry = __builtin_bit_cast(u32, s);
        }
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y = x[4 * i + j] / s;
                // clamp without losing a NaN
                y = y > 448.f ? 448.f : y;
                y = y < -448.f ? -448.f : y;
                v[j] = y;
            }
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
            q[i] = (u32)w;
        }
        for (int j0 = 0;;) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (r[i] < 0) continue;
                if (c < H) store16<STREAM>(out + (u64)r[i] * H + c, q);
                if (scale_lane) sf[sf_at(r[i])] = entry;
            }
            j0 += kAhead;
            if (j0 >= k) break;
            read_places(pos + (u64)t * k, j0, k, rows, r);
        }
        return;
    }
    const int blk = t - T;
    if (!m_indices || blk >= pad_blocks(rows)) return;
    for_padding_rows(m_indices, blk, rows, [&](int r) {
        if (c < H) *(u32x4*)(out + (u64)r * H + c) = u32x4{0u, 0u, 0u, 0u};
        if (scale_lane) sf[sf_at(r)] = UE8M0 ? 0x7f7f7f7fu : 0x3f800000u;
    });
}

// ---------------------------------------------------------------- combine
// One wave a (token, piece of 512 elements): 8 consecutive elements a lane, the
// residual and the token's rows loaded eight at a time (a decode step's 8 rows in
// one round trip) and added in j order in FP32.  A dropped assignment (pos
// outside the rows) is not read at all.
struct CombineArgs {
    const u16* in;
    const int* pos;
    const float* weights;
    const u16* residual;
    u16* Y;
    int T, k, rows, N, pieces;
};
template <bool VEC, bool STREAM>
__global__ void __launch_bounds__(256) dg_moe_combine_kernel(const CombineArgs a) {
    const u16* __restrict__ in = a.in;
    const int* __restrict__ pos = a.pos;
    const float* __restrict__ weights = a.weights;
    const u16* __restrict__ residual = a.residual;
    u16* __restrict__ Y = a.Y;
    const int T = a.T, k = a.k, rows = a.rows, N = a.N, pieces = a.pieces;
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = unit / pieces;
    if (t >= T) return;
    const int c0 = unit % pieces * 512;
    // element i of this lane: 8 neighbours, or 64 apart where rows are not aligned
    auto col = [&](int i) { return VEC ? c0 + lane * 8 + i : c0 + lane + 64 * i; };
    const bool in_range = col(0) < N;
    auto load = [&](const u16* p) {            // eight BF16, two a word
        u32x4 w = {0u, 0u, 0u, 0u};
        if constexpr (VEC) {
            if (in_range) w = load16<STREAM>(p + col(0));
        } else {
            w = load_spread(p, c0 + lane, N);
        }
        return w;
    };
    auto value = [](u32x4 w, int i) { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); };
    u32x4 res = {0u, 0u, 0u, 0u};
    if (residual) res = load(residual + (u64)t * N);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        int r[kAhead];
        read_places(pos + (u64)t * k, j0, k, rows, r);
        u32x4 w[kAhead];
        float wt[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            wt[i] = r[i] < 0 ? 0.f : weights ? weights[(u64)t * k + j0 + i] : 1.f;
            w[i] = u32x4{0u, 0u, 0u, 0u};
            if (r[i] >= 0) w[i] = load(in + (u64)r[i] * N);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(wt[i], value(w[i], e), acc[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += value(res, e);
    u16* dst = Y + (u64)t * N;
    if constexpr (VEC) {
        if (in_range)
            store16<STREAM>(dst + col(0), u32x4{to_bf16x2(acc[0], acc[1]), to_bf16x2(acc[2], acc[3]),
                                                to_bf16x2(acc[4], acc[5]), to_bf16x2(acc[6], acc[7])});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col(i) < N) dst[col(i)] = to_bf16(acc[i]);
    }
}

// One workgroup a token: its four waves take every fourth 512-element piece,
// read dY once and each of the token's rows once, write w dY and keep the dot
// products of up to four rows in registers (a token with more goes round again
// and finds dY in the cache).  The four waves' partial products are added in
// wave order.  Workgroups past the tokens clear the padding rows.
struct CombineBackwardArgs {
    const u16* dY;
    const u16* in;
    const int* pos;
    const float* weights;
    const int* m_indices;
    u16* d_in;
    float* d_weights;
    int T, k, rows, N;
};
template <bool VEC, bool STREAM>
__global__ void __launch_bounds__(256) dg_moe_combine_backward_kernel(const CombineBackwardArgs a) {
    const u16* __restrict__ dY = a.dY;
    const u16* __restrict__ in = a.in;
    const int* __restrict__ pos = a.pos;
    const float* __restrict__ weights = a.weights;
    const int* __restrict__ m_indices = a.m_indices;
    u16* __restrict__ d_in = a.d_in;
    float* __restrict__ d_weights = a.d_weights;
    const int T = a.T, k = a.k, rows = a.rows, N = a.N;
    __shared__ float part[4][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x;
    auto col = [&](int c0, int i) { return VEC ? c0 + lane * 8 + i : c0 + lane + 64 * i; };
    auto load = [&](const u16* p, int c0, float (&v)[8]) {
        u32x4 w = {0u, 0u, 0u, 0u};
        if constexpr (VEC) {
            if (col(c0, 0) < N) w = load16<STREAM>(p + col(c0, 0));
        } else {
            w = load_spread(p, c0 + lane, N);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    };
    auto store = [&](u16* p, int c0, const float (&v)[8]) {
        if constexpr (VEC) {
            if (col(c0, 0) < N)
                store16<STREAM>(p + col(c0, 0), u32x4{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]),
                                                      to_bf16x2(v[4], v[5]), to_bf16x2(v[6], v[7])});
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col(c0, i) < N) p[col(c0, i)] = to_bf16(v[i]);
        }
    };
    if (t >= T) {
        const int blk = t - T;
        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for_padding_rows(m_indices, blk, rows, [&](int r) {
            for (int c0 = wave * 512; c0 < N; c0 += 2048) store(d_in + (u64)r * N, c0, zero);
        });
        return;
    }
    for (int j0 = 0; j0 < k; j0 += 4) {
        int r[4];
        float w[4], dot[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int at = j0 + jj < k ? pos[(u64)t * k + j0 + jj] : -1;
            r[jj] = (u32)at < (u32)rows ? at : -1;
            w[jj] = r[jj] < 0 ? 0.f : weights ? weights[(u64)t * k + j0 + jj] : 1.f;
            dot[jj] = 0.f;
        }
        for (int c0 = wave * 512; c0 < N; c0 += 2048) {
            float g[8];
            load(dY + (u64)t * N, c0, g);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (r[jj] < 0) continue;
                float v[8];
                if (d_weights) {
                    load(in + (u64)r[jj] * N, c0, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[jj] = __builtin_fmaf(g[i], v[i], dot[jj]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = w[jj] * g[i];
                store(d_in + (u64)r[jj] * N, c0, v);
            }
        }
        if (!d_weights) continue;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
            for (int d = 32; d > 0; d /= 2) dot[jj] += __shfl_xor(dot[jj], d);
            if (lane == 0) part[wave][jj] = dot[jj];
        }
        __syncthreads();
        if (threadIdx.x < 4 && j0 + (int)threadIdx.x < k) {
            const int jj = threadIdx.x;
            d_weights[(u64)t * k + j0 + jj] = part[0][jj] + part[1][jj] + part[2][jj] + part[3][jj];
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side
dg_status check_sort(const void* ids, const void* pos, const void* groups, int T, int topk, int G) {
    // an array of no elements may be NULL (so it is for torch's empty tensors)
    if ((T != 0 && (!ids || !pos)) || !groups) return set_error(DG_ERR_INVALID_ARG, "moe_sort: NULL pointer");
    if (T < 0 || topk <= 0 || G <= 0) return set_error(DG_ERR_INVALID_ARG, "moe_sort: sizes must be positive (T may be 0)");
    if (G > kMaxExperts) return set_error(DG_ERR_UNSUPPORTED, "moe_sort: at most 1024 experts");
    if ((int64_t)T * topk > (1 << 30)) return set_error(DG_ERR_UNSUPPORTED, "moe_sort: more than 2^30 assignments");
    if (!aligned(ids, 4) || !aligned(pos, 4) || !aligned(groups, 4))
        return set_error(DG_ERR_ALIGNMENT, "moe_sort: arrays must be 4-byte aligned");
    return DG_OK;
}

dg_status sort(const int32_t* ids, int32_t* pos, int32_t* m_indices, int32_t* group_rows, int T, int topk, int G,
               int masked_rows, int rows, void* stream) {
    const int n = T * topk;
    int bits = 0;
    while ((1 << bits) < G) ++bits;
    // One block (one launch) up to the 4096 ids of its one step; otherwise blocks of
    // 1024 ids or more, counted by a launch of their own (3063 ids, 7 experts: 6.1 us
    // against 1.7 + 4.7 us and a launch between).
    int chunk = kSortStep, blocks = 1;
    u32* hist = nullptr;
    StreamScratch scratch;               // held until both kernels are launched
    if (n > chunk) {
        const int steps = (n + kSortThreads - 1) / kSortThreads;
        chunk = (steps + kSortBlocks - 1) / kSortBlocks * kSortThreads;
        blocks = (n + chunk - 1) / chunk;
        dg_status s = stream_scratch(stream, (size_t)blocks * G * sizeof(u32), &scratch);
        if (s != DG_OK) return s;
        hist = static_cast<u32*>(scratch.p);
        s = launch_rows("moe_sort (count)", dg_moe_count_kernel, dim3(blocks), kSortThreads, stream,
                        CountArgs{ids, hist, n, G, chunk});
        if (s != DG_OK) return s;
    }
    return launch_rows("moe_sort (place)", dg_moe_place_kernel, dim3(blocks), kSortThreads, stream,
                       SortArgs{ids, hist, pos, m_indices, group_rows, n, G, bits, chunk, masked_rows, rows});
}

// the arguments dispatch, combine and combine backward share
dg_status check_rows(const char* what, const void* x, const void* pos, const void* rows_ptr, int T, int topk, int rows,
                     int width) {
    // arrays of no elements may be NULL
    if ((T != 0 && (!x || !pos)) || (rows != 0 && !rows_ptr))
        return set_error(DG_ERR_INVALID_ARG, std::string(what) + ": NULL pointer");
    if (T < 0 || topk <= 0 || rows < 0 || width <= 0)
        return set_error(DG_ERR_INVALID_ARG, std::string(what) + ": sizes must be positive (T and rows may be 0)");
    if (!aligned(x, 16) || !aligned(rows_ptr, 16))
        return set_error(DG_ERR_ALIGNMENT, std::string(what) + ": token and row arrays must be 16-byte aligned");
    if (!aligned(pos, 4)) return set_error(DG_ERR_ALIGNMENT, std::string(what) + ": pos must be 4-byte aligned");
    return DG_OK;
}

// workgroups of four one-wave units; 0: too many for one launch
unsigned grid_of(int64_t units) { return fits_launch((units + 3) / 4) ? (unsigned)((units + 3) / 4) : 0u; }

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

int64_t dg_moe_sorted_rows(int T, int topk, int num_experts) {
    if (T < 0 || topk <= 0 || num_experts <= 0) return -1;
    const int64_t n = (int64_t)T * topk;
    const int64_t used = n < num_experts ? n : num_experts;
    return (n + used * (kAlign - 1) + kAlign - 1) / kAlign * kAlign;
}

dg_status dg_moe_sort_contiguous(const int32_t* expert_ids, int32_t* pos, int32_t* m_indices, int32_t* ks, int T,
                                 int topk, int num_experts, int rows, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_sort(expert_ids, pos, ks, T, topk, num_experts);
        if (s != DG_OK) return s;
        if (rows != 0 && !m_indices) return set_error(DG_ERR_INVALID_ARG, "moe_sort: NULL pointer");
        if (!aligned(m_indices, 4)) return set_error(DG_ERR_ALIGNMENT, "moe_sort: arrays must be 4-byte aligned");
        if (rows < 0) return set_error(DG_ERR_INVALID_ARG, "moe_sort: rows must not be negative");
        if (rows % kAlign) return set_error(DG_ERR_ALIGNMENT, "moe_sort: rows must be a multiple of the M alignment (128)");
        return sort(expert_ids, pos, m_indices, ks, T, topk, num_experts, 0, rows, stream);
    });
}

dg_status dg_moe_sort_masked(const int32_t* expert_ids, int32_t* pos, int32_t* masked_m, int T, int topk,
                             int num_experts, int M_max, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_sort(expert_ids, pos, masked_m, T, topk, num_experts);
        if (s != DG_OK) return s;
        if (M_max <= 0) return set_error(DG_ERR_INVALID_ARG, "moe_sort: M_max must be positive");
        if ((int64_t)M_max * num_experts > INT_MAX) return set_error(DG_ERR_UNSUPPORTED, "moe_sort: more than 2^31 rows");
        return sort(expert_ids, pos, nullptr, masked_m, T, topk, num_experts, M_max, M_max * num_experts, stream);
    });
}

dg_status dg_moe_dispatch_bf16(const void* X, const int32_t* pos, const int32_t* m_indices, void* rows_out, int T,
                               int topk, int rows, int H, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_rows("moe_dispatch_bf16", X, pos, rows_out, T, topk, rows, H);
        if (s != DG_OK) return s;
        if (m_indices && !aligned(m_indices, 4))
            return set_error(DG_ERR_ALIGNMENT, "moe_dispatch_bf16: m_indices must be 4-byte aligned");
        const int pieces = (H + kPiece - 1) / kPiece;
        const int64_t units = ((int64_t)T + (m_indices ? pad_blocks(rows) : 0)) * pieces;
        if (units == 0) return DG_OK;
        const unsigned grid = grid_of(units);
        if (!grid) return set_error(DG_ERR_UNSUPPORTED, "moe_dispatch_bf16: too many tokens for one launch");
        const bool stream_it = 2 * (int64_t)T * (topk + (int64_t)1) * H >= kStreamBytes;
        auto* kernel = H % 8 ? dg_moe_dispatch_bf16_kernel<false, false>
                     : stream_it ? dg_moe_dispatch_bf16_kernel<true, true> : dg_moe_dispatch_bf16_kernel<true, false>;
        return launch_rows("moe_dispatch_bf16", kernel, dim3(grid), 256, stream,
                           DispatchArgs{static_cast<const u16*>(X), pos, m_indices, rows_out, nullptr, T, topk, rows, rows, H,
                                        pieces});
    });
}

dg_status dg_moe_dispatch_fp8(const void* X, const int32_t* pos, const int32_t* m_indices, void* rows_out, void* sf,
                              int T, int topk, int rows, int group_rows, int H, int ue8m0, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_rows("moe_dispatch_fp8", X, pos, rows_out, T, topk, rows, H);
        if (s != DG_OK) return s;
        if (!sf && rows != 0) return set_error(DG_ERR_INVALID_ARG, "moe_dispatch_fp8: NULL pointer");
        if (!aligned(sf, 4) || (m_indices && !aligned(m_indices, 4)))
            return set_error(DG_ERR_ALIGNMENT, "moe_dispatch_fp8: scales and m_indices must be 4-byte aligned");
        if (H % 128) return set_error(DG_ERR_UNSUPPORTED, "moe_dispatch_fp8: H must be a multiple of 128 (the scale block)");
        if (rows > 0 && (group_rows <= 0 || rows % group_rows))
            return set_error(DG_ERR_INVALID_ARG, "moe_dispatch_fp8: rows must be a multiple of group_rows");
        const int pieces = (H + kPiece - 1) / kPiece;
        const int64_t units = ((int64_t)T + (m_indices ? pad_blocks(rows) : 0)) * pieces;
        if (units == 0 || rows == 0) return DG_OK;
        const unsigned grid = grid_of(units);
        if (!grid) return set_error(DG_ERR_UNSUPPORTED, "moe_dispatch_fp8: too many tokens for one launch");
        const bool stream_it = (int64_t)T * (topk + (int64_t)2) * H >= kStreamBytes;
        auto* kernel = ue8m0 ? (stream_it ? dg_moe_dispatch_fp8_kernel<true, true> : dg_moe_dispatch_fp8_kernel<true, false>)
                             : (stream_it ? dg_moe_dispatch_fp8_kernel<false, true> : dg_moe_dispatch_fp8_kernel<false, false>);
        return launch_rows("moe_dispatch_fp8", kernel, dim3(grid), 256, stream,
                           DispatchArgs{static_cast<const u16*>(X), pos, m_indices, rows_out, static_cast<u32*>(sf), T, topk, rows,
                                        group_rows, H, pieces});
    });
}

dg_status dg_moe_combine(const void* rows_in, const int32_t* pos, const float* weights, const void* residual, void* Y,
                         int T, int topk, int rows, int N, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_rows("moe_combine", Y, pos, rows_in, T, topk, rows, N);
        if (s != DG_OK) return s;
        if ((residual && !aligned(residual, 16)) || (weights && !aligned(weights, 4)))
            return set_error(DG_ERR_ALIGNMENT, "moe_combine: residual must be 16-byte, weights 4-byte aligned");
        const int pieces = (N + 511) / 512;
        if (T == 0) return DG_OK;
        const unsigned grid = grid_of((int64_t)T * pieces);
        if (!grid) return set_error(DG_ERR_UNSUPPORTED, "moe_combine: too many tokens for one launch");
        const bool stream_it = 2 * (int64_t)T * (topk + (int64_t)(residual ? 2 : 1)) * N >= kStreamBytes;
        auto* kernel = N % 8 ? dg_moe_combine_kernel<false, false>
                     : stream_it ? dg_moe_combine_kernel<true, true> : dg_moe_combine_kernel<true, false>;
        return launch_rows("moe_combine", kernel, dim3(grid), 256, stream,
                           CombineArgs{static_cast<const u16*>(rows_in), pos, weights, static_cast<const u16*>(residual),
                                       static_cast<u16*>(Y), T, topk, rows, N, pieces});
    });
}

dg_status dg_moe_combine_backward(const void* dY, const void* rows_in, const int32_t* pos, const float* weights,
                                  const int32_t* m_indices, void* d_rows, float* d_weights, int T, int topk, int rows,
                                  int N, void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_rows("moe_combine_backward", dY, pos, d_rows, T, topk, rows, N);
        if (s != DG_OK) return s;
        if (d_weights && !rows_in && rows != 0)
            return set_error(DG_ERR_INVALID_ARG, "moe_combine_backward: the weights' gradient needs the rows");
        if ((rows_in && !aligned(rows_in, 16)) || (weights && !aligned(weights, 4)) || (d_weights && !aligned(d_weights, 4)) ||
            (m_indices && !aligned(m_indices, 4)))
            return set_error(DG_ERR_ALIGNMENT, "moe_combine_backward: rows must be 16-byte, the other arrays 4-byte aligned");
        const int64_t blocks = (int64_t)T + (m_indices ? pad_blocks(rows) : 0);
        if (blocks == 0) return DG_OK;
        if (!fits_launch(blocks)) return set_error(DG_ERR_UNSUPPORTED, "moe_combine_backward: too many tokens for one launch");
        const bool stream_it = 2 * (int64_t)T * (topk * (int64_t)(d_weights ? 2 : 1) + 1) * N >= kStreamBytes;
        auto* kernel = N % 8 ? dg_moe_combine_backward_kernel<false, false>
                     : stream_it ? dg_moe_combine_backward_kernel<true, true> : dg_moe_combine_backward_kernel<true, false>;
        return launch_rows("moe_combine_backward", kernel, dim3((unsigned)blocks), 256, stream,
                           CombineBackwardArgs{static_cast<const u16*>(dY), static_cast<const u16*>(rows_in), pos, weights,
                                               m_indices, static_cast<u16*>(d_rows), d_weights, T, topk, rows, N});
    });
}

}  // extern "C"
