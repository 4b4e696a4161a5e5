// Root-mean-square norm with the residual's addition (hipcc, gfx950), BF16 and
// quantised outputs, and its gradient.  The operations and their layouts are
// specified in include/dg.h.
//
//   s = x + r,  q = (mean(s^2) + eps)^-1/2,  y = s q w
//   gradient, with n = s q and g = dy w:   dx = q (g - n mean(g n)) + ds,   dw = sum over rows of dy n
//
// A pass over rows: a few operations an element (about 20 more where it
// quantises), so what bounds it is HBM, and for few rows the launch and one
// round trip.  One workgroup holds a row in registers between its one read and
// the writes, 8 consecutive elements a lane and chunk, so that a row is read
// once; sums are FP32 from lane to row.
#include <utility>

#include "row_kernels.h"

namespace dg {
namespace {

// The largest row: 1024 lanes of four chunks.
constexpr int kMaxWidth = 32768;

// Eight elements of the weight, FP32 or BF16
__device__ __forceinline__ void load_weight(const void* weight, int wide, int c, int H, float (&w)[8]) {
    if (!weight) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
    } else if (wide) {
        const float* p = static_cast<const float*>(weight);
        if (c + 8 <= H) {
            __builtin_memcpy(w, p + c, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = c + i < H ? p[c + i] : 0.f;
        }
    } else {
        unpack8(load8(static_cast<const u16*>(weight), c, H), w);
    }
}

template <int D>
__device__ __forceinline__ float add_rotated(float v) {
    return v + __builtin_bit_cast(float, rotate16<D>(__builtin_bit_cast(u32, v)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
    auto part = [&](int lane) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    };
    return (part(0) + part(16)) + (part(32) + part(48));
}

// Workgroups go to the 8 XCDs in turn.  Here XCD x takes the x-th eighth of the rows, so that
// neighbouring rows, whose scales are neighbours in memory, are written through one L2.
constexpr u32 kXcds = 8;
__device__ __forceinline__ u32 row_of(u32 block, u32 each) { return block % kXcds * each + block / kXcds; }

struct NormArgs {
    const u16* X;
    const u16* residual;
    const void* weight;
    u16* S;
    u16* Y;
    u8* Q;
    u32* sf;
    float eps;
    int wide_weight, ue8m0, T, H;
    u32 each;                              // rows an XCD takes
};

// No pointer here is __restrict__: S may be X or the residual, Y may be X.  A lane reads its
// elements of a row before it writes them.
template <int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS) dg_rms_norm_kernel(const NormArgs a) {
    const int tid = threadIdx.x, lane = tid & 63;
    const u32 t = row_of(blockIdx.x, a.each);
    if (t >= (u32)a.T) return;
    const int H = a.H;
    const u64 at = (u64)t * (u64)H;
    u32x4 xs[CHUNKS], rs[CHUNKS];
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) xs[k] = load8(a.X + at, (k * THREADS + tid) * 8, H);
    if (a.residual) {
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) rs[k] = load8(a.residual + at, (k * THREADS + tid) * 8, H);
    }
    float s[CHUNKS][8];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        unpack8(xs[k], s[k]);
        if (a.residual) {
            float r[8];
            unpack8(rs[k], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[k][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(s[k][i], s[k][i], sum);
    }
    sum = wave_sum(sum);
    if constexpr (THREADS > 64) {
        __shared__ float parts[THREADS / 64];
        if (lane == 0) parts[tid >> 6] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) sum += parts[w];
    }
    const float q = 1.f / __builtin_sqrtf(sum / (float)H + a.eps);
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        const int c = (k * THREADS + tid) * 8;
        if (a.S) store8(a.S + at, c, H, pack8(s[k]));
        float y[8], w[8];
        load_weight(a.weight, a.wide_weight, c, H, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = s[k][i] * q * w[i];
        if (a.Y) store8(a.Y + at, c, H, pack8(y));
        if (!a.Q) continue;
        // one scale per 16 lanes (H is a multiple of 128), as dg_moe_dispatch_fp8: the largest magnitude over
        // the bit patterns, the correctly rounded quotient
        u32 top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u32 m = __builtin_bit_cast(u32, y[i]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        top = max16(top);
        float scale = __builtin_bit_cast(float, top) / 448.f;
        if (scale < 0x1p-126f) scale = 0x1p-126f;
        if (top == 0u) scale = 1.f;
        if (a.ue8m0) {
            const u32 bits = __builtin_bit_cast(u32, scale);
            u32 e = (bits >> 23) + ((bits & 0x7fffffu) ? 1u : 0u);
            if (e > 255u) e = 255u;
            scale = __builtin_bit_cast(float, e == 255u ? 0x7fc00000u : e << 23);
            if (c >= H) e = 127u;
            // a wave's chunk is 512 columns: one word of four blocks
            const u32 word = (u32)__builtin_amdgcn_readlane((int)e, 0) | (u32)__builtin_amdgcn_readlane((int)e, 16) << 8 |
                             (u32)__builtin_amdgcn_readlane((int)e, 32) << 16 |
                             (u32)__builtin_amdgcn_readlane((int)e, 48) << 24;
            if (lane == 0 && c < H) a.sf[(u64)(c >> 9) * (u32)a.T + t] = word;
        } else if ((lane & 15) == 0 && c < H) {
            a.sf[(u64)(c >> 7) * (u32)a.T + t] = __builtin_bit_cast(u32, scale);
        }
        u32 code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = y[4 * h + i] / scale;
                v[i] = v[i] > 448.f ? 448.f : v[i];          // (a NaN passes both)
                v[i] = v[i] < -448.f ? -448.f : v[i];
            }
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            code[h] = (u32)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
        }
        if (c < H) *(u64*)(a.Q + at + c) = (u64)code[1] << 32 | code[0];
    }
}

// Gradient.  A workgroup is `teams` teams of THREADS lanes, a row a team at a time; the weight's gradient of a
// team's rows stays in registers (in LDS for rows of several chunks), the teams' meet in LDS, and the sum goes to row b
// of `partial`, whose columns a second kernel adds, all in a fixed order.  Few partial rows count: written and read back
// they were a quarter of the pass (8192 x 4096: 1024 workgroups of one team 60 us, 45 of it without the weight's gradient).
struct NormBackwardArgs {
    const u16* dY;
    const u16* S;
    const void* weight;
    const u16* dS;
    u16* dX;
    float* partial;
    float eps;
    int wide_weight, T, H;
    int teams, turns;
};
template <int THREADS, int CHUNKS>
__global__ void __launch_bounds__(1024) dg_rms_norm_backward_kernel(const NormBackwardArgs a) {
    constexpr int WAVES = THREADS / 64;
    const int team = __builtin_amdgcn_readfirstlane(threadIdx.x / THREADS), tid = threadIdx.x % THREADS;
    const int lane = threadIdx.x & 63, wave = tid >> 6;
    const int H = a.H;
    __shared__ float parts[2][2][16];                        // [turn][sum][wave of the workgroup]
    // the teams' sums (one chunk), or this team's (several): a lane's own eight a chunk
    __shared__ __attribute__((aligned(16))) float gathered[THREADS < 1024 || CHUNKS > 1 ? THREADS * CHUNKS * 8 : 1];
    float dw[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    f32x4* const own = (f32x4*)gathered + 2 * tid;           // chunk k: 2 THREADS k further
    if constexpr (CHUNKS > 1) {
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) own[2 * THREADS * k] = own[2 * THREADS * k + 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // (the weight of one chunk is kept; that of more is read from the cache each time, for want of registers)
    if constexpr (CHUNKS == 1) load_weight(a.weight, a.wide_weight, tid * 8, H, w);
    auto weight_of = [&](int k) {
        if constexpr (CHUNKS > 1) load_weight(a.weight, a.wide_weight, (k * THREADS + tid) * 8, H, w);
    };
    for (int turn = 0; turn < a.turns; ++turn) {
        const u32 t = ((u32)turn * gridDim.x + blockIdx.x) * (u32)a.teams + (u32)team;
        const u64 at = (u64)t * (u64)H;
        u32x4 xs[CHUNKS], ys[CHUNKS], ds[CHUNKS];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int c = (k * THREADS + tid) * 8;
            xs[k] = ys[k] = ds[k] = u32x4{0u, 0u, 0u, 0u};
            if (t < (u32)a.T) {
                xs[k] = load8(a.S + at, c, H);
                ys[k] = load8(a.dY + at, c, H);
                if (a.dS) ds[k] = load8(a.dS + at, c, H);
            }
        }
        float ss = 0.f, gs = 0.f;              // sums of s^2 and of g s
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            float s[8], y[8];
            weight_of(k);
            unpack8(xs[k], s);
            unpack8(ys[k], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(s[i], s[i], ss);
                gs = __builtin_fmaf(y[i] * w[i], s[i], gs);
            }
        }
        ss = wave_sum(ss);
        gs = wave_sum(gs);
        if constexpr (WAVES > 1) {
            // (two sets in turn: a wave writes a set again only after the barrier of the row between)
            float(&set)[2][16] = parts[turn & 1];
            if (lane == 0) {
                set[0][team * WAVES + wave] = ss;
                set[1][team * WAVES + wave] = gs;
            }
            __syncthreads();
            ss = gs = 0.f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                ss += set[0][team * WAVES + i];
                gs += set[1][team * WAVES + i];
            }
        }
        // (opaque: otherwise the unpacked values are kept over the barrier, in twice the registers)
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) asm volatile("" : "+v"(xs[k]), "+v"(ys[k]));
        if (t >= (u32)a.T) continue;
        const float q = 1.f / __builtin_sqrtf(ss / (float)H + a.eps);
        const float back = gs / (float)H * q * q;          // mean(g n) q, so that n mean(g n) = s back
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int c = (k * THREADS + tid) * 8;
            float s[8], y[8], v[8];
            weight_of(k);
            unpack8(xs[k], s);
            unpack8(ys[k], y);
            if constexpr (CHUNKS > 1) {
                f32x4* const sum = own + 2 * THREADS * k;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4 n;
#pragma unroll
                    for (int e = 0; e < 4; ++e) n[e] = y[4 * h + e] * (s[4 * h + e] * q);
                    sum[h] += n;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (CHUNKS == 1) dw[i] = __builtin_fmaf(y[i], s[i] * q, dw[i]);
                v[i] = q * __builtin_fmaf(-s[i], back, y[i] * w[i]);
            }
            if (a.dS) {
                float d[8];
                unpack8(ds[k], d);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += d[i];
            }
            if (a.dX) store8(a.dX + at, c, H, pack8(v));
        }
    }
    if (!a.partial) return;
    float* to = a.partial + (u64)blockIdx.x * (u64)H;
    if constexpr (THREADS < 1024) {
        // team after team adds its sums; the last stores them
        for (int i = 0; i < a.teams; ++i) {
            __syncthreads();
            if (team != i) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 v = {dw[4 * h], dw[4 * h + 1], dw[4 * h + 2], dw[4 * h + 3]};
                if (i > 0) v = own[h] + v;
                if (i + 1 < a.teams) own[h] = v;
#pragma unroll
                for (int e = 0; e < 4; ++e) dw[4 * h + e] = v[e];
            }
        }
        if (team != a.teams - 1) return;
    }
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        const int c = (k * THREADS + tid) * 8;
        if constexpr (CHUNKS > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[i] = own[2 * THREADS * k + (i >> 2)][i & 3];
        }
        if (c + 8 <= H) {
            __builtin_memcpy(to + c, dw, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < H) to[c + i] = dw[i];
        }
    }
}

constexpr int kBackwardGroups = 256;

// Lanes and chunks of 8 elements each that hold a row.
struct Shape {
    int threads, chunks;
};
// Forward: as many lanes as chunks of the row where rows are few or wide; a wave alone (no barrier) or four and
// two chunks a lane where many narrow rows fill the CUs.  us, 1024 lanes and 256 (64): 32 x 7168 to E4M3
// 4.5 and 6.1, 8192 x 7168 in BF16 and E4M3 106 and 110, 8192 x 4096 72 and 58; 8192 x 1024 48, 18 and (15.6), 32 x
// 1024 3.8, 3.4 and (4.1).
Shape forward_shape(int T, int H) {
    if (H <= 512) return {64, 1};
    if (H <= 1024 && T > 512) return {64, 2};
    if (H <= 2048) return {256, 1};
    if (H <= 4096 && T > 512) return {256, 2};
    int chunks = 1;
    while (1024 * chunks * 8 < H) chunks *= 2;
    return {1024, chunks};
}
Shape backward_shape(int H) {
    int threads = 64, chunks = 1;
    while (threads < 1024 && threads * 8 < H) threads *= 2;
    while (threads * chunks * 8 < H) chunks *= 2;
    return {threads, chunks};
}

template <template <int, int> class K, typename Args, int... SHAPES>
dg_status launch_shape(const char* what, Shape s, unsigned grid, int teams, void* stream, const Args& a,
                       std::integer_sequence<int, SHAPES...>) {
    void (*kernel)(Args) = nullptr;
    (void)((s.threads * 16 + s.chunks == SHAPES && (kernel = K<SHAPES / 16, SHAPES % 16>::f)) || ...);
    return launch_rows(what, kernel, dim3(grid), s.threads * teams, stream, a);
}
// threads * 16 + chunks of the shapes above
using ForwardShapes = std::integer_sequence<int, 64 * 16 + 1, 64 * 16 + 2, 256 * 16 + 1, 256 * 16 + 2, 1024 * 16 + 1,
                                            1024 * 16 + 2, 1024 * 16 + 4>;
using BackwardShapes = std::integer_sequence<int, 64 * 16 + 1, 128 * 16 + 1, 256 * 16 + 1, 512 * 16 + 1, 1024 * 16 + 1,
                                             1024 * 16 + 2, 1024 * 16 + 4>;
template <int T, int C>
struct Forward {
    static constexpr auto f = dg_rms_norm_kernel<T, C>;
};
template <int T, int C>
struct Backward {
    static constexpr auto f = dg_rms_norm_backward_kernel<T, C>;
};

dg_status check_norm(const char* what, bool null, const void* weight, int weight_type, float eps, int T, int H) {
    const std::string name(what);
    if (T < 0 || H <= 0) return set_error(DG_ERR_INVALID_ARG, name + ": sizes must be positive (T may be 0)");
    if (null) return set_error(DG_ERR_INVALID_ARG, name + ": NULL pointer");
    if (H > kMaxWidth) return set_error(DG_ERR_UNSUPPORTED, name + ": rows are at most 32768 wide");
    if (weight && weight_type != DG_TYPE_F32 && weight_type != DG_TYPE_BF16)
        return set_error(DG_ERR_INVALID_ARG, name + ": unknown weight type");
    if (!(eps >= 0.f)) return set_error(DG_ERR_INVALID_ARG, name + ": eps must not be negative");
    if (weight && !aligned(weight, 16)) return set_error(DG_ERR_ALIGNMENT, name + ": weight must be 16-byte aligned");
    return DG_OK;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_rms_norm(const void* X, const dg_norm* norm, int T, int H, void* stream) {
    return guarded([&]() -> dg_status {
        if (!norm) return set_error(DG_ERR_INVALID_ARG, "rms_norm: NULL pointer");
        const dg_norm n = *norm;
        const bool null = T > 0 && (!X || (n.Q && !n.sf) || (!n.Y && !n.Q && !n.S));
        dg_status s = check_norm("rms_norm", null, n.weight, n.weight_type, n.eps, T, H);
        if (s != DG_OK) return s;
        if (!aligned(X, 16) || !aligned(n.residual, 16) || !aligned(n.S, 16) || !aligned(n.Y, 16) || !aligned(n.Q, 16))
            return set_error(DG_ERR_ALIGNMENT, "rms_norm: row arrays must be 16-byte aligned");
        if (!aligned(n.sf, 4)) return set_error(DG_ERR_ALIGNMENT, "rms_norm: scales must be 4-byte aligned");
        if (n.S && n.S == n.Y) return set_error(DG_ERR_INVALID_ARG, "rms_norm: S and Y must not be the same array");
        if (n.Q && H % 128)
            return set_error(DG_ERR_UNSUPPORTED, "rms_norm: H must be a multiple of 128 (the scale block) for E4M3 rows");
        if (T == 0) return DG_OK;
        const Shape shape = forward_shape(T, H);
        const u32 each = ((u32)T + kXcds - 1) / kXcds;
        if (!fits_launch((int64_t)each * kXcds, shape.threads))
            return set_error(DG_ERR_UNSUPPORTED, "rms_norm: too many rows for one launch");
        return launch_shape<Forward>("rms_norm", shape, each * kXcds, 1, stream,
                                     NormArgs{static_cast<const u16*>(X), static_cast<const u16*>(n.residual), n.weight,
                                              static_cast<u16*>(n.S), static_cast<u16*>(n.Y), static_cast<u8*>(n.Q),
                                              static_cast<u32*>(n.sf), n.eps, n.weight_type == DG_TYPE_F32, n.ue8m0 != 0, T,
                                              H, each},
                                     ForwardShapes{});
    });
}

dg_status dg_rms_norm_backward(const void* dY, const void* S, const void* weight, int weight_type, float eps,
                               const void* dS, void* dX, float* dweight, int T, int H, void* stream) {
    return guarded([&]() -> dg_status {
        const bool null = (T > 0 && (!dY || !S)) || (!dX && !dweight && T > 0);
        dg_status s = check_norm("rms_norm_backward", null, weight, weight_type, eps, T, H);
        if (s != DG_OK) return s;
        if (!aligned(dY, 16) || !aligned(S, 16) || !aligned(dS, 16) || !aligned(dX, 16))
            return set_error(DG_ERR_ALIGNMENT, "rms_norm_backward: row arrays must be 16-byte aligned");
        if (!aligned(dweight, 4)) return set_error(DG_ERR_ALIGNMENT, "rms_norm_backward: dweight must be 4-byte aligned");
        const Shape shape = backward_shape(H);
        // 1024 lanes a workgroup and a workgroup a CU; fewer teams where there are not the rows for that, two
        // workgroups a CU (of up to 512 lanes a row they fit) where each still has two turns.  us with 256, 512 and
        // 1024: 8192 x 4096 52.5, 48.8, 53.9; 8192 x 1024 18.5, 17.5, 20.7; 2048 x 2048 12.7, 14.4, 15.5; 8192 x
        // 7168 97.9, 99.9, 108.8.  (The next row's loads ahead of the present one's sums: 52.1 and 57.2 for the first.)
        int teams = 1024 / shape.threads, groups = kBackwardGroups;
        while (teams > 1 && (int64_t)groups * teams > T) teams /= 2;
        if (shape.threads < 1024 && T >= (int64_t)4 * groups * teams) groups *= 2;
        const unsigned grid = (unsigned)std::min(((int64_t)T + teams - 1) / teams, (int64_t)groups);
        const int turns = grid ? (int)(((int64_t)T + (int64_t)grid * teams - 1) / ((int64_t)grid * teams)) : 0;
        float* partial = nullptr;
        StreamScratch scratch;               // held until both kernels are launched
        if (dweight && T > 0) {
            s = stream_scratch(stream, (size_t)grid * (size_t)H * sizeof(float), &scratch);
            if (s != DG_OK) return s;
            partial = static_cast<float*>(scratch.p);
        }
        if (T > 0) {
            s = launch_shape<Backward>("rms_norm_backward", shape, grid, teams, stream,
                                       NormBackwardArgs{static_cast<const u16*>(dY), static_cast<const u16*>(S), weight,
                                                        static_cast<const u16*>(dS), static_cast<u16*>(dX), partial, eps,
                                                        weight_type == DG_TYPE_F32, T, H, teams, turns},
                                       BackwardShapes{});
            if (s != DG_OK) return s;
        }
        return dweight ? column_sums("rms_norm_backward (weight)", partial, nullptr, (int)grid, 1, H, 1, dweight, stream) : DG_OK;
    });
}

}  // extern "C"
