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
#include "row_kernels.h"

namespace dg {
namespace {

// The largest row: 1024 lanes of 8 chunks.
constexpr int kMaxWidth = 65536;

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

// Gradient.  Workgroup b takes rows b, b + grid, ...: the weight's gradient of its rows stays in
// registers and goes to row b of `partial`, whose columns a second kernel adds in a fixed order.
struct NormBackwardArgs {
    const u16* dY;
    const u16* S;
    const void* weight;
    const u16* dS;
    u16* dX;
    float* partial;
    float eps;
    int wide_weight, T, H;
};
template <int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS) dg_rms_norm_backward_kernel(const NormBackwardArgs a) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int H = a.H;
    __shared__ float parts[2][2][THREADS / 64];
    float dw[CHUNKS][8];
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
    int turn = 0;
    for (u32 t = blockIdx.x; t < (u32)a.T; t += gridDim.x, turn ^= 1) {
        const u64 at = (u64)t * (u64)H;
        u32x4 xs[CHUNKS], ys[CHUNKS], ds[CHUNKS];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int c = (k * THREADS + tid) * 8;
            xs[k] = load8(a.S + at, c, H);
            ys[k] = load8(a.dY + at, c, H);
        }
        if (a.dS) {
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) ds[k] = load8(a.dS + at, (k * THREADS + tid) * 8, H);
        }
        float ss = 0.f, gs = 0.f;              // sums of s^2 and of g s
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            float s[8], y[8], w[8];
            unpack8(xs[k], s);
            unpack8(ys[k], y);
            load_weight(a.weight, a.wide_weight, (k * THREADS + tid) * 8, H, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(s[i], s[i], ss);
                gs = __builtin_fmaf(y[i] * w[i], s[i], gs);
            }
        }
        ss = wave_sum(ss);
        gs = wave_sum(gs);
        if constexpr (THREADS > 64) {
            // (two sets in turn: a wave writes a set again only after the barrier of the row between)
            if (lane == 0) {
                parts[turn][0][tid >> 6] = ss;
                parts[turn][1][tid >> 6] = gs;
            }
            __syncthreads();
            ss = gs = 0.f;
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) {
                ss += parts[turn][0][w];
                gs += parts[turn][1][w];
            }
        }
        const float q = 1.f / __builtin_sqrtf(ss / (float)H + a.eps);
        const float back = gs / (float)H * q * q;          // mean(g n) q, so that n mean(g n) = s back
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int c = (k * THREADS + tid) * 8;
            float s[8], y[8], w[8], v[8];
            unpack8(xs[k], s);
            unpack8(ys[k], y);
            load_weight(a.weight, a.wide_weight, c, H, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[k][i] = __builtin_fmaf(y[i], s[i] * q, dw[k][i]);
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
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        const int c = (k * THREADS + tid) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < H) to[c + i] = dw[k][i];
    }
}

// Lanes and chunks that hold a row of H, at most `chunks` chunks where 1024 lanes suffice.
struct Shape {
    int threads, chunks;
};
Shape shape_of(int H, int chunks) {
    int threads = 64;
    while (threads < 1024 && threads * chunks * 8 < H) threads *= 4;
    while (threads * chunks * 8 < H) chunks *= 2;
    while (chunks > 1 && threads * (chunks / 2) * 8 >= H) chunks /= 2;
    return {threads, chunks};
}

template <template <int, int> class K, typename Args>
dg_status launch_shape(const char* what, Shape s, unsigned grid, void* stream, const Args& a) {
    void (*kernel)(Args) = nullptr;
    switch (s.threads * 16 + s.chunks) {
        case 64 * 16 + 1: kernel = K<64, 1>::f; break;
        case 64 * 16 + 2: kernel = K<64, 2>::f; break;
        case 64 * 16 + 4: kernel = K<64, 4>::f; break;
        case 256 * 16 + 1: kernel = K<256, 1>::f; break;
        case 256 * 16 + 2: kernel = K<256, 2>::f; break;
        case 256 * 16 + 4: kernel = K<256, 4>::f; break;
        case 1024 * 16 + 1: kernel = K<1024, 1>::f; break;
        case 1024 * 16 + 2: kernel = K<1024, 2>::f; break;
        case 1024 * 16 + 4: kernel = K<1024, 4>::f; break;
        default: kernel = K<1024, 8>::f; break;
    }
    return launch_rows(what, kernel, dim3(grid), s.threads, stream, a);
}
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
    if (H > kMaxWidth) return set_error(DG_ERR_UNSUPPORTED, name + ": rows are at most 65536 wide");
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
        const Shape shape = shape_of(H, 4);
        const u32 each = ((u32)T + kXcds - 1) / kXcds;
        if (!fits_launch((int64_t)each * kXcds, shape.threads))
            return set_error(DG_ERR_UNSUPPORTED, "rms_norm: too many rows for one launch");
        return launch_shape<Forward>("rms_norm", shape, each * kXcds, stream,
                                     NormArgs{static_cast<const u16*>(X), static_cast<const u16*>(n.residual), n.weight,
                                              static_cast<u16*>(n.S), static_cast<u16*>(n.Y), static_cast<u8*>(n.Q),
                                              static_cast<u32*>(n.sf), n.eps, n.weight_type == DG_TYPE_F32, n.ue8m0 != 0, T,
                                              H, each});
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
        const Shape shape = shape_of(H, 4);
        const unsigned grid = (unsigned)std::min(T, 1024);
        float* partial = nullptr;
        StreamScratch scratch;               // held until both kernels are launched
        if (dweight && T > 0) {
            s = stream_scratch(stream, (size_t)grid * (size_t)H * sizeof(float), &scratch);
            if (s != DG_OK) return s;
            partial = static_cast<float*>(scratch.p);
        }
        if (T > 0) {
            s = launch_shape<Backward>("rms_norm_backward", shape, grid, stream,
                                       NormBackwardArgs{static_cast<const u16*>(dY), static_cast<const u16*>(S), weight,
                                                        static_cast<const u16*>(dS), static_cast<u16*>(dX), partial, eps,
                                                        weight_type == DG_TYPE_F32, T, H});
            if (s != DG_OK) return s;
        }
        return dweight ? column_sums("rms_norm_backward (weight)", partial, nullptr, (int)grid, 1, H, 1, dweight, stream) : DG_OK;
    });
}

}  // extern "C"
