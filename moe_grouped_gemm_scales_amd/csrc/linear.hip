// Backward side of the products with a fused epilogue (hipcc, gfx950): the
// activation's gradient with the bias gradient in the same pass, and the
// K-contiguous rewrite of BF16 operands for the NN and TN products.  The
// operations are specified in include/dg.h.
#include "row_kernels.h"

namespace dg {
namespace {

// ---------------------------------------------------------------- K-contiguous rewrite
// X [rows_k][cols] -> Xt [cols][pitch], columns [rows_k, k_end) of Xt zero.  One
// workgroup a 64 x 64 block through LDS: 16-byte loads along cols, 16-byte
// stores along K.  A row of the LDS block is 33 words, so the gather of a
// column (four lanes 16 rows apart, 16 columns a wave) touches 32 distinct
// banks.  K blocks fastest, as in the FP8 rewrite.
struct TransposeArgs {
    const u16* X;
    u16* Xt;
    int rows_k, cols, k_blocks;
    long long pitch;
};
__global__ void __launch_bounds__(256) dg_transpose_bf16_kernel(const TransposeArgs a) {
    const u16* __restrict__ X = a.X;
    u16* __restrict__ Xt = a.Xt;
    const int rows_k = a.rows_k, cols = a.cols, k_blocks = a.k_blocks;
    const long long pitch = a.pitch;
    __shared__ __attribute__((aligned(4))) u16 tile[64][66];
    const int tid = threadIdx.x;
    const int k0 = (int)(blockIdx.x % (u32)k_blocks) * 64, c0 = (int)(blockIdx.x / (u32)k_blocks) * 64;
    X += (u64)blockIdx.z * (u64)rows_k * (u64)cols;
    Xt += (u64)blockIdx.z * (u64)cols * (u64)pitch;
    const int r = tid >> 2, piece = (tid & 3) * 16;
    {
        const int k = k0 + r, c = c0 + piece;
        u32 w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        if (k < rows_k) {
            const u16* src = X + (u64)k * (u64)cols + c;
            if ((cols & 7) == 0) {                          // every 8-element group is whole and aligned
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (c + 8 * h < cols) {
                        const u32x4 x = *(const u32x4*)(src + 8 * h);
                        w[4 * h] = x.x; w[4 * h + 1] = x.y; w[4 * h + 2] = x.z; w[4 * h + 3] = x.w;
                    }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols) w[i >> 1] |= (u32)src[i] << (16 * (i & 1));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) *(u32*)&tile[r][piece + 2 * j] = w[j];
    }
    __syncthreads();
    const int c = c0 + r;
    if (c < cols) {
        u32 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (u32)tile[piece + 2 * j][r] | ((u32)tile[piece + 2 * j + 1][r] << 16);
        u16* dst = Xt + (u64)c * (u64)pitch + k0 + piece;
        *(u32x4*)dst = u32x4{w[0], w[1], w[2], w[3]};
        *(u32x4*)(dst + 8) = u32x4{w[4], w[5], w[6], w[7]};
    }
}

// ---------------------------------------------------------------- whole K blocks
// X [rows][cols] -> Xp [rows][pitch], columns past cols zero: the K-contiguous operand of a product
// whose K ends inside a block.  16 bytes a store; rows of X have any alignment, their elements are
// read one by one with clamped indices, all eight together.
// Bound by HBM: 8192 x 4478 (147 MB) 37.9 us, 3.9 TB/s.  The whole NN product of 8192 x 4096 over
// K = 4478 takes 264 us, 220 over 4480, which is read as stored; over 1000 85, over 1024 68.
struct PadArgs {
    const u16* X;
    u16* Xp;
    u32 cols, pieces;
    u64 total;
};
__global__ void __launch_bounds__(256) dg_pad_rows_bf16_kernel(const PadArgs a) {
    for (u64 i = (u64)blockIdx.x * 256u + threadIdx.x; i < a.total; i += (u64)gridDim.x * 256u) {
        const u64 row = i / a.pieces;
        const u32 c = (u32)(i - row * a.pieces) * 8u;
        const u16* src = a.X + row * a.cols;
        u32 v[8];
#pragma unroll
        for (u32 e = 0; e < 8; ++e) v[e] = src[c + e < a.cols ? c + e : a.cols - 1];
        u32x4 w;
#pragma unroll
        for (u32 h = 0; h < 4; ++h)
            w[h] = (c + 2 * h < a.cols ? v[2 * h] : 0u) | (c + 2 * h + 1 < a.cols ? v[2 * h + 1] << 16 : 0u);
        *(u32x4*)(a.Xp + i * 8) = w;
    }
}

// ---------------------------------------------------------------- activation and bias gradient
// d act / d z in FP32.  exp2 and the reciprocal are the hardware's (1 ulp), Phi's tail is the
// rational fit of the forward epilogue (relative error 7e-8 before FP32's roundings, its
// e^(-z^2/2) shared with the density): errors of FP32's own size, which the bias
// gradient's sum averages.  With the device library's expf, erff and division the
// pass was bound by its arithmetic (8192 x 4096, GELU: 55 us against 45; 2304 x
// 2112, tanh form: 12.4 against 9.2).  A fit that keeps only the absolute error
// small (1.5e-7 of erf) has three terms fewer and is off by 1 % at z = -8: 43.7 us
// against 44.5.
// Past |z| = 16 the slopes are 0 or 1 to the last bit (SiLU: past 200 its tail is
// below FP32); z is cut there, so that no infinity meets a zero.  A NaN stays a NaN.
__device__ __forceinline__ float cut(float z, float far) { return z > far ? far : z < -far ? -far : z; }
__device__ __forceinline__ float logistic2(float x) {      // 1 / (1 + 2^-x)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x));
}
template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == DG_ACT_RELU) return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    if constexpr (ACT == DG_ACT_SILU) {
        z = cut(z, 200.f);
        const float s = logistic2(1.44269504f * z);
        return s * __builtin_fmaf(z, 1.f - s, 1.f);
    }
    if constexpr (ACT == DG_ACT_GELU) {
        z = cut(z, 16.f);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.30405593f, __builtin_fabsf(z), 1.f));
        const float e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
        float y = __builtin_fmaf(t, 0.036534112f, -0.15392894f);
        y = __builtin_fmaf(t, y, 0.18981865f);
        y = __builtin_fmaf(t, y, -0.041117497f);
        y = __builtin_fmaf(t, y, 0.12256832f);
        y = __builtin_fmaf(t, y, 0.10271288f);
        y = __builtin_fmaf(t, y, 0.12215308f);
        const float tail = __builtin_fmaf(t, y, 0.12125936f) * t * e;       // Phi(-|z|)
        return __builtin_fmaf(0.39894228f * z, e, z < 0.f ? tail : 1.f - tail);
    }
    if constexpr (ACT == DG_ACT_GELU_TANH) {
        z = cut(z, 16.f);
        const float s = logistic2(2.30220820f * z * __builtin_fmaf(0.044715f * z, z, 1.f));
        return __builtin_fmaf(z * s * (1.f - s), __builtin_fmaf(0.21406445f * z, z, 1.59576912f), s);
    }
    return 1.f;
}

// dZ = dD slope(Z), and the column sums of dZ (FP32, before its rounding) of the
// workgroup's rows.  A workgroup takes 512 columns of `chunk` rows, 16 at a time:
// 8 columns a lane, its four waves every fourth row.  A wave's loads of the 16
// are all issued before its first use of one (4 rows of dD and Z in flight), the
// waves' sums meet in LDS and are added in wave order.  Contiguous form: the rows
// of a chunk (it divides 128) belong to the expert of its first row; padding rows (-1)
// get dZ = 0, rows past the last segment are untouched.  partial [chunks][N], or
// nullptr: no bias gradient.
constexpr int kStep = 16;                 // rows a workgroup holds at once
constexpr int kWaveRows = kStep / 4;
struct BackwardArgs {
    const u16* dD;
    const u16* Z;
    const int* m_indices;
    u16* dZ;
    float* partial;
    int rows, N, G, chunk;
};
// STREAM: dD and Z are read with the non-temporal hint (8192 x 4096: 46.6 us against
// 51.4; 4096 x 4096, 100 MB in all, 27.9 against 26.2, so only from kStreamBytes on).
// dZ is not: the products read it next.
template <int ACT, bool VEC, bool STREAM>
__global__ void __launch_bounds__(256) dg_epilogue_backward_kernel(const BackwardArgs a) {
    const u16* __restrict__ dD = a.dD;
    const u16* __restrict__ Z = a.Z;
    const int* __restrict__ m_indices = a.m_indices;
    u16* __restrict__ dZ = a.dZ;
    float* __restrict__ partial = a.partial;
    const int rows = a.rows, N = a.N, G = a.G;
    __shared__ __attribute__((aligned(16))) float sums[4][512];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = (int)blockIdx.y * 512;
    const int first = (int)blockIdx.x * a.chunk;
    const int last = rows - first < a.chunk ? rows : first + a.chunk;
    auto col = [&](int i) { return VEC ? c0 + lane * 8 + i : c0 + lane + 64 * i; };
    auto load = [&](const u16* p) {        // eight BF16
        u32x4 w = {0u, 0u, 0u, 0u};
        if constexpr (VEC) {
            if (col(0) < N) {
                if constexpr (STREAM) w = __builtin_nontemporal_load((const u32x4*)(p + col(0)));
                else w = *(const u32x4*)(p + col(0));
            }
        } else {
            w = load_spread(p, c0 + lane, N);
        }
        return w;
    };
    const int owner = m_indices ? m_indices[first] : 0;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int r0 = first + wave; r0 < last; r0 += kStep) {
        // the expert of each of this wave's four rows (below 0: padding, or no row)
        int expert[kWaveRows];
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i)
            expert[i] = r0 + 4 * i >= last ? kPadding - 1 : m_indices ? m_indices[r0 + 4 * i] : 0;
        u32x4 d[kWaveRows], z[kWaveRows];
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i) {
            d[i] = z[i] = u32x4{0u, 0u, 0u, 0u};
            if ((u32)expert[i] < (u32)G) {
                const u64 at = (u64)(r0 + 4 * i) * N;
                d[i] = load(dD + at);
                if constexpr (ACT != DG_ACT_NONE) z[i] = load(Z + at);
            }
        }
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i) {
            const bool real = (u32)expert[i] < (u32)G;
            if (!real && expert[i] != kPadding) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = e & 1 ? bf16_hi(d[i][e >> 1]) : bf16_lo(d[i][e >> 1]);
                if constexpr (ACT != DG_ACT_NONE)
                    if (real) v[e] *= slope<ACT>(e & 1 ? bf16_hi(z[i][e >> 1]) : bf16_lo(z[i][e >> 1]));
                if (real && expert[i] == owner) acc[e] += v[e];
            }
            if (!dZ) continue;
            u16* dst = dZ + (u64)(r0 + 4 * i) * N;
            if constexpr (VEC) {
                if (col(0) < N)
                    *(u32x4*)(dst + col(0)) = u32x4{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]),
                                                    to_bf16x2(v[6], v[7])};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col(e) < N) dst[col(e)] = to_bf16(v[e]);
            }
        }
    }
    if (!partial) return;
    if constexpr (VEC) {
        *(f32x4*)&sums[wave][lane * 8] = f32x4{acc[0], acc[1], acc[2], acc[3]};
        *(f32x4*)&sums[wave][lane * 8 + 4] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[wave][col(e) - c0] = acc[e];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = (int)threadIdx.x + 256 * h;
        if (c0 + c < N) partial[(u64)blockIdx.x * N + c0 + c] = sums[0][c] + sums[1][c] + sums[2][c] + sums[3][c];
    }
}

// dbias[g][n]: the partial sums of the chunks that belong to expert g.  A workgroup
// takes 16 columns; its 16 waves of four 16-lane rows take 64 parts of the chunks, eight
// loads in flight, and the parts are added in a fixed order: the same sum on every run.
// (As 64 columns a workgroup in 16 parts 32768 x 512 had eight workgroups and took 22.8 us
// here; now 7.1.)
constexpr int kSumWaves = 16;
constexpr int kSumCols = 16;
constexpr int kSumParts = 64 * kSumWaves / kSumCols;
struct BiasSumArgs {
    const float* partial;
    const int* m_indices;
    float* dbias;
    int chunks, chunk, N;
};
__global__ void __launch_bounds__(64 * kSumWaves) dg_bias_sum_kernel(const BiasSumArgs a) {
    const float* __restrict__ partial = a.partial;
    const int* __restrict__ m_indices = a.m_indices;
    __shared__ float sums[kSumParts][kSumCols];
    const int tid = threadIdx.x, col = tid % kSumCols, part = tid / kSumCols;
    const int n = (int)blockIdx.x * kSumCols + col, g = blockIdx.y;
    const int each = (a.chunks + kSumParts - 1) / kSumParts;
    const int first = part * each, last = a.chunks - first < each ? a.chunks : first + each;
    float s = 0.f;
    for (int c = first; c < last; c += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool mine = c + i < last && (!m_indices || m_indices[(u64)(c + i) * a.chunk] == g);
            v[i] = mine && n < a.N ? partial[(u64)(c + i) * a.N + n] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i];
    }
    sums[part][col] = s;
    __syncthreads();
    if (tid >= 64) return;
    // four 16-lane rows a quarter of the parts each, then the quarters
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumParts / 4; ++w) t += sums[part * (kSumParts / 4) + w][col];
    t += __shfl_xor(t, 16);
    t += __shfl_xor(t, 32);
    if (part == 0 && n < a.N) a.dbias[(u64)g * a.N + n] = t;
}

// Rows a workgroup takes: as many as still give this many workgroups (at least 16), since
// each writes partial sums.  Measured with 16, 32, 64 and 128 rows, us: 1024 x 1024 7.7, 10.3,
// 15.6, 26.3; 8192 x 4096 51.6, 44.2, 48.0, 52.8; 65536 x 4096 392, 383, 370, 336.
constexpr int kBackwardGroups = 2048;

template <int ACT>
dg_status launch_backward(dim3 grid, void* stream, const BackwardArgs& a) {
    const bool stream_it = int64_t(6) * a.rows * a.N >= kStreamBytes;
    auto* kernel = a.N % 8 ? dg_epilogue_backward_kernel<ACT, false, false>
                 : stream_it ? dg_epilogue_backward_kernel<ACT, true, true> : dg_epilogue_backward_kernel<ACT, true, false>;
    return launch_rows("epilogue_backward", kernel, grid, 256, stream, a);
}

dg_status epilogue_backward(const void* dD, const void* Z, int act, const int32_t* m_indices, void* dZ, float* dbias,
                            int rows, int N, int G, void* stream) {
    if (rows != 0 && (!dD || (act != DG_ACT_NONE && !Z)))
        return set_error(DG_ERR_INVALID_ARG, "epilogue_backward: dD and (with an activation) Z must be non-NULL");
    if (act < DG_ACT_NONE || act > DG_ACT_GELU_TANH)
        return set_error(DG_ERR_INVALID_ARG, "epilogue_backward: unknown activation");
    if (rows < 0 || N <= 0 || G <= 0)
        return set_error(DG_ERR_INVALID_ARG, "epilogue_backward: sizes must be positive (M may be 0)");
    if (!aligned(dD, 16) || !aligned(Z, 16) || !aligned(dZ, 16) || !aligned(dbias, 4) || !aligned(m_indices, 4))
        return set_error(DG_ERR_ALIGNMENT, "epilogue_backward: dD, Z and dZ must be 16-byte, the rest 4-byte aligned");
    int chunk = 128;
    while (chunk > kStep && ((int64_t)rows + chunk - 1) / chunk * ((N + 511) / 512) < kBackwardGroups) chunk /= 2;
    const int chunks = (int)(((int64_t)rows + chunk - 1) / chunk);
    if (G > 65535 || N > 65535 * 512 || !fits_launch(chunks) || !fits_launch((N + kSumCols - 1) / kSumCols, 64 * kSumWaves))
        return set_error(DG_ERR_UNSUPPORTED, "epilogue_backward: too many rows, groups or columns for one launch");
    float* partial = nullptr;
    StreamScratch scratch;               // held until both kernels are launched
    if (dbias && chunks > 0) {
        dg_status s = stream_scratch(stream, (size_t)chunks * (size_t)N * sizeof(float), &scratch);
        if (s != DG_OK) return s;
        partial = static_cast<float*>(scratch.p);
    }
    if (chunks > 0 && (dZ || dbias)) {
        const dim3 grid(chunks, (N + 511) / 512);
        auto* f = act == DG_ACT_RELU ? launch_backward<DG_ACT_RELU> : act == DG_ACT_SILU ? launch_backward<DG_ACT_SILU>
                : act == DG_ACT_GELU ? launch_backward<DG_ACT_GELU>
                : act == DG_ACT_GELU_TANH ? launch_backward<DG_ACT_GELU_TANH> : launch_backward<DG_ACT_NONE>;
        dg_status s = f(grid, stream, BackwardArgs{static_cast<const u16*>(dD), static_cast<const u16*>(Z), m_indices,
                                                   static_cast<u16*>(dZ), partial, rows, N, G, chunk});
        if (s != DG_OK) return s;
    }
    if (!dbias) return DG_OK;
    return launch_rows("epilogue_backward (bias)", dg_bias_sum_kernel, dim3((N + kSumCols - 1) / kSumCols, G), 64 * kSumWaves, stream,
                       BiasSumArgs{partial, m_indices, dbias, chunks, chunk, N});
}

}  // namespace

dg_status transpose_bf16(const void* x, void* xt, int groups, int rows_k, int cols, int k_end, int64_t pitch,
                         void* stream) {
    const int k_blocks = k_end / 64;
    const uint64_t blocks = (uint64_t)k_blocks * (uint64_t)((cols + 63) / 64);
    if (!fits_launch((int64_t)blocks) || groups > 65535)
        return set_error(DG_ERR_UNSUPPORTED, "operand too large for the K-contiguous rewrite");
    if (blocks == 0) return DG_OK;
    return launch_rows("K-contiguous rewrite", dg_transpose_bf16_kernel, dim3((unsigned)blocks, 1, (unsigned)groups), 256, stream,
                       TransposeArgs{static_cast<const u16*>(x), static_cast<u16*>(xt), rows_k, cols, k_blocks, (long long)pitch});
}

dg_status pad_rows_bf16(const void* x, void* xp, int rows, int cols, int pitch, void* stream) {
    const u32 pieces = (u32)pitch / 8u;
    const u64 total = (u64)rows * pieces;
    if (total == 0) return DG_OK;
    const unsigned grid = (unsigned)std::min<u64>((total + 255) / 256, 1u << 16);
    return launch_rows("copy to whole K blocks", dg_pad_rows_bf16_kernel, dim3(grid), 256, stream,
                       PadArgs{static_cast<const u16*>(x), static_cast<u16*>(xp), (u32)cols, pieces, total});
}

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_epilogue_backward(const void* dD, const void* Z, int activation, void* dZ, float* dbias, int M, int N,
                               void* stream) {
    return guarded([&]() -> dg_status {
        return epilogue_backward(dD, Z, activation, nullptr, dZ, dbias, M, N, 1, stream);
    });
}

dg_status dg_m_grouped_epilogue_backward_contiguous(const void* dD, const void* Z, int activation,
                                                    const int32_t* m_indices, void* dZ, float* dbias, int M, int N,
                                                    int num_groups, void* stream) {
    return guarded([&]() -> dg_status {
        if (!m_indices && M != 0) return set_error(DG_ERR_INVALID_ARG, "m_indices must be non-NULL");
        if (M > 0 && M % dg_get_mk_alignment_for_contiguous_layout() != 0)
            return set_error(DG_ERR_ALIGNMENT, "contiguous M must be a multiple of the M alignment (128)");
        return epilogue_backward(dD, Z, activation, m_indices, dZ, dbias, M, N, num_groups, stream);
    });
}

}  // extern "C"
