// Activations kept for the backward pass in 8 bits (hipcc, gfx950): BF16 rows to
// E4M3 with one power-of-two scale per 1x128 block, back to BF16, and the fused
// epilogue's backward pass on pre-activations kept so.  The operations and their
// layouts are specified in include/dg.h.
//
//   scale 2^e, e the least with amax <= 448 2^e;  code = E4M3(x 2^-e);  kept value code 2^e
//
// Power-of-two scales: dividing by one is exact, so the one rounding is the code's, and a kept
// value has four significant bits, which BF16 holds, so that restoring rounds nothing.
// Every pass moves data, 16 lanes a block, 8 elements a lane, and is bound by HBM.
#include <climits>

#include "activation.h"
#include "row_kernels.h"

namespace dg {
namespace {

constexpr int kBlock = 128;
constexpr int kGroups = 16;            // of 16 lanes in a workgroup of 256
constexpr int kRounds = 4;             // blocks a group takes, their loads in flight together

// Eight codes from column c of a row of N; zeros past N.
__device__ __forceinline__ u64 load_codes(const u8* row, int c, int N) {
    u64 w = 0;
    if (c + 8 <= N) {
        __builtin_memcpy(&w, row + c, 8);
    } else if (c < N) {
#pragma unroll
        for (int i = 0; i < 7; ++i) w |= (u64)(c + i < N ? row[c + i] : (u8)0) << (8 * i);
    }
    return w;
}
__device__ __forceinline__ void store_codes(u8* row, int c, int N, u64 w) {
    if (c + 8 <= N) {
        __builtin_memcpy(row + c, &w, 8);
    } else if (c < N) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (c + i < N) row[c + i] = (u8)(w >> (8 * i));
    }
}
// 2^(byte - 127); byte 255 (a block that held an infinity or NaN) is NaN, byte 0 2^-127.
__device__ __forceinline__ float scale_of(u32 byte) {
    return __builtin_bit_cast(float, byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}
__device__ __forceinline__ void kept_values(u64 codes, float scale, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = (int)(u32)(codes >> (32 * h));
        v[4 * h] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * scale;
        v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * scale;
        v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * scale;
        v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * scale;
    }
}

// A workgroup takes kRounds * kGroups consecutive blocks (row-major), 16 lanes each.
// m_indices (or nullptr): rows with -1 are cleared, other negative rows are left alone.
struct KeepArgs {
    const u16* X;
    const int* m_indices;
    u8* codes;
    u8* scales;
    u32 blocks, row_blocks;
    int N;
};
__device__ __forceinline__ int row_index(const int* m_indices, u32 row) { return m_indices ? m_indices[row] : 0; }

__global__ void __launch_bounds__(256) dg_checkpoint_kernel(const KeepArgs a) {
    const int in = threadIdx.x & 15;
    u32 row[kRounds];
    int c[kRounds], index[kRounds];
    u32x4 w[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const u32 b = ((u32)blockIdx.x * kRounds + r) * kGroups + (threadIdx.x >> 4);
        row[r] = b / a.row_blocks;
        c[r] = (int)(b - row[r] * a.row_blocks) * kBlock + in * 8;
        index[r] = b < a.blocks ? row_index(a.m_indices, row[r]) : kPadding - 1;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        w[r] = u32x4{0u, 0u, 0u, 0u};
        if (index[r] >= 0) w[r] = load8(a.X + (u64)row[r] * (u64)a.N, c[r], a.N);
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        // the largest magnitude over the bit patterns: an infinity or NaN comes out on top
        u32 top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32 hi = w[r][i] >> 16 & 0x7fffu, lo = w[r][i] & 0x7fffu;
            top = hi > top ? hi : top;
            top = lo > top ? lo : top;
        }
        top = max16(top);
        // 448 = 1.75 2^8: the exponent less 8, one more where the mantissa (7 bits) is above 0.75
        u32 e = (top >> 7) + ((top & 0x7fu) > 0x60u ? 1u : 0u);
        e = top >= 0x7f80u ? 255u : top == 0u ? 127u : e > 9u ? e - 8u : 1u;
        if (index[r] < kPadding) continue;
        const float inverse = e == 255u ? __builtin_bit_cast(float, 0x7fc00000u) : __builtin_bit_cast(float, (254u - e) << 23);
        float v[8];
        unpack8(w[r], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inverse;
        // the largest scale: 256 times it, what magnitudes above 248 would round to, is past BF16
        if (e == 247u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -240.f), 240.f);
        }
        u32 code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
            code[h] = (u32)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], p, true);
        }
        store_codes(a.codes + (u64)row[r] * (u64)a.N, c[r], a.N, (u64)code[1] << 32 | code[0]);
        if (in == 0) a.scales[(u64)row[r] * a.row_blocks + (u32)c[r] / kBlock] = (u8)e;
    }
}

struct RestoreArgs {
    const u8* codes;
    const u8* scales;
    const int* m_indices;
    u16* X;
    u32 blocks, row_blocks;
    int N;
};
__global__ void __launch_bounds__(256) dg_checkpoint_restore_kernel(const RestoreArgs a) {
    const int in = threadIdx.x & 15;
    u32 row[kRounds], e[kRounds];
    int c[kRounds], index[kRounds];
    u64 w[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const u32 b = ((u32)blockIdx.x * kRounds + r) * kGroups + (threadIdx.x >> 4);
        row[r] = b / a.row_blocks;
        c[r] = (int)(b - row[r] * a.row_blocks) * kBlock + in * 8;
        index[r] = b < a.blocks ? row_index(a.m_indices, row[r]) : kPadding - 1;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        w[r] = 0;
        e[r] = 127u;
        if (index[r] >= 0) {
            w[r] = load_codes(a.codes + (u64)row[r] * (u64)a.N, c[r], a.N);
            e[r] = a.scales[(u64)row[r] * a.row_blocks + (u32)c[r] / kBlock];
        }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (index[r] < kPadding) continue;
        float v[8];
        kept_values(w[r], scale_of(e[r]), v);
        store8(a.X + (u64)row[r] * (u64)a.N, c[r], a.N, pack8(v));
    }
}

// ---------------------------------------------------------------- epilogue backward
// dZ = dD slope(z) and H = activation(z) with z the kept value, and the column sums of dZ (FP32, before its
// rounding) of the workgroup's rows: the split of dg_epilogue_backward, 512 columns of `chunk` rows a
// workgroup, 8 columns a lane, each wave every fourth row; two rows in flight (four: 61.0 us against 55.4 for 8192 x
// 4096, GELU, for want of registers; one 54.4 there, but 8192 x 1024 47 against 43 at 128 rows a workgroup).
// Rows a workgroup: as many as still give 1024 workgroups.  us with 16, 32 and 64: 2048 x 4096 18.2, 19.7, 26.6;
// 8192 x 4096 56.9, 55.4, 55.0, and in four experts, whose partial sums are read four times, 68.2, 63.3, 58.2.
constexpr int kWorkgroups = 1024;
constexpr int kWaveRows = 2;
constexpr int kStep = 4 * kWaveRows;
struct KeptBackwardArgs {
    const u16* dD;
    const u8* codes;
    const u8* scales;
    const int* m_indices;
    u16* dZ;
    u16* H;
    float* partial;
    int rows, N, G, chunk;
    u32 row_blocks;
};
template <int ACT>
__global__ void __launch_bounds__(256) dg_epilogue_backward_fp8_kernel(const KeptBackwardArgs a) {
    const int rows = a.rows, N = a.N, G = a.G;
    __shared__ __attribute__((aligned(16))) float sums[4][512];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = (int)blockIdx.y * 512, c = c0 + lane * 8;
    const int first = (int)blockIdx.x * a.chunk;
    const int last = rows - first < a.chunk ? rows : first + a.chunk;
    const u32 block = c < N ? (u32)c / kBlock : 0u;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    // the experts of the chunk's (at most 128) rows, two a lane: read row by row, their loads are waited for in front of
    // each turn's
    int index[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = first + lane + 64 * h;
        index[h] = a.m_indices && r < last ? a.m_indices[r] : 0;
    }
    const int owner = __builtin_amdgcn_readlane(index[0], 0);
    for (int r0 = first + wave; r0 < last; r0 += kStep) {
        // the expert of each of this wave's two rows (below 0: padding, or no row)
        int expert[kWaveRows];
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i) {
            const int in = r0 - first + 4 * i;
            const int of = __builtin_amdgcn_readlane(in < 64 ? index[0] : index[1], in & 63);
            expert[i] = r0 + 4 * i >= last ? kPadding - 1 : of;
        }
        u32x4 d[kWaveRows];
        u64 z[kWaveRows];
        u32 scale[kWaveRows];
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i) {
            d[i] = u32x4{0u, 0u, 0u, 0u};
            z[i] = 0;
            scale[i] = 127u;
            if ((u32)expert[i] < (u32)G) {
                const u64 row = (u64)(r0 + 4 * i);
                d[i] = load8(a.dD + row * (u64)N, c, N);
                z[i] = load_codes(a.codes + row * (u64)N, c, N);
                scale[i] = a.scales[row * a.row_blocks + block];
            }
        }
#pragma unroll
        for (int i = 0; i < kWaveRows; ++i) {
            const bool real = (u32)expert[i] < (u32)G;
            if (!real && expert[i] != kPadding) continue;
            float v[8], h[8];
            unpack8(d[i], v);
            kept_values(z[i], scale_of(scale[i]), h);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = slope<ACT>(h[e], h[e]);         // (0 of 0, so a padding row's H is cleared too)
                if (real) v[e] *= s;
                if (real && expert[i] == owner) acc[e] += v[e];
            }
            const u64 at = (u64)(r0 + 4 * i) * (u64)N;
            if (a.dZ) store8(a.dZ + at, c, N, pack8(v));
            if (a.H) store8(a.H + at, c, N, pack8(h));
        }
    }
    if (!a.partial) return;
    *(f32x4*)&sums[wave][lane * 8] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    *(f32x4*)&sums[wave][lane * 8 + 4] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = (int)threadIdx.x + 256 * h;
        if (c0 + n < N) a.partial[(u64)blockIdx.x * N + c0 + n] = sums[0][n] + sums[1][n] + sums[2][n] + sums[3][n];
    }
}

dg_status check_kept(const char* what, const void* x, const void* codes, const void* scales, const int32_t* m_indices,
                     int M, int N) {
    const std::string name(what);
    if (M < 0 || N <= 0) return set_error(DG_ERR_INVALID_ARG, name + ": sizes must be positive (M may be 0)");
    if (N > INT_MAX - 2 * kBlock) return set_error(DG_ERR_UNSUPPORTED, name + ": rows are too wide");
    if (M > 0 && (!x || !codes || !scales)) return set_error(DG_ERR_INVALID_ARG, name + ": NULL pointer");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(m_indices, 4))
        return set_error(DG_ERR_ALIGNMENT, name + ": rows and codes must be 16-byte, m_indices 4-byte aligned");
    return DG_OK;
}

// the grid that takes the blocks of M rows; 0: too many for one launch
unsigned block_grid(int M, int row_blocks) {
    const int64_t groups = ((int64_t)M * row_blocks + kRounds * kGroups - 1) / (kRounds * kGroups);
    return fits_launch(groups) ? (unsigned)groups : 0u;
}
int blocks_of(int N) { return N / kBlock + (N % kBlock != 0); }

dg_status backward(const void* dD, const void* codes, const void* scales, int act, const int32_t* m_indices, void* dZ,
                   void* H, float* dbias, int rows, int N, int G, void* stream) {
    dg_status s = check_kept("epilogue_backward_fp8", dD, codes, scales, m_indices, rows, N);
    if (s != DG_OK) return s;
    if (act < DG_ACT_NONE || act > DG_ACT_GELU_TANH)
        return set_error(DG_ERR_INVALID_ARG, "epilogue_backward_fp8: unknown activation");
    if (G <= 0) return set_error(DG_ERR_INVALID_ARG, "epilogue_backward_fp8: sizes must be positive (M may be 0)");
    if (H && (H == dZ || H == dD))
        return set_error(DG_ERR_INVALID_ARG, "epilogue_backward_fp8: H must be an array of its own");
    if (!aligned(dZ, 16) || !aligned(H, 16) || !aligned(dbias, 4))
        return set_error(DG_ERR_ALIGNMENT, "epilogue_backward_fp8: dZ and H must be 16-byte, dbias 4-byte aligned");
    const int chunk = backward_chunk(rows, N, kWorkgroups);
    const int chunks = (int)(((int64_t)rows + chunk - 1) / chunk);
    if (N > 65535 * 512 || !fits_launch(chunks) || !column_sums_fit(N, G))
        return set_error(DG_ERR_UNSUPPORTED, "epilogue_backward_fp8: too many rows, groups or columns for one launch");
    float* partial = nullptr;
    StreamScratch scratch;               // held until both kernels are launched
    if (dbias && chunks > 0) {
        s = stream_scratch(stream, (size_t)chunks * (size_t)N * sizeof(float), &scratch);
        if (s != DG_OK) return s;
        partial = static_cast<float*>(scratch.p);
    }
    if (chunks > 0 && (dZ || H || dbias)) {
        auto* kernel = act == DG_ACT_RELU ? dg_epilogue_backward_fp8_kernel<DG_ACT_RELU>
                     : act == DG_ACT_SILU ? dg_epilogue_backward_fp8_kernel<DG_ACT_SILU>
                     : act == DG_ACT_GELU ? dg_epilogue_backward_fp8_kernel<DG_ACT_GELU>
                     : act == DG_ACT_GELU_TANH ? dg_epilogue_backward_fp8_kernel<DG_ACT_GELU_TANH>
                                               : dg_epilogue_backward_fp8_kernel<DG_ACT_NONE>;
        s = launch_rows("epilogue_backward_fp8", kernel, dim3(chunks, (N + 511) / 512), 256, stream,
                        KeptBackwardArgs{static_cast<const u16*>(dD), static_cast<const u8*>(codes),
                                         static_cast<const u8*>(scales), m_indices, static_cast<u16*>(dZ),
                                         static_cast<u16*>(H), partial, rows, N, G, chunk, (u32)blocks_of(N)});
        if (s != DG_OK) return s;
    }
    if (!dbias) return DG_OK;
    return column_sums("epilogue_backward_fp8 (bias)", partial, m_indices, chunks, chunk, N, G, dbias, stream);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_checkpoint_fp8(const void* X, const int32_t* m_indices, void* codes, void* scales, int M, int N,
                            void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_kept("checkpoint_fp8", X, codes, scales, m_indices, M, N);
        if (s != DG_OK || M == 0) return s;
        const unsigned grid = block_grid(M, blocks_of(N));
        if (!grid) return set_error(DG_ERR_UNSUPPORTED, "checkpoint_fp8: too many rows for one launch");
        return launch_rows("checkpoint_fp8", dg_checkpoint_kernel, dim3(grid), 256, stream,
                           KeepArgs{static_cast<const u16*>(X), m_indices, static_cast<u8*>(codes), static_cast<u8*>(scales),
                                    (u32)M * (u32)blocks_of(N), (u32)blocks_of(N), N});
    });
}

dg_status dg_checkpoint_restore(const void* codes, const void* scales, const int32_t* m_indices, void* X, int M, int N,
                                void* stream) {
    return guarded([&]() -> dg_status {
        dg_status s = check_kept("checkpoint_restore", X, codes, scales, m_indices, M, N);
        if (s != DG_OK || M == 0) return s;
        const unsigned grid = block_grid(M, blocks_of(N));
        if (!grid) return set_error(DG_ERR_UNSUPPORTED, "checkpoint_restore: too many rows for one launch");
        return launch_rows("checkpoint_restore", dg_checkpoint_restore_kernel, dim3(grid), 256, stream,
                           RestoreArgs{static_cast<const u8*>(codes), static_cast<const u8*>(scales), m_indices,
                                       static_cast<u16*>(X), (u32)M * (u32)blocks_of(N), (u32)blocks_of(N), N});
    });
}

dg_status dg_epilogue_backward_fp8(const void* dD, const void* codes, const void* scales, int activation, void* dZ,
                                   void* H, float* dbias, int M, int N, void* stream) {
    return guarded([&]() -> dg_status {
        return backward(dD, codes, scales, activation, nullptr, dZ, H, dbias, M, N, 1, stream);
    });
}

dg_status dg_m_grouped_epilogue_backward_fp8_contiguous(const void* dD, const void* codes, const void* scales,
                                                        int activation, const int32_t* m_indices, void* dZ, void* H,
                                                        float* dbias, int M, int N, int num_groups, void* stream) {
    return guarded([&]() -> dg_status {
        if (!m_indices && M != 0) return set_error(DG_ERR_INVALID_ARG, "m_indices must be non-NULL");
        if (M > 0 && M % dg_get_mk_alignment_for_contiguous_layout() != 0)
            return set_error(DG_ERR_ALIGNMENT, "contiguous M must be a multiple of the M alignment (128)");
        return backward(dD, codes, scales, activation, m_indices, dZ, H, dbias, M, N, num_groups, stream);
    });
}

}  // extern "C"
