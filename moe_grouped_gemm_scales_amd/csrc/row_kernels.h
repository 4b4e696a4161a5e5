// What the kernels over BF16 rows share (moe.hip, linear.hip): conversions, and
// the launch of a kernel that takes one by-value struct.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "dg_internal.h"

namespace dg {
namespace {

typedef unsigned char u8;
typedef unsigned short u16;
typedef unsigned int u32;
typedef unsigned long long u64;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kPadding = -1;           // m_indices of a padding row inside a segment

__device__ __forceinline__ float bf16_lo(u32 w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(u32 w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
__device__ __forceinline__ u16 to_bf16(float f) { return __builtin_bit_cast(u16, (__bf16)f); }   // nearest-even
__device__ __forceinline__ u32 to_bf16x2(float lo, float hi) { return (u32)to_bf16(lo) | ((u32)to_bf16(hi) << 16); }

// Eight BF16 of a row whose width N is no multiple of 8, 64 apart from column c, two a word;
// zeros past N.  Past the end the last element is read instead and dropped, so that the
// eight loads are issued together: with a branch round each they were waited for one by one
// (epilogue backward, 300 x 515: 13.3 us against 8.5; combine of 86 x 5 rows of 1977: 7.8
// against 4.4).
__device__ __forceinline__ u32x4 load_spread(const u16* p, int c, int N) {
    u32 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[c + 64 * i < N ? c + 64 * i : N - 1];
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (c + 128 * i < N ? v[2 * i] : 0u) | (c + 128 * i + 64 < N ? v[2 * i + 1] << 16 : 0u);
    return w;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A launch has fewer than 2^32 work items along each axis: workgroups of 256 or 1024
// items that fit in one axis.
inline bool fits_launch(int64_t workgroups, int items = 256) { return workgroups * items < (int64_t(1) << 32); }

// Launches kernel(args).  The status is this launch's own: an error that an earlier call of the
// thread left behind, ours or another library's, is neither reported nor cleared.
template <typename Args>
dg_status launch_rows(const char* what, void (*kernel)(Args), dim3 grid, int items, void* stream, Args args) {
    void* argv[] = {&args};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(items), argv, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? DG_OK : set_error(DG_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

}  // namespace
}  // namespace dg
