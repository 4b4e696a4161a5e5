// Routing of tokens to experts (hipcc, gfx950): the topk experts of each token
// and their weights from a router's logits, and the gradient of the logits.  The
// operations are specified in include/dg.h.
//
//   score p = softmax(l) or 1 / (1 + e^-l),  choice value v = p + bias
//   topk of v (among the best groups), w = scale p / (sum of the chosen p, or 1)
//
// One wave a token: the logits are read once, coalesced, and a choice is a few
// cross-lane steps.  A token's logits are at most 4 KB, so the pass is bound by
// latency and by the wave's own instructions, not by HBM.
#include <cmath>
#include <type_traits>

#include "row_kernels.h"

namespace dg {
namespace {

constexpr int kMaxExperts = 1024;      // 16 a lane
constexpr int kMaxTopk = 64;           // a chosen expert a lane

struct RouteArgs {
    const void* logits;
    const float* bias;
    int* ids;
    float* weights;
    int T, E, k, groups, group_size, kept, best, renormalise;
    int whole_lanes;                   // lanes a group, where groups are a power of two of whole lanes; 0: not so
    float scale;
};

__device__ __forceinline__ float logit(const void* p, int wide, u64 at) {
    return wide ? static_cast<const float*>(p)[at] : bf16_lo(static_cast<const u16*>(p)[at]);
}

// Sums and maxima over the wave, the same in every lane: rotations within 16 lanes, then the four 16s.
// (By shuffles through LDS each of six steps waits for the one before: about 100 clocks a step.)
template <int D>
__device__ __forceinline__ double rotated(double v) {
    const u64 b = __builtin_bit_cast(u64, v);
    return __builtin_bit_cast(double, (u64)rotate16<D>((u32)(b >> 32)) << 32 | rotate16<D>((u32)b));
}
template <int D>
__device__ __forceinline__ float rotated(float v) {
    return __builtin_bit_cast(float, rotate16<D>(__builtin_bit_cast(u32, v)));
}
__device__ __forceinline__ double of_lane(double v, int lane) {
    const u64 b = __builtin_bit_cast(u64, v);
    return __builtin_bit_cast(double, (u64)(u32)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32 |
                                          (u32)__builtin_amdgcn_readlane((int)b, lane));
}
__device__ __forceinline__ float of_lane(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
    v += rotated<8>(v);
    v += rotated<4>(v);
    v += rotated<2>(v);
    v += rotated<1>(v);
    return (of_lane(v, 0) + of_lane(v, 16)) + (of_lane(v, 32) + of_lane(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, rotated<8>(v));
    v = fmaxf(v, rotated<4>(v));
    v = fmaxf(v, rotated<2>(v));
    v = fmaxf(v, rotated<1>(v));
    return fmaxf(fmaxf(of_lane(v, 0), of_lane(v, 16)), fmaxf(of_lane(v, 32), of_lane(v, 48)));
}
__device__ __forceinline__ u32 wave_max(u32 v) {
    v = max16(v);
    auto part = [&](int lane) { return (u32)__builtin_amdgcn_readlane((int)v, lane); };
    const u32 a = part(0), b = part(16), c = part(32), d = part(48);
    const u32 x = a > b ? a : b, y = c > d ? c : d;
    return x > y ? x : y;
}

// A choice value as an integer of the same order; 0: the expert is not available.  A NaN (of
// its logit, or of a softmax whose row holds one) ranks below every number.
__device__ __forceinline__ u64 rank_of(double v) {
    v = v == v ? v : -1e300;
    const u64 b = __builtin_bit_cast(u64, v);
    const u32 hi = (u32)(b >> 32), flip = (u32)((int)hi >> 31);         // negative: all bits, else the sign alone
    return (u64)(hi ^ (flip | 0x80000000u)) << 32 | ((u32)b ^ flip);
}
__device__ __forceinline__ double value_of(u64 r) {
    return __builtin_bit_cast(double, (r >> 63) ? r & ~(1ull << 63) : ~r);
}

template <int CTRL>
__device__ __forceinline__ u64 moved(u64 v) {
    const u32 hi = (u32)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, 0xf, 0xf, true);
    return (u64)hi << 32 | (u32)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// Whether lane's group g of L neighbouring lanes is among the a.kept best, from the two largest ranks of each lane's
// part: the sum of its best one or two values, of equals the lower group first.
__device__ __forceinline__ bool group_kept(const RouteArgs& a, u64 b1, u64 b2, int g, int L) {
    auto merge = [&](u64 o1, u64 o2) {
        const u64 lower = o1 < b1 ? o1 : b1, second = o2 > b2 ? o2 : b2;
        b1 = o1 > b1 ? o1 : b1;
        b2 = lower > second ? lower : second;
    };
    // neighbours, pairs, quads and eights: the other half's lanes all hold its two, so a mirror image will do
    if (L > 1) merge(moved<0xB1>(b1), moved<0xB1>(b2));
    if (L > 2) merge(moved<0x4E>(b1), moved<0x4E>(b2));
    if (L > 4) merge(moved<0x141>(b1), moved<0x141>(b2));
    if (L > 8) merge(moved<0x140>(b1), moved<0x140>(b2));
    for (int d = 16; d < L; d *= 2) merge(__shfl_xor(b1, d), __shfl_xor(b2, d));
    double worth = -INFINITY;
    if (b1) worth = value_of(b1) + (a.best > 1 && b2 ? value_of(b2) : 0.0);
    // lane s of a group compares with the groups s, s + L, ...
    int better = 0;
    const int sub = (int)(threadIdx.x & 63) % L;
    for (int h = sub; h < a.groups + sub; h += L) {            // (as many turns in every lane)
        const double o = __shfl(worth, h < a.groups ? h * L : 0);
        const u64 ahead = __ballot(h < a.groups && (o > worth || (o == worth && h < g)));
        better += __popcll(ahead >> (g * L) & ((1ull << L) - 1));
    }
    return better < a.kept;
}

// What a wave's lanes wrote to LDS is read by others of the same wave: in order, without a barrier.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// e^x for x <= 0 (a NaN stays one): x = n ln 2 + r, the Taylor series of e^r to r^13 (|r| <= 0.347: 4e-18 of it
// left), times 2^n.  Step by step for all N, so that a coefficient is one scalar operand for them; the device library's
// function, a branch round each, took 80 instructions a value with the quotient, this 30.
template <int N>
__device__ __forceinline__ void exp_of(double (&x)[N]) {
    constexpr double kFactorial[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                                       1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800};
    double n[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = x[i] < -800.0 ? -800.0 : x[i];                 // (0 from -746 on)
        n[i] = __builtin_rint(x[i] * 1.4426950408889634);
        // ln 2 in two parts, the first with zeros behind, so that n times it is exact
        x[i] = __builtin_fma(n[i], -0x1.62e42fefa38p-1, x[i]);
        x[i] = __builtin_fma(n[i], -0x1.ef35793c7673p-45, x[i]);
        y[i] = kFactorial[13];
    }
#pragma unroll
    for (int c = 12; c >= 0; --c) {
        double k = kFactorial[c];
        asm("" : "+s"(k));                                    // (a scalar pair, not moved to vector registers)
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __builtin_fma(y[i], x[i], k);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_amdgcn_ldexp(y[i], (int)n[i]);
}
// 1 / x for x from 1 to 2^10 (or NaN): the hardware's estimate (2^-22 or better) and two Newton steps
__device__ __forceinline__ double reciprocal(double x) {
    double r = __builtin_amdgcn_rcp(x);
    r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

// The lane's PER logits from expert e on; -inf past the last expert.
template <int PER, bool WIDE>
__device__ __forceinline__ void read_logits(const void* logits, u64 row, int e, int E, float (&l)[PER]) {
    const int at = e < E ? e : E - 1;
    if (E % PER == 0) {                           // whole pieces, of whatever alignment; lanes past the end read the last
        const u64 from = row + (u32)(e < E ? e : E - PER);
        if constexpr (WIDE) {
            __builtin_memcpy(l, static_cast<const float*>(logits) + from, 4 * PER);
        } else {
            u16 w[PER];
            __builtin_memcpy(w, static_cast<const u16*>(logits) + from, 2 * PER);
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = bf16_lo(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = logit(logits, WIDE, row + (u32)(at + i < E ? at + i : E - 1));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (e + i >= E) l[i] = -INFINITY;
}

// Tokens (waves) of a workgroup: the dispatch of 8192 workgroups of one wave takes 4 us by itself; the tokens of few
// are spread over the CUs.  (Past 256 experts four tokens' values do not fit beside other workgroups' in LDS.)
constexpr int waves_of(int per) { return per <= 4 ? 4 : 1; }
constexpr int kSpread = 1024;

// Lane i has experts i PER to i PER + PER - 1, so that the lowest lane among equals has the lowest expert.
// Choice values are 64-bit numbers: 256 scores of 8192 tokens hold pairs that FP32 scores
// tell apart wrongly, and a choice is not rounded but made.
template <int PER, bool WIDE, bool SIGMOID>
__global__ void __launch_bounds__(64 * waves_of(PER)) dg_moe_route_kernel(const RouteArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const u32 t = blockIdx.x * (blockDim.x >> 6) + (u32)wave;
    if (t >= (u32)a.T) return;
    const int E = a.E, e0 = lane * PER;
    __shared__ double scores[waves_of(PER)][PER * 64];
    __shared__ u64 ranks[waves_of(PER)][PER * 64];
    double* const score = scores[wave];
    float l[PER], bias[PER];
    double p[PER];
    u64 rank[PER];
    read_logits<PER, WIDE>(a.logits, (u64)t * (u32)E, e0, E, l);
    if (a.bias) {
        read_logits<PER, true>(a.bias, 0, e0, E, bias);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) bias[i] = 0.f;
    }
    if constexpr (SIGMOID) {
        // 1 / (1 + e^-|l|), times e^-|l| below zero
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] = -(double)__builtin_fabsf(l[i]);
        exp_of(p);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const double r = reciprocal(1.0 + p[i]);
            p[i] = l[i] < 0.f ? p[i] * r : r;
        }
    } else {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] = (double)l[i] - (double)top;
        exp_of(p);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (l[i] == -INFINITY) p[i] = 0.0;
            sum += p[i];
        }
        sum = reciprocal(wave_sum(sum));
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] *= sum;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const double v = p[i] + (double)bias[i];
        rank[i] = l[i] == -INFINITY || v == -INFINITY ? 0ull : rank_of(v);
        score[e0 + i] = p[i];
    }
    if (a.groups > 1 && !a.whole_lanes) {
        // groups that do not end with a lane: L lanes a group, through LDS
        u64* const shared_rank = ranks[wave];
#pragma unroll
        for (int i = 0; i < PER; ++i) shared_rank[e0 + i] = rank[i];
        wave_fence();
        int L = 64;
        while (L * a.groups > 64) L /= 2;
        const int g = lane / L, sub = lane % L;
        u64 b1 = 0, b2 = 0;
        if (g < a.groups)
            for (int j = sub; j < a.group_size; j += L) {
                const u64 r = shared_rank[g * a.group_size + j];
                b2 = r > b1 ? b1 : r > b2 ? r : b2;
                b1 = r > b1 ? r : b1;
            }
        if (!group_kept(a, b1, b2, g, L) && g < a.groups)
            for (int j = sub; j < a.group_size; j += L) shared_rank[g * a.group_size + j] = 0ull;
        wave_fence();
#pragma unroll
        for (int i = 0; i < PER; ++i) rank[i] = shared_rank[e0 + i];
    }
    // a lane's values largest first (of equals the lower expert), so that each turn below looks at the first alone; of
    // many values the sort costs more than looking at all
    constexpr bool SORTED = PER <= 4;
    int expert[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) expert[i] = e0 + i;
    if constexpr (SORTED) {
#pragma unroll
        for (int n = PER - 1; n > 0; --n)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool swap = rank[i + 1] > rank[i];
                const u64 r = swap ? rank[i] : rank[i + 1];
                const int e = swap ? expert[i] : expert[i + 1];
                rank[i] = swap ? rank[i + 1] : rank[i];
                expert[i] = swap ? expert[i + 1] : expert[i];
                rank[i + 1] = r;
                expert[i + 1] = e;
            }
    }
    if (a.whole_lanes) {
        // a.whole_lanes lanes a group, whose two best are already the first of each lane's
        u64 b1 = rank[0], b2 = 0;
        if constexpr (SORTED && PER > 1) {
            b2 = rank[1];
        } else {
#pragma unroll
            for (int i = 1; i < PER; ++i) {
                b2 = rank[i] > b1 ? b1 : rank[i] > b2 ? rank[i] : b2;
                b1 = rank[i] > b1 ? rank[i] : b1;
            }
        }
        if (!group_kept(a, b1, b2, lane / a.whole_lanes, a.whole_lanes)) {
#pragma unroll
            for (int i = 0; i < PER; ++i) rank[i] = 0ull;
        }
    }
    wave_fence();                                 // (the scores)
    // the best of the wave, k times: the largest upper word, then among its lanes the largest
    // lower word, then the lowest lane; the first step mostly leaves one lane
    int id = -1;                                  // of choice `lane`
    for (int j = 0; j < a.k; ++j) {
        u64 best = rank[0];
        int at = expert[0];
        if constexpr (!SORTED) {
#pragma unroll
            for (int i = 1; i < PER; ++i) {
                at = rank[i] > best ? expert[i] : at;
                best = rank[i] > best ? rank[i] : best;
            }
        }
        const u32 hi = wave_max((u32)(best >> 32));
        if (hi == 0u) break;                      // none is available
        bool mine = (u32)(best >> 32) == hi;
        u64 with = __ballot(mine);
        if (with & (with - 1)) {
            const u32 lo = wave_max(mine ? (u32)best : 0u);
            with = __ballot(mine && (u32)best == lo);
        }
        const int winner = __builtin_ctzll(with);
        const int chosen = __builtin_amdgcn_readlane(at, winner);
        if (lane == j) id = chosen;
        if constexpr (SORTED) {
            const bool won = lane == winner;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                rank[i] = won ? (i + 1 < PER ? rank[i + 1 < PER ? i + 1 : i] : 0ull) : rank[i];
                if (i + 1 < PER) expert[i] = won ? expert[i + 1] : expert[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (expert[i] == chosen) rank[i] = 0ull;
        }
    }
    double w = id >= 0 ? score[id] : 0.0;
    if (a.renormalise) {
        const double sum = wave_sum(w);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (lane < a.k) {
        a.ids[(u64)t * (u32)a.k + lane] = id;
        a.weights[(u64)t * (u32)a.k + lane] = (float)((double)a.scale * w);
    }
}

// Gradient: from that of the weights, dp of the chosen experts, then through the scores' function.
//   sigmoid: dl = dp p (1 - p);  softmax: dl_e = p_e (dp_e - sum_j dp_j p_j)
//   dp_j = scale dw_j, or renormalised, with r_j = p_j / P, P the sum of the chosen p: dp_j p_j = scale r_j
//   (dw_j - sum_i dw_i r_i), which add up to zero, so that a softmax's other experts get nothing
// An expert that ids names twice gets both terms, in j order.
struct RouteBackwardArgs {
    const void* logits;
    const int* ids;
    const float* d_weights;
    void* d_logits;
    int T, E, k;
    float scale;
};
template <int PER, bool WIDE, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(256) dg_moe_route_backward_kernel(const RouteBackwardArgs a) {
    const int lane = threadIdx.x & 63;
    const u32 t = blockIdx.x * (blockDim.x >> 6) + (u32)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= (u32)a.T) return;
    const int E = a.E;
    const u64 row = (u64)t * (u32)E;
    // (lanes past the last choice read it, so that the loads are issued together)
    const u64 mine = (u64)t * (u32)a.k + (u32)(lane < a.k ? lane : a.k - 1);
    int id = a.ids[mine];
    const float given = a.d_weights[mine];
    if (lane >= a.k || (u32)id >= (u32)E) id = -1;
    const float dw = id >= 0 ? a.scale * given : 0.f;
    const float lj = id >= 0 ? logit(a.logits, WIDE, row + (u32)id) : -INFINITY;
    float p[PER];                              // softmax without renormalising: of every expert
    float c;                                   // choice `lane`'s term
    float every = 0.f;                         // ... and what every expert has subtracted, times its p
    if constexpr (SIGMOID) {
        // p = e^min(l,0) / (1 + e^-|l|), 1 - p that of -l; the ratios p_j / P from powers relative to the
        // largest, which do not all vanish where every chosen logit is far below zero
        const float small = 1.f / (1.f + expf(-fabsf(lj))), rest = (lj > 0.f ? expf(-lj) : 1.f) * small;
        if constexpr (RENORM) {
            const float top = fminf(wave_max(lj), 0.f);
            const float s = lj == -INFINITY ? 0.f : expf(fminf(lj, 0.f) - top) * small;
            const float P = wave_sum(s);
            const float r = P > 0.f ? s / P : P != P ? P : 0.f;
            c = r * rest * (dw - wave_sum(dw * r));
        } else {
            c = dw * (lj > 0.f ? 1.f : expf(lj)) * small * rest;
        }
    } else if constexpr (RENORM) {
        const float top = wave_max(lj);
        const float s = lj == -INFINITY ? 0.f : expf(lj - top);
        const float P = wave_sum(s);
        const float r = P > 0.f ? s / P : P != P ? P : 0.f;
        c = r * (dw - wave_sum(dw * r));
    } else {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] = logit(a.logits, WIDE, row + (u32)(lane + 64 * i < E ? lane + 64 * i : E - 1));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (lane + 64 * i >= E) p[i] = -INFINITY;
            top = fmaxf(top, p[i]);
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            p[i] = p[i] == -INFINITY ? 0.f : expf(p[i] - top);
            sum += p[i];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) p[i] *= inv;
        c = dw;
        every = wave_sum(lj == -INFINITY ? 0.f : dw * (expf(lj - top) * inv));
    }
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) out[i] = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(id, j);
        const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, c), j));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == lane + 64 * i) out[i] += v;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        if constexpr (!SIGMOID && !RENORM) out[i] = p[i] * (out[i] - every);
        if (e >= E) continue;
        if constexpr (WIDE) static_cast<float*>(a.d_logits)[row + e] = out[i];
        else static_cast<u16*>(a.d_logits)[row + e] = to_bf16(out[i]);
    }
}

template <int PER>
dg_status launch_route(bool wide, bool sigmoid, unsigned T, void* stream, const RouteArgs& a) {
    auto* kernel = wide ? (sigmoid ? dg_moe_route_kernel<PER, true, true> : dg_moe_route_kernel<PER, true, false>)
                        : (sigmoid ? dg_moe_route_kernel<PER, false, true> : dg_moe_route_kernel<PER, false, false>);
    const unsigned waves = T >= kSpread ? waves_of(PER) : 1;
    return launch_rows("moe_route", kernel, dim3((T + waves - 1) / waves), 64 * waves, stream, a);
}
template <int PER, bool WIDE>
dg_status launch_route_backward(bool sigmoid, bool renorm, unsigned T, void* stream, const RouteBackwardArgs& a) {
    auto* kernel = sigmoid ? (renorm ? dg_moe_route_backward_kernel<PER, WIDE, true, true>
                                     : dg_moe_route_backward_kernel<PER, WIDE, true, false>)
                           : (renorm ? dg_moe_route_backward_kernel<PER, WIDE, false, true>
                                     : dg_moe_route_backward_kernel<PER, WIDE, false, false>);
    const unsigned waves = T >= kSpread ? 4 : 1;
    return launch_rows("moe_route_backward", kernel, dim3((T + waves - 1) / waves), 64 * waves, stream, a);
}

dg_status check_route(const char* what, bool null, const dg_routing* r, int logits_type, int T, int E, int k) {
    const std::string name(what);
    if (!r || null) return set_error(DG_ERR_INVALID_ARG, name + ": NULL pointer");
    if (T < 0 || E <= 0 || k <= 0)
        return set_error(DG_ERR_INVALID_ARG, name + ": sizes must be positive (T may be 0)");
    if (logits_type != DG_TYPE_F32 && logits_type != DG_TYPE_BF16)
        return set_error(DG_ERR_INVALID_ARG, name + ": unknown type of the logits");
    if (r->score != DG_SCORE_SOFTMAX && r->score != DG_SCORE_SIGMOID)
        return set_error(DG_ERR_INVALID_ARG, name + ": unknown score");
    if (E > kMaxExperts) return set_error(DG_ERR_UNSUPPORTED, name + ": at most 1024 experts");
    if (k > E) return set_error(DG_ERR_INVALID_ARG, name + ": topk is larger than the number of experts");
    if (k > kMaxTopk) return set_error(DG_ERR_UNSUPPORTED, name + ": topk is at most 64");
    if (!fits_launch(T, 64)) return set_error(DG_ERR_UNSUPPORTED, name + ": too many tokens for one launch");
    return DG_OK;
}

// experts a lane
int per_lane(int E) {
    int per = 1;
    while (per * 64 < E) per *= 2;
    return per;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_moe_route(const void* logits, int logits_type, const float* bias, const dg_routing* routing,
                       int32_t* expert_ids, float* weights, int T, int num_experts, int topk, void* stream) {
    return guarded([&]() -> dg_status {
        const bool null = T > 0 && (!logits || !expert_ids || !weights);
        dg_status s = check_route("moe_route", null, routing, logits_type, T, num_experts, topk);
        if (s != DG_OK) return s;
        const dg_routing r = *routing;
        if (r.groups <= 0 || num_experts % r.groups || r.topk_groups <= 0 || r.topk_groups > r.groups)
            return set_error(DG_ERR_INVALID_ARG, "moe_route: groups must divide the experts, topk_groups be 1 to groups");
        if (r.groups > 64) return set_error(DG_ERR_UNSUPPORTED, "moe_route: at most 64 groups");
        if (r.group_best != 1 && r.group_best != 2)
            return set_error(DG_ERR_INVALID_ARG, "moe_route: group_best must be 1 or 2");
        const int size = num_experts / r.groups;
        if (topk > r.topk_groups * size)
            return set_error(DG_ERR_INVALID_ARG, "moe_route: topk is larger than the experts of topk_groups groups");
        const bool wide = logits_type == DG_TYPE_F32;
        if (!aligned(logits, wide ? 4 : 2) || !aligned(bias, 4) || !aligned(expert_ids, 4) || !aligned(weights, 4))
            return set_error(DG_ERR_ALIGNMENT, "moe_route: arrays must be aligned to their elements");
        if (T == 0) return DG_OK;
        const int groups = r.topk_groups < r.groups ? r.groups : 1, per = per_lane(num_experts), lanes = size / per;
        const bool whole = groups > 1 && size % per == 0 && (lanes & (lanes - 1)) == 0;
        const RouteArgs a{logits, bias, expert_ids, weights, T, num_experts, topk, groups, size, r.topk_groups,
                          r.group_best, r.renormalise != 0, whole ? lanes : 0, r.scale};
        const bool sigmoid = r.score == DG_SCORE_SIGMOID;
        switch (per) {
            case 1: return launch_route<1>(wide, sigmoid, (unsigned)T, stream, a);
            case 2: return launch_route<2>(wide, sigmoid, (unsigned)T, stream, a);
            case 4: return launch_route<4>(wide, sigmoid, (unsigned)T, stream, a);
            case 8: return launch_route<8>(wide, sigmoid, (unsigned)T, stream, a);
            default: return launch_route<16>(wide, sigmoid, (unsigned)T, stream, a);
        }
    });
}

dg_status dg_moe_route_backward(const void* logits, int logits_type, const int32_t* expert_ids, const float* d_weights,
                                const dg_routing* routing, void* d_logits, int T, int num_experts, int topk,
                                void* stream) {
    return guarded([&]() -> dg_status {
        const bool null = T > 0 && (!logits || !expert_ids || !d_weights || !d_logits);
        dg_status s = check_route("moe_route_backward", null, routing, logits_type, T, num_experts, topk);
        if (s != DG_OK) return s;
        const bool wide = logits_type == DG_TYPE_F32;
        if (!aligned(logits, wide ? 4 : 2) || !aligned(d_logits, wide ? 4 : 2) || !aligned(expert_ids, 4) ||
            !aligned(d_weights, 4))
            return set_error(DG_ERR_ALIGNMENT, "moe_route_backward: arrays must be aligned to their elements");
        if (T == 0) return DG_OK;
        const RouteBackwardArgs a{logits, expert_ids, d_weights, d_logits, T, num_experts, topk, routing->scale};
        const bool sigmoid = routing->score == DG_SCORE_SIGMOID, renorm = routing->renormalise != 0;
        auto launch = [&](auto per) {
            constexpr int PER = decltype(per)::value;
            return wide ? launch_route_backward<PER, true>(sigmoid, renorm, (unsigned)T, stream, a)
                        : launch_route_backward<PER, false>(sigmoid, renorm, (unsigned)T, stream, a);
        };
        switch (per_lane(num_experts)) {
            case 1: return launch(std::integral_constant<int, 1>{});
            case 2: return launch(std::integral_constant<int, 2>{});
            case 4: return launch(std::integral_constant<int, 4>{});
            case 8: return launch(std::integral_constant<int, 8>{});
            default: return launch(std::integral_constant<int, 16>{});
        }
    });
}

}  // extern "C"
