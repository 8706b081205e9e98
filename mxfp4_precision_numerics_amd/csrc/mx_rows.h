// mx_rows.h -- rows of router logits shared by a few lanes: loads, reductions
// (their operations are the attention's too), softmax statistics (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

// ---------------------------------------------------------------------------
// Reductions over the L lanes (8, 16, 32 or 64) that share a row: exchanges
// with the neighbour, the other pair, the other quad and the other eight are
// DPP moves, the wider ones shuffles.  Every lane gets the result, in a fixed
// order.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

struct MaxF { __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); } };
struct AddF { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };

constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

template <int L, class T, class Op>
__device__ __forceinline__ T row_reduce(T v, Op op) {
    v = op(v, dpp<DPP_XOR1>(v));
    v = op(v, dpp<DPP_XOR2>(v));
    v = op(v, dpp<DPP_HALF_MIRROR>(v));       // the other quad of 8 lanes
    if constexpr (L >= 16) v = op(v, dpp<DPP_MIRROR>(v));   // the other half of 16
    if constexpr (L >= 32) v = op(v, __shfl_xor(v, 16));
    if constexpr (L >= 64) v = op(v, __shfl_xor(v, 32));
    return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    else return ((const float*)p)[i];
}

// A lane's experts of a row: C chunks of four, chunk c at 4 (lane + L c).
// Lanes past the row's end read its last experts again and take `past`: loads
// without branches are all under way at once.  vec: experts % 4 == 0 and
// aligned rows, a chunk is one load.
template <bool BF16, int L, int C>
__device__ __forceinline__ void load_row(const void* logits, int64_t base, int experts, int vec, int lane, float* v,
                                         float past = -__builtin_inff()) {
    if (vec) {
        if constexpr (BF16) {
            uint2 w[C];
#pragma unroll
            for (int c = 0; c < C; ++c)
                w[c] = *(const uint2*)((const uint16_t*)logits + base + min(4 * (lane + L * c), experts - 4));
#pragma unroll
            for (int c = 0; c < C; ++c) {
                v[4 * c + 0] = bf16lo(w[c].x);
                v[4 * c + 1] = bf16hi(w[c].x);
                v[4 * c + 2] = bf16lo(w[c].y);
                v[4 * c + 3] = bf16hi(w[c].y);
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float4 w = *(const float4*)((const float*)logits + base + min(4 * (lane + L * c), experts - 4));
                v[4 * c + 0] = w.x;
                v[4 * c + 1] = w.y;
                v[4 * c + 2] = w.z;
                v[4 * c + 3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * C; ++i)
            v[i] = load_logit<BF16>(logits, base + min(4 * (lane + L * (i >> 2)) + (i & 3), experts - 1));
    }
    if (experts < 4 * L * C) {
#pragma unroll
        for (int i = 0; i < 4 * C; ++i)
            v[i] = 4 * (lane + L * (i >> 2)) + (i & 3) < experts ? v[i] : past;
    }
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// e^x and 1 / (1 + e^-x) by the exponential and reciprocal instructions, for
// every expert of a row: e^x is off by |x| 2^-23 relative, which the sums and
// keys it goes into hold at a share of e^x itself.  Sigmoid keys, bias
// included, are good to 3e-7 absolute; softmax ones too but for their sum's
// rounding, which a row's keys share.  Sums are as good as with expf but for
// 5% (weights without renormalisation, 64 normal logits: median 4.0e-8 off,
// with expf 3.7e-8, for 20.4 us in place of 17.8 at 65536 x 256).  The weights
// of the chosen few use expf and a division.
__device__ __forceinline__ float quick_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float quick_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + quick_exp(-x));
}

// e^x, x <= 0, to the exponential instruction's own last place: what the
// product x log2(e) loses, r, comes back as the factor 2^r = 1 + r ln 2.
__device__ __forceinline__ float soft_exp(float x) {
    x = x < -150.0f ? -150.0f : x;            // (0 all the same, and no inf - inf below)
    const float t = x * 1.44269504f;
    const float r = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269504f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e * r, 0.693147181f, e);
}

// Row maximum and sum of exp(l - max) of a softmax; a row of -inf alone gives
// (0, 0), and its scores are 0.  KEEP: v becomes exp(l - max), accurately.
template <int L, int N, bool KEEP>
__device__ __forceinline__ void softmax_stats(float* v, float& top, float& sum) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = row_reduce<L>(m, MaxF());
    top = m == -__builtin_inff() ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float e = KEEP ? soft_exp(v[i] - top) : quick_exp(v[i] - top);
        if (KEEP) v[i] = e;
        s += e;
    }
    sum = row_reduce<L>(s, AddF());
}

}  // namespace mx
