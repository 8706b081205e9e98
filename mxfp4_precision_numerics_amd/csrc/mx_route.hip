// mx_route.hip -- routing tokens to experts: scores, selection, weights, their
// gradient, and the dispatch plan the grouped kernels read (gfx950).
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_device.h"
#include "mx_host.h"

namespace {

using namespace mx;

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_TOP_K = 32;
constexpr int MAX_GROUPS = 64;

struct RouteArgs {
    const void* logits;
    int64_t tokens, ld;       // row pitch in elements
    int experts;
    const float* bias;        // or null
    int score;                // MX_SOFTMAX, MX_SIGMOID
    int groups, top_groups, group_best;
    int group_size, share_log2;   // experts of a group; lanes that scan one together
    float group_inv;              // 1 / group_size
    int row_floats, score_at;     // LDS of a row, and where its groups' scores begin
    int top_k, renorm;
    float scale;
    int vec, vec_bias;        // rows, the bias can be read four experts at a time
    int32_t* ids;
    float* weights;
};

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

// ---------------------------------------------------------------------------
// Keys.  The bits of an fp32 key, flipped so that they grow with it as an
// unsigned number, are the leading mantissa and exponent bits of a double
// whose exponent's top bits are fixed (a positive normal number whatever the
// key), and 1023 - e, e the expert's index, its lowest ten bits.  So a larger
// double is a larger key, or of equal keys the lower index; all keys of a row
// are distinct, and keeping the larger or the smaller of two, index and all,
// is one v_max_f64 or v_min_f64, which this GPU issues as fast as the fp32
// ones.  A pair of an fp32 key and an index would take a comparison and two
// selects for each.
// Unsigned key 0 is an expert that cannot be chosen; NaN takes the place of
// -inf, behind every number.
// ---------------------------------------------------------------------------
struct MaxD {
    // (fmax() would quiet its operands first; these are never NaN)
    __device__ __forceinline__ double operator()(double a, double b) const {
        double r;
        asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
};
struct MinD {
    __device__ __forceinline__ double operator()(double a, double b) const {
        double r;
        asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
};

__device__ __forceinline__ double make_key(uint32_t u, int e) {
    const uint32_t hi = __builtin_amdgcn_alignbit(1u, u, 3);       // 001 and the upper 29 bits
    const uint32_t lo = (u << 29) | (uint32_t)((MAX_EXPERTS - 1) ^ e);
    return __hiloint2double((int)hi, (int)lo);
}
// The key is the result of an addition: not -0, which would sort below 0, and
// no signalling NaN, so the plain instruction turns NaN into -inf.
__device__ __forceinline__ double pack_key(float key, int e) {
    uint32_t b;
    asm("v_max_f32 %0, %1, %2" : "=v"(b) : "s"(0xFF800000u), "v"(key));
    const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return make_key(key == -__builtin_inff() ? 0u : u, e);
}
__device__ __forceinline__ bool key_there(double d) {
    return __builtin_amdgcn_alignbit((uint32_t)__double2hiint(d), (uint32_t)__double2loint(d), 29) != 0;
}
__device__ __forceinline__ int key_index(double d) {
    return MAX_EXPERTS - 1 - (__double2loint(d) & (MAX_EXPERTS - 1));
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

// The chosen experts' part in their sum, renormalised: lane j holds chosen
// expert j (there = it exists).  Softmax: p is the softmax over the chosen
// logits.  Sigmoid: p = s / sum s; below -40 the scores are e^l to 24 bits, so
// when the largest chosen logit is that low they are all scaled by its
// e^-l, and scores that would underflow keep their proportions.
// Every lane of the row calls it.
template <int L>
__device__ __forceinline__ float renormalised(float l, bool there, bool softmax, float& s) {
    const float ninf = -__builtin_inff();
    float top = row_reduce<L>(there ? l : ninf, MaxF());
    top = top == ninf ? 0.0f : top;
    s = softmax ? 0.0f : sigmoid(l);
    const float part = !there ? 0.0f : softmax || top < -40.0f ? expf(l - top) : s;
    const float sum = row_reduce<L>(part, AddF());
    return there ? part / sum : 0.0f;
}

// ---------------------------------------------------------------------------
// Group scores and the mask of the groups that stay (bit g).  The lanes of a
// row put their keys into LDS, or where groups are whole chunks of four
// experts (QUADS) only the two best of each chunk.  Each group has four spare
// words behind it, so that lanes scanning neighbouring groups meet different
// banks; 2^n lanes share the scan of a group, as many as there are.  A group's
// place is the number of groups before it.  Rows lie within a wave, so its own
// order is enough.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The two best of (b1 >= b2) and x: the median of the three is the new second.
// A NaN x (a quiet one: keys are results of additions) changes neither: the
// instruction gives the least of the three but NaN.  The builtin will not do:
// with a constant -inf as b2 the compiler makes it the minimum of b1 and x,
// which is b1 for a NaN.
__device__ __forceinline__ void best_two(float& b1, float& b2, float x) {
    float second;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(second) : "v"(b1), "v"(b2), "v"(x));
    b2 = second;
    b1 = fmaxf(b1, x);
}

__device__ __forceinline__ int group_of(int e, float inv) { return (int)(((float)e + 0.5f) * inv); }

template <int L, int C, bool QUADS>
__device__ __forceinline__ void drop_groups(const RouteArgs& a, float* keys, int lane, float* v) {
    const float none = -__builtin_inff(), inv = a.group_inv;
    const int size = a.group_size, share = 1 << a.share_log2;
    float* score = keys + a.score_at;
    int own[C];                                            // QUADS: the group of each chunk
    if constexpr (QUADS) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = 4 * (lane + L * c);
            own[c] = group_of(e, inv);
            float b1 = none, b2 = none;
#pragma unroll
            for (int i = 0; i < 4; ++i) best_two(b1, b2, v[4 * c + i]);
            if (e < a.experts) *(float2*)(keys + e / 2 + 4 * own[c]) = make_float2(b1, b2);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) {
            const int e = 4 * (lane + L * (i >> 2)) + (i & 3);
            if (e < a.experts) keys[e + 4 * group_of(e, inv)] = v[i];
        }
    }
    wave_fence();
    for (int at = lane; at < a.groups * share; at += L) {
        const int g = at >> a.share_log2, part = at & (share - 1);
        float b1 = none, b2 = none;
        if constexpr (QUADS) {
            const float* of = keys + g * (size / 2 + 4);
            for (int i = 2 * part; i < size / 2; i += 2 * share) {
                const float2 x = *(const float2*)(of + i);
                best_two(b1, b2, x.x);
                b2 = fmaxf(b2, x.y);
            }
        } else {
            const float* of = keys + g * (size + 4);
            for (int i = part; i < size; i += share) best_two(b1, b2, of[i]);
        }
        // (a group's lanes run the loop over `at` together)
        for (int o = 1; o < share; o *= 2) {
            const float p1 = __shfl_xor(b1, o), p2 = __shfl_xor(b2, o);
            best_two(b1, b2, p1);
            b2 = fmaxf(b2, p2);
        }
        // a sum of two lowest values stays above the score of an empty group
        if (part == 0) score[g] = a.group_best > 1 && b2 != none ? fmaxf(b1 + b2, -FLT_MAX) : b1;
    }
    wave_fence();
    uint64_t kept = 0;
    const int shift = (threadIdx.x & 63) & ~(L - 1);
    for (int g0 = 0; g0 < a.groups; g0 += L) {
        const int g = g0 + lane;
        const float mine = score[min(g, a.groups - 1)];
        int before = 0;
        for (int h = 0; h < a.groups; h += 4) {            // (the scores' end is filled up to a float4)
            const float4 s = *(const float4*)(score + h);
            const float q[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                before += h + i < a.groups && (h + i < g ? q[i] >= mine : q[i] > mine);
        }
        uint64_t m = __ballot(g < a.groups && before < a.top_groups) >> shift;
        if constexpr (L < 64) m &= (1ull << L) - 1;
        kept |= m << g0;
    }
    const bool wide = a.groups > 32;
    const uint32_t low = (uint32_t)kept, high = (uint32_t)(kept >> 32);
    auto stays = [&](int g) { return ((wide && g >= 32 ? high : low) >> (g & 31)) & 1; };
    if constexpr (QUADS) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool yes = stays(own[c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * c + i] = yes ? v[4 * c + i] : none;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * C; ++i)
            v[i] = stays(group_of(4 * (lane + L * (i >> 2)) + (i & 3), inv)) ? v[i] : none;
    }
}

// ---------------------------------------------------------------------------
// The K largest keys of a row in order, K a power of two: every lane sorts its
// own, then log2(L) times a lane and its partner keep the larger half of both
// lists.  Of two descending lists a and b the K largest are max(a_i, b_K-1-i),
// a bitonic list, which log2(K) rounds of exchanges put in order.  There are
// no branches and no serial chain of K row maxima.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void exchange(double& a, double& b) {
    const double x = MaxD()(a, b);
    b = MinD()(a, b);
    a = x;
}
template <int K>
__device__ __forceinline__ void bitonic_merge(double* v) {
#pragma unroll
    for (int h = K / 2; h; h /= 2)
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (!(i & h)) exchange(v[i], v[i + h]);
}
// Descending order of K values by odd-even merges.
template <int K>
__device__ __forceinline__ void sort_down(double* v) {
#pragma unroll
    for (int p = 1; p < K; p *= 2)
#pragma unroll
        for (int q = p; q; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < K; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < K && (i + j) / (2 * p) == (i + j + q) / (2 * p)) exchange(v[i + j], v[i + j + q]);
}
template <int K, class From>
__device__ __forceinline__ void keep_larger(double* v, From from) {
    double o[K];
#pragma unroll
    for (int i = 0; i < K; ++i) o[i] = from(v[K - 1 - i]);
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = MaxD()(v[i], o[i]);
    bitonic_merge<K>(v);
}
template <int K, int L, int N>
__device__ __forceinline__ void row_largest(double* key, double* list) {
    const double none = make_key(0u, MAX_EXPERTS - 1);     // below every key there is
#pragma unroll
    for (int i = 0; i < K; ++i) list[i] = i < N ? key[i] : none;
    sort_down<(N < K ? N : K)>(list);
#pragma unroll
    for (int at = K; at < N; at += K) {
        sort_down<K>(key + at);
#pragma unroll
        for (int i = 0; i < K; ++i) list[i] = MaxD()(list[i], key[at + K - 1 - i]);
        bitonic_merge<K>(list);
    }
    keep_larger<K>(list, [](double d) { return dpp<DPP_XOR1>(d); });
    keep_larger<K>(list, [](double d) { return dpp<DPP_XOR2>(d); });
    keep_larger<K>(list, [](double d) { return dpp<DPP_HALF_MIRROR>(d); });
    if constexpr (L >= 16) keep_larger<K>(list, [](double d) { return dpp<DPP_MIRROR>(d); });
    if constexpr (L >= 32) keep_larger<K>(list, [](double d) { return __shfl_xor(d, 16); });
    if constexpr (L >= 64) keep_larger<K>(list, [](double d) { return __shfl_xor(d, 32); });
}

// Bound by the vector units: for 256 experts in groups 196 instructions a row,
// of which the keys' sort is a third.  65536 tokens, top 8 of 256 fp32 in 8
// groups: 29 us (2.3 TB/s read; 22 us of it the instructions alone); without
// bias and groups 17 us (4.1 TB/s).  16384 tokens, top 4 of 32: 3.5 us.
// K = 8: up to eight experts by the merged lists; K = 0: any number, one row
// maximum after the other (top 16 of 256 there 41 us, top 32 148).
template <bool BF16, int L, int C, int K>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    constexpr int N = 4 * C, ROWS = 256 / L;
    extern __shared__ float4 smem[];
    const int lane = threadIdx.x & (L - 1), r = threadIdx.x / L;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS + r;
    const bool live = row0 < a.tokens;
    const int64_t row = live ? row0 : a.tokens - 1;
    const int64_t base = row * a.ld;
    const bool softmax = a.score == MX_SOFTMAX;
    float v[N];
    load_row<BF16, L, C>(a.logits, base, a.experts, a.vec, lane, v);

    const bool by_score = a.bias || (a.groups > 1 && a.group_best > 1);
    float top = 0.0f, sum = 1.0f;
    if (softmax && (by_score || !a.renorm)) softmax_stats<L, N, false>(v, top, sum);
    if (by_score) {
        const float inv = 1.0f / sum;
        float b[N];
        if (a.bias) {
            load_row<false, L, C>(a.bias, 0, a.experts, a.vec_bias, lane, b, 0.0f);
            // A bias of -inf takes its expert away also where the score is NaN,
            // which the sum does not do.  In bits -inf is above every number,
            // so one maximum of all of them shows whether there is one to look
            // for (a comparison at every expert: 44.1 us against 43.7 for
            // both directions of the grouped size above).
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) most = max(most, __float_as_uint(b[i]));
            if (__any(most >= 0xFF800000u)) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = b[i] == -__builtin_inff() ? b[i] : v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) b[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = softmax ? quick_exp(v[i] - top) * inv : quick_sigmoid(v[i]);
            v[i] = v[i] == -__builtin_inff() ? v[i] : s + b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += 0.0f;          // -0 counts as 0
    }
    if (a.groups > 1) {
        float* keys = (float*)smem + r * a.row_floats;
        if (a.group_size % 4 == 0) drop_groups<L, C, true>(a, keys, lane, v);
        else drop_groups<L, C, false>(a, keys, lane, v);
    }

    double key[N], mine = make_key(0u, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = pack_key(v[i], 4 * (lane + L * (i >> 2)) + (i & 3));
    if constexpr (K > 0) {
        double list[K];
        row_largest<K, L, N>(key, list);
#pragma unroll
        for (int j = 0; j < K; ++j) mine = lane == j ? list[j] : mine;
    } else {
        const double none = mine;
        for (int j = 0; j < a.top_k; ++j) {
            double m = key[0];
#pragma unroll
            for (int i = 1; i < N; ++i) m = MaxD()(m, key[i]);
            m = row_reduce<L>(m, MaxD());
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = key[i] == m ? none : key[i];
            mine = lane == j ? m : mine;
        }
    }

    const bool there = lane < a.top_k && key_there(mine);
    const int id = there ? key_index(mine) : -1;
    const float l = there ? load_logit<BF16>(a.logits, base + id) : 0.0f;
    float w;
    if (a.renorm) {
        float s;
        w = renormalised<L>(l, there, softmax, s);
    } else {
        w = !there ? 0.0f : softmax ? expf(l - top) / sum : sigmoid(l);
    }
    if (live && lane < a.top_k) {
        a.ids[row * a.top_k + lane] = id;
        a.weights[row * a.top_k + lane] = a.scale * w;
    }
}

// ---------------------------------------------------------------------------
// Gradient of the weights with respect to the logits (the choice is held
// fixed).  With ds_j = scale dw_j at the chosen experts:
//   softmax          dl_e = s_e (ds_e - sum_j ds_j s_j)        (every expert)
//   softmax, renorm  dl_j = p_j (ds_j - sum_m ds_m p_m)
//   sigmoid          dl_j = ds_j s_j (1 - s_j)
//   sigmoid, renorm  dl_j = p_j (1 - s_j)(ds_j - sum_m ds_m p_m)
// Only the first reads a whole row of logits.  The dense row is put together
// in LDS and written once, with non-temporal stores: no dirty lines are left
// for the kernel's end (both directions of 65536 x 256: 48.0 us without, 44.1
// with them; of 16384 x 256: 12.9 and 10.3).  Bound by memory: the write, and
// the lines that the chosen logits lie in.  65536 tokens, top 8 of 256 fp32:
// 15 us; the dense one 24 us (5.9 TB/s).
// ---------------------------------------------------------------------------
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

struct RouteBwdArgs {
    const void* logits;
    int64_t tokens, ld;
    int experts, score, top_k, renorm;
    float scale;
    int vec, vec_out;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int64_t dld;
};

template <bool BF16, int L, int C>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
    constexpr int N = 4 * C, ROWS = 256 / L;
    __shared__ float4 rows_of[ROWS][L * C];
    const int lane = threadIdx.x & (L - 1), r = threadIdx.x / L;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS + r;
    const bool live = row0 < a.tokens;
    const int64_t row = live ? row0 : a.tokens - 1;
    const int64_t base = row * a.ld;
    const bool softmax = a.score == MX_SOFTMAX, dense = softmax && !a.renorm;
    float v[N];
    float top = 0.0f, sum = 1.0f;
    if (dense) {
        load_row<BF16, L, C>(a.logits, base, a.experts, a.vec, lane, v);
        softmax_stats<L, N, true>(v, top, sum);
    }
    const int id = lane < a.top_k ? a.ids[row * a.top_k + lane] : -1;
    const bool there = id >= 0 && id < a.experts;
    const float ds = there ? a.scale * a.dweights[row * a.top_k + lane] : 0.0f;
    const float l = there ? load_logit<BF16>(a.logits, base + id) : 0.0f;
    const float inv = 1.0f / sum;
    float put = ds, dot = 0.0f;
    if (a.renorm) {
        float s;
        const float p = renormalised<L>(l, there, softmax, s);
        dot = row_reduce<L>(there ? ds * p : 0.0f, AddF());
        put = p * (ds - dot) * (softmax ? 1.0f : sigmoid(-l));
    } else if (softmax) {
        dot = row_reduce<L>(there ? ds * (expf(l - top) / sum) : 0.0f, AddF());
    } else {
        put = ds * sigmoid(l) * sigmoid(-l);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) rows_of[r][lane + L * c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    if (there) ((float*)rows_of[r])[id] = put;
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const float4 q = rows_of[r][lane + L * c];
        float o[4] = {q.x, q.y, q.z, q.w};
        const int e = 4 * (lane + L * c);
        if (dense) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = v[4 * c + i] == 0.0f ? 0.0f : v[4 * c + i] * inv * (o[i] - dot);     // (also where dot is NaN)
        }
        if (a.vec_out && e < a.experts) {
            if constexpr (BF16) {
                const u32x2v w = {f32_to_bf16_rne(o[0]) | f32_to_bf16_rne(o[1]) << 16,
                                  f32_to_bf16_rne(o[2]) | f32_to_bf16_rne(o[3]) << 16};
                __builtin_nontemporal_store(w, (u32x2v*)((uint16_t*)a.dlogits + row * a.dld + e));
            } else {
                const f32x4v w = {o[0], o[1], o[2], o[3]};
                __builtin_nontemporal_store(w, (f32x4v*)((float*)a.dlogits + row * a.dld + e));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (e + i >= a.experts) continue;
                if constexpr (BF16) ((uint16_t*)a.dlogits)[row * a.dld + e + i] = (uint16_t)f32_to_bf16_rne(o[i]);
                else ((float*)a.dlogits)[row * a.dld + e + i] = o[i];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch plan: a stable counting sort of the assignments i = t * top_k + j
// by expert.  Assignments without an expert sort into one more bin behind the
// last group.
//
// One launch counts each workgroup's share by expert, a second one places it:
// an assignment goes to its group's start, plus its expert's count in the
// workgroups, waves and rounds of 64 before it, plus its rank in its own
// round, where the lanes with the same expert find each other by comparing
// the bits of its number (one ballot a bit).  All are integers: the result is
// the same every run.
//
// Bound by latency: 524288 assignments over 256 experts take 4.2 + 11.4 us for
// 6 MB; of the second launch 3.9 us are every workgroup reading the counts of
// all, 2.1 us the scattered writes of row_index.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024, PLAN_WAVES = PLAN_THREADS / 64;
constexpr int PLAN_BINS = MAX_EXPERTS + 1;
constexpr int PLAN_ALONE = 2048;             // assignments that one workgroup sorts by itself
constexpr int PLAN_AHEAD = 16;               // loads of counts in flight

struct PlanArgs {
    const int32_t* ids;
    int64_t assignments;
    int top_k, experts;
    int pitch;                // words of a workgroup's counts: experts, rounded up to a multiple of 4
    int64_t chunk;            // assignments of a workgroup, a multiple of a tile
    int blocks;               // workgroups with assignments
    int32_t* counts;          // [workgroups][pitch]
    int32_t *offsets, *row_index, *slot;
};

__device__ __forceinline__ int plan_bin(const PlanArgs& a, int64_t i) {
    const int id = a.ids[i];
    return id >= 0 && id < a.experts ? id : a.experts;
}

__global__ __launch_bounds__(PLAN_THREADS) void plan_count_kernel(PlanArgs a) {
    __shared__ int hist[PLAN_BINS];
    for (int e = threadIdx.x; e <= a.experts; e += PLAN_THREADS) hist[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, end = min(begin + a.chunk, a.assignments);
    for (int64_t i = begin + threadIdx.x; i < end; i += 2 * PLAN_THREADS) {
        const int64_t j = i + PLAN_THREADS;
        const int e = plan_bin(a, i), f = j < end ? plan_bin(a, j) : -1;
        atomicAdd(&hist[e], 1);
        if (f >= 0) atomicAdd(&hist[f], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.pitch; e += PLAN_THREADS)
        a.counts[(int64_t)blockIdx.x * a.pitch + e] = e < a.experts ? hist[e] : 0;
}

// Exclusive prefix sums of n counts in LDS, by one wave: each lane sums a run
// of its own, the lanes' sums are scanned, and the run is added up again.
__device__ __forceinline__ void wave_scan(const int* in, int* out, int n) {
    const int lane = threadIdx.x & 63, per = (n + 63) / 64;
    const int begin = min(n, lane * per), end = min(n, begin + per);
    int own = 0;
    for (int i = begin; i < end; ++i) own += in[i];
    int x = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
    }
    int run = x - own;
    for (int i = begin; i < end; ++i) {
        const int c = in[i];
        out[i] = run;
        run += c;
    }
}

// A tile is Q rounds of 64 assignments for each wave.
template <int Q>
__global__ __launch_bounds__(PLAN_THREADS) void plan_scatter_kernel(PlanArgs a) {
    __shared__ int total[PLAN_BINS], before[PLAN_BINS], base[PLAN_BINS], before_all;
    union Scratch {
        uint16_t wave_count[PLAN_WAVES][PLAN_BINS + 3];
        int4 sums[2][PLAN_WAVES][64];         // of 256 experts: over all workgroups, over those before this one
    };
    __shared__ Scratch scratch;
    auto& wave_count = scratch.wave_count;
    constexpr int TILE = PLAN_THREADS * Q;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bins = a.experts + 1;
    for (int e = tid; e < bins; e += PLAN_THREADS) total[e] = before[e] = 0;
    __syncthreads();
    if (a.blocks <= 1) {                      // one workgroup counts for itself
        for (int64_t i = tid; i < a.assignments; i += PLAN_THREADS) atomicAdd(&total[plan_bin(a, i)], 1);
    } else {
        // a wave takes every 16th workgroup's counts, four experts a lane, with
        // PLAN_AHEAD of them under way at once; then the waves' sums are added
        const int quads = a.pitch / 4;
        for (int q0 = 0; q0 < quads; q0 += 64) {
            const int quad = min(q0 + lane, quads - 1);
            int4 all = {0, 0, 0, 0}, mine = {0, 0, 0, 0};
            for (int b0 = wave; b0 < a.blocks; b0 += PLAN_AHEAD * PLAN_WAVES) {
                int4 n[PLAN_AHEAD];
#pragma unroll
                for (int i = 0; i < PLAN_AHEAD; ++i)
                    n[i] = ((const int4*)a.counts)[(int64_t)min(b0 + i * PLAN_WAVES, a.blocks - 1) * quads + quad];
#pragma unroll
                for (int i = 0; i < PLAN_AHEAD; ++i) {
                    const int b = b0 + i * PLAN_WAVES;
                    if (b >= a.blocks) continue;
                    all.x += n[i].x; all.y += n[i].y; all.z += n[i].z; all.w += n[i].w;
                    if (b >= (int)blockIdx.x) continue;
                    mine.x += n[i].x; mine.y += n[i].y; mine.z += n[i].z; mine.w += n[i].w;
                }
            }
            scratch.sums[0][wave][lane] = all;
            scratch.sums[1][wave][lane] = mine;
            __syncthreads();
            const int which = tid >> 8, e = 4 * q0 + (tid & 255);
            if (which < 2 && e < a.experts) {
                int sum = 0;
#pragma unroll
                for (int w = 0; w < PLAN_WAVES; ++w) sum += ((const int*)scratch.sums[which][w])[tid & 255];
                (which ? before : total)[e] = sum;
            }
            __syncthreads();
        }
    }
    __syncthreads();
    if (wave == 0) wave_scan(total, base, bins);
    if (wave == 1) {                          // what is not some expert's lies in the last bin
        int sum = 0;
        for (int e = lane; e < a.experts; e += 64) sum += before[e];
#pragma unroll
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) before_all = sum;
    }
    __syncthreads();
    for (int e = tid; e < bins; e += PLAN_THREADS) {
        if (blockIdx.x == 0) a.offsets[e] = base[e];
        base[e] += e < a.experts ? before[e] : (int)((int64_t)blockIdx.x * a.chunk) - before_all;
    }
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, end = min(begin + a.chunk, a.assignments);
    for (int64_t at = begin; at < end; at += TILE) {
        const int64_t first = at + wave * 64 * Q + lane;
        int e[Q], rank[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) e[q] = first + 64 * q < end ? plan_bin(a, first + 64 * q) : 0;
        uint16_t* count = wave_count[wave];
        for (int b = lane; b < bins; b += 64) count[b] = 0;
        wave_fence();
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const bool live = first + 64 * q < end;
            uint64_t same = __ballot(live);
            for (int bit = 1; bit <= a.experts; bit <<= 1) {
                const uint64_t set = __ballot((e[q] & bit) != 0);
                same &= (e[q] & bit) ? set : ~set;
            }
            const int ahead = __popcll(same & ((1ull << lane) - 1)), held = count[e[q]];
            rank[q] = held + ahead;
            wave_fence();
            if (live && ahead == 0) count[e[q]] = (uint16_t)(held + __popcll(same));
            wave_fence();
        }
        __syncthreads();
        for (int b = tid; b < bins; b += PLAN_THREADS) {
            int n[PLAN_WAVES], run = 0;
#pragma unroll
            for (int w = 0; w < PLAN_WAVES; ++w) n[w] = wave_count[w][b];
#pragma unroll
            for (int w = 0; w < PLAN_WAVES; ++w) {
                wave_count[w][b] = (uint16_t)run;
                run += n[w];
            }
            total[b] = run;                   // this tile's count
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int64_t i = first + 64 * q;
            if (i >= end) continue;
            const int pos = base[e[q]] + count[e[q]] + rank[q];
            a.row_index[pos] = (int)((uint32_t)i / (uint32_t)a.top_k);
            a.slot[i] = e[q] < a.experts ? pos : -1;
        }
        __syncthreads();
        for (int b = tid; b < bins; b += PLAN_THREADS) base[b] += total[b];
    }
}

// Rounds of a wave in a tile and assignments of a workgroup.  A few
// assignments are sorted by one workgroup in one launch, before two launches
// would be done (2048 over 32 experts: 4.6 us, in two launches 6.9; 4096: 7.2
// and 6.9).  More are spread in small tiles until there are 256 workgroups,
// each of which adds up the counts of all; then the tiles grow (524288 over
// 256 experts: two rounds 15.1 us, one 15.6, four 16.9).
struct PlanShape {
    int rounds;
    int64_t chunk, blocks;
};
PlanShape plan_shape(int64_t n) {
    const int rounds = (n > PLAN_THREADS && n <= PLAN_ALONE) || n > 256 * PLAN_THREADS ? 2 : 1;
    const int64_t tile = rounds * PLAN_THREADS, tiles = max((int64_t)1, ceil_div(n, tile));
    const int64_t chunk = tile * (n <= PLAN_ALONE ? tiles : ceil_div(tiles, 256));
    return {rounds, chunk, ceil_div(n, chunk)};
}
int plan_pitch(int experts) { return (experts + 3) & ~3; }

template <bool B, int L, int C>
void launch_route(RouteArgs a, hipStream_t s) {
    constexpr int ROWS = 256 / L;
    size_t lds = 0;
    if (a.groups > 1) {
        a.group_size = a.experts / a.groups;
        a.group_inv = 1.0f / (float)a.group_size;
        while ((2 << a.share_log2) * a.groups <= L) ++a.share_log2;
        const int words = a.group_size % 4 == 0 ? a.experts / 2 : a.experts;
        a.score_at = (words + 4 * a.groups + 3) & ~3;
        a.row_floats = a.score_at + ((a.groups + 3) & ~3);
        lds = sizeof(float) * ROWS * (size_t)a.row_floats;
    }
    const dim3 grid((uint32_t)ceil_div(a.tokens, ROWS));
    // merged lists cost the same for any number up to 8, a row maximum each time the same again.
    // 65536 tokens, both directions, maxima / lists: 32 experts, top 4: 9.5 / 10.2 us; 128: 20.5 / 19.8
    // (top 3: 19.5 / 19.5); 256: 35.1 / 32.9 (top 3: 33.0 / 32.1, top 2: 30.9 / 31.5)
    if (a.top_k >= (C >= 4 ? 4 : 5) && a.top_k <= 8) hipLaunchKernelGGL((route_kernel<B, L, C, 8>), grid, dim3(256), lds, s, a);
    else hipLaunchKernelGGL((route_kernel<B, L, C, 0>), grid, dim3(256), lds, s, a);
}
template <bool B, int L, int C>
void launch_route(const RouteBwdArgs& a, hipStream_t s) {
    constexpr int ROWS = 256 / L;
    hipLaunchKernelGGL((route_bwd_kernel<B, L, C>), dim3((uint32_t)ceil_div(a.tokens, ROWS)), dim3(256), 0, s, a);
}

// The lanes that share a row and the chunks of four experts each holds: enough
// for the experts, and a lane for each chosen one.  With many tokens half as
// many lanes take a row: there is one step less between lanes, for twice the
// rows.  With few tokens twice the waves are done sooner.  Both directions,
// few / many tokens' lanes, top 8 of 256: 6.7 / 7.7 us at 4096 tokens,
// 8.7 / 8.5 at 8192, 36.9 / 35.9 at 65536; there of 64: 18.1 / 14.4, of 512:
// 58.4 / 52.7, of 1024: 114 / 100.
constexpr int64_t MANY_TOKENS = 8192;

template <bool B, class A>
void dispatch_route(const A& a, hipStream_t s) {
    const int e = a.experts, k = a.top_k;
    const bool many = a.tokens >= MANY_TOKENS && k <= 8;
    if (e <= 32 && k <= 8) launch_route<B, 8, 1>(a, s);
    else if (e <= 64 && many) launch_route<B, 8, 2>(a, s);
    else if (e <= 128 && many) launch_route<B, 8, 4>(a, s);
    else if (e <= 256 && many) launch_route<B, 8, 8>(a, s);
    else if (e <= 512 && many) launch_route<B, 16, 8>(a, s);
    else if (many) launch_route<B, 32, 8>(a, s);
    else if (e <= 64 && k <= 16) launch_route<B, 16, 1>(a, s);
    else if (e <= 128 && k <= 16) launch_route<B, 16, 2>(a, s);
    else if (e <= 256 && k <= 16) launch_route<B, 16, 4>(a, s);
    else if (e <= 512) launch_route<B, 32, 4>(a, s);
    else launch_route<B, 64, 4>(a, s);
}

mx_status check_route(mx_dtype lt, int64_t tokens, int32_t experts, int64_t ld, mx_score score, int32_t top_k,
                      float scale) {
    if (lt != MX_F32 && lt != MX_BF16) return MX_ERR_DTYPE;
    if (score != MX_SOFTMAX && score != MX_SIGMOID) return MX_ERR_UNSUPPORTED;
    if (tokens < 0 || experts < 1 || experts > MAX_EXPERTS) return MX_ERR_SHAPE;
    if (top_k < 1 || top_k > experts || top_k > MAX_TOP_K) return MX_ERR_SHAPE;
    if (ld && ld < experts) return MX_ERR_SHAPE;
    if (!(scale - scale == 0.0f)) return MX_ERR_SHAPE;
    if (tokens > (int64_t)INT32_MAX / top_k) return MX_ERR_SHAPE;
    if (tokens > ((int64_t)1 << 24)) return MX_ERR_SHAPE;   // 64 lanes a token at most, fewer than 2^32 threads
    return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_route(const void* logits, mx_dtype lt, int64_t tokens, int32_t experts, int64_t logits_ld,
                   const float* bias, mx_score score, int32_t groups, int32_t top_groups, int32_t group_best,
                   int32_t top_k, int renorm, float scale, int32_t* ids, float* weights, mx_stream stream) {
    const mx_status bad = check_route(lt, tokens, experts, logits_ld, score, top_k, scale);
    if (bad != MX_OK) return bad;
    if (groups < 1 || groups > MAX_GROUPS || experts % groups || top_groups < 1 || top_groups > groups)
        return MX_ERR_SHAPE;
    if (group_best != 1 && group_best != 2) return MX_ERR_SHAPE;
    if (top_k > top_groups * (experts / groups)) return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!logits || !ids || !weights) return MX_ERR_NULL;
    if (!aligned_to(logits, type_bytes(lt)) || !aligned_to(bias, 4) || !aligned_to(ids, 4) || !aligned_to(weights, 4))
        return MX_ERR_ALIGN;
    RouteArgs a{};
    a.logits = logits;
    a.tokens = tokens;
    a.ld = logits_ld ? logits_ld : experts;
    a.experts = experts;
    a.bias = bias;
    a.score = score;
    a.groups = groups == top_groups ? 1 : groups;      // every group stays
    a.top_groups = top_groups;
    a.group_best = group_best;
    a.top_k = top_k;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.vec = experts % 4 == 0 && a.ld % 4 == 0 && aligned_to(logits, 4 * type_bytes(lt));
    a.vec_bias = experts % 4 == 0 && aligned_to(bias, 16);
    (void)hipGetLastError();
    if (lt == MX_BF16) dispatch_route<true>(a, (hipStream_t)stream);
    else dispatch_route<false>(a, (hipStream_t)stream);
    return launch_status();
}

mx_status mx_route_bwd(const void* logits, mx_dtype lt, int64_t tokens, int32_t experts, int64_t logits_ld,
                       mx_score score, int32_t top_k, int renorm, float scale, const int32_t* ids,
                       const float* dweights, void* dlogits, int64_t dlogits_ld, mx_stream stream) {
    const mx_status bad = check_route(lt, tokens, experts, logits_ld, score, top_k, scale);
    if (bad != MX_OK) return bad;
    if (dlogits_ld && dlogits_ld < experts) return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!logits || !ids || !dweights || !dlogits) return MX_ERR_NULL;
    if (!aligned_to(logits, type_bytes(lt)) || !aligned_to(ids, 4) || !aligned_to(dweights, 4) ||
        !aligned_to(dlogits, type_bytes(lt)))
        return MX_ERR_ALIGN;
    RouteBwdArgs a{logits, tokens, logits_ld ? logits_ld : experts, experts, score, top_k, renorm != 0, scale, 0, 0,
                   ids, dweights, dlogits, dlogits_ld ? dlogits_ld : experts};
    a.vec = experts % 4 == 0 && a.ld % 4 == 0 && aligned_to(logits, 4 * type_bytes(lt));
    a.vec_out = experts % 4 == 0 && a.dld % 4 == 0 && aligned_to(dlogits, 4 * type_bytes(lt));
    (void)hipGetLastError();
    if (lt == MX_BF16) dispatch_route<true>(a, (hipStream_t)stream);
    else dispatch_route<false>(a, (hipStream_t)stream);
    return launch_status();
}

int64_t mx_route_plan_workspace(int64_t tokens, int32_t top_k, int32_t experts) {
    if (tokens < 0 || top_k < 1 || experts < 1 || experts > MAX_EXPERTS || tokens > (int64_t)INT32_MAX / top_k)
        return 0;
    const int64_t blocks = plan_shape(tokens * top_k).blocks;
    return blocks <= 1 ? 0 : 4 * blocks * plan_pitch(experts);
}

mx_status mx_route_plan(const int32_t* ids, int64_t tokens, int32_t top_k, int32_t experts, int32_t* offsets,
                        int32_t* row_index, int32_t* slot, void* workspace, mx_stream stream) {
    if (tokens < 0 || experts < 1 || experts > MAX_EXPERTS || top_k < 1) return MX_ERR_SHAPE;
    if (tokens > (int64_t)INT32_MAX / top_k) return MX_ERR_SHAPE;
    if (!offsets) return MX_ERR_NULL;
    const int64_t n = tokens * top_k;
    const PlanShape shape = plan_shape(n);
    if (n > 0 && (!ids || !row_index || !slot || (shape.blocks > 1 && !workspace))) return MX_ERR_NULL;
    if (!aligned_to(ids, 4) || !aligned_to(offsets, 4) || !aligned_to(row_index, 4) || !aligned_to(slot, 4) ||
        !aligned_to(workspace, 16))
        return MX_ERR_ALIGN;
    PlanArgs a{ids, n, top_k, experts, plan_pitch(experts), shape.chunk, (int)shape.blocks, (int32_t*)workspace,
               offsets, row_index, slot};
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (a.blocks > 1) hipLaunchKernelGGL(plan_count_kernel, dim3(a.blocks), dim3(PLAN_THREADS), 0, s, a);
    // with nothing to sort one workgroup writes the offsets, all 0
    const dim3 grid(max(a.blocks, 1));
    if (shape.rounds == 2) hipLaunchKernelGGL(plan_scatter_kernel<2>, grid, dim3(PLAN_THREADS), 0, s, a);
    else hipLaunchKernelGGL(plan_scatter_kernel<1>, grid, dim3(PLAN_THREADS), 0, s, a);
    return launch_status();
}

}  // extern "C"
