// mx_balance.hip -- a router's balance loss, its experts' counts, and its
// gradient (gfx950).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_device.h"
#include "mx_host.h"
#include "mx_rows.h"

namespace {

using namespace mx;

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_IDS = 1024;                // of a token
constexpr int THREADS = 1024;                // of a workgroup that sums scores
constexpr int MAX_BLOCKS = 256;              // of them

struct BalanceArgs {
    const void* logits;
    int64_t tokens, ld;
    int experts, score, vec;
    const int32_t* ids;
    int64_t assignments;
    int top_k;
    float* sums;              // [blocks][experts]
    int32_t* counts;          // [blocks][experts + 1]: assignments, then tokens with scores
    int blocks;
};

// The scores of a row from its logits, in place, and (sigmoid) the factor 1 -
// sigmoid(l) that the gradient needs.  A row of -inf alone has scores 0.
// Sigmoid scores whose sum would underflow (every logit below -40, where the
// sigmoid is e^l to 24 bits) are those of a softmax.
template <int L, int N, bool SLOPES>
__device__ __forceinline__ void row_scores(float* v, bool softmax, float* rest) {
    float top, sum;
    if (!softmax) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
        top = row_reduce<L>(m, MaxF());
    }
    if (softmax || top < -40.0f) {
        softmax_stats<L, N, true>(v, top, sum);
        if constexpr (SLOPES) {
#pragma unroll
            for (int i = 0; i < N; ++i) rest[i] = 1.0f;
        }
    } else {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = soft_exp(-fabsf(v[i])), r = __builtin_amdgcn_rcpf(1.0f + e);     // (NaN stays NaN)
            const bool up = v[i] >= 0.0f;
            if constexpr (SLOPES) rest[i] = up ? e * r : r;
            v[i] = up ? r : e * r;
            sum += v[i];
        }
        sum = row_reduce<L>(sum, AddF());
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= inv;
}

// Sums of the scores over a workgroup's tokens, and its assignments by expert.
// L lanes share a row, as in the router.  Sums per expert stay in the registers of
// the lanes that hold the expert, so a token costs no atomics; few, large
// workgroups leave few rows to be added up.  65536 x 256 in fp32: 19.6 us (3.6
// TB/s); the vector instructions, 27 an element, two of them exponential and
// reciprocal, take three quarters of the issue slots.  16384 x 32 in bf16 4.7 us.
template <bool BF16, int L, int C>
__global__ __launch_bounds__(THREADS) void balance_kernel(BalanceArgs a) {
    constexpr int N = 4 * C, ROWS = THREADS / L, E = 4 * L * C;
    __shared__ float part[THREADS / 64][E];
    __shared__ int count[E + 1];
    for (int e = threadIdx.x; e <= a.experts; e += THREADS) count[e] = 0;
    __syncthreads();
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.assignments; i += (int64_t)a.blocks * THREADS) {
        const int id = a.ids[i];
        if (id >= 0 && id < a.experts) atomicAdd(&count[id], 1);
    }
    const int lane = threadIdx.x & (L - 1), r = threadIdx.x / L;
    const bool softmax = a.score == MX_SOFTMAX;
    float acc[N] = {};
    int used = 0;
    // the next rows are under way while these are worked on
    const int64_t step = (int64_t)a.blocks * ROWS;
    float v[N], next[N];
    int64_t row = (int64_t)blockIdx.x * ROWS + r;
    load_row<BF16, L, C>(a.logits, min(row, a.tokens - 1) * a.ld, a.experts, a.vec, lane, next);
    for (; row - r < a.tokens; row += step) {
        const bool live = row < a.tokens;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = next[i];
        load_row<BF16, L, C>(a.logits, min(row + step, a.tokens - 1) * a.ld, a.experts, a.vec, lane, next);
        float any = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) any = v[i] == -__builtin_inff() ? any : 1.0f;
        const bool scored = row_reduce<L>(any, MaxF()) > 0.0f;     // (by all lanes of the row)
        used += live && lane == 0 && scored;
        row_scores<L, N, false>(v, softmax, nullptr);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += live ? v[i] : 0.0f;
    }
    // the rows of a wave, then the waves
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int d = 32; d >= L; d >>= 1) acc[i] += __shfl_xor(acc[i], d);
    }
    const int at = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (at < L) {
#pragma unroll
        for (int i = 0; i < N; ++i) part[wave][4 * (lane + L * (i >> 2)) + (i & 3)] = acc[i];
    }
    if (used) atomicAdd(&count[a.experts], used);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) s += part[w][e];
        a.sums[(int64_t)blockIdx.x * a.experts + e] = s;
    }
    for (int e = threadIdx.x; e <= a.experts; e += THREADS)
        a.counts[(int64_t)blockIdx.x * (a.experts + 1) + e] = count[e];
}

// The workgroups' sums and counts, then the slopes and the loss.  Threads side
// by side take neighbouring experts, 2^lanes_log2 of them, and the others
// further workgroups' rows, eight at a time.
__global__ __launch_bounds__(THREADS) void balance_loss_kernel(const float* sums, const int32_t* counts, int blocks,
                                                               int experts, int lanes_log2, int32_t* out_counts,
                                                               float* slope, float* loss) {
    __shared__ double part[THREADS], total[THREADS / 64];
    __shared__ long long made_part[THREADS], made[THREADS / 64];
    constexpr int AHEAD = 8;
    const int e = threadIdx.x & ((1 << lanes_log2) - 1), first = threadIdx.x >> lanes_log2, step = THREADS >> lanes_log2;
    double s = 0.0;
    int c = 0;
    for (int b0 = first; b0 < blocks; b0 += AHEAD * step) {
        float x[AHEAD];
        int y[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int b = min(b0 + i * step, blocks - 1), at = min(e, experts - 1);
            x[i] = sums[(int64_t)b * experts + at];
            y[i] = counts[(int64_t)b * (experts + 1) + at];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = b0 + i * step < blocks && e < experts;
            s += in ? (double)x[i] : 0.0;
            c += in ? y[i] : 0;
        }
    }
    int used = 0;
    for (int b = threadIdx.x; b < blocks; b += THREADS) used += counts[(int64_t)b * (experts + 1) + experts];
    part[threadIdx.x] = s;
    made_part[threadIdx.x] = (long long)c << 32 | (uint32_t)used;      // (their sums stay below 2^31 each)
    __syncthreads();
    s = 0.0;
    long long n = made_part[threadIdx.x];
    c = 0;
    if (threadIdx.x < 1 << lanes_log2) {
        for (int i = threadIdx.x; i < THREADS; i += 1 << lanes_log2) {
            s += part[i];
            c += (int)(made_part[i] >> 32);
        }
        if (e < experts) out_counts[e] = c;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
    if ((threadIdx.x & 63) == 0) made[threadIdx.x >> 6] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) n += made[w];
    const double all = (double)(n >> 32) * (double)(uint32_t)n;
    const bool mine = threadIdx.x < 1 << lanes_log2 && e < experts;
    const double k = mine && all > 0.0 ? (double)experts * (double)c / all : 0.0;
    if (mine) slope[e] = (float)k;
    double l = mine && all > 0.0 ? k * s : 0.0;
#pragma unroll
    for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
    if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        l = 0.0;
        for (int w = 0; w < THREADS / 64; ++w) l += total[w];
        *loss = (float)l;
    }
}

struct BalanceBwdArgs {
    const void* logits;
    int64_t tokens, ld;
    int experts, score, vec, vec_slope, vec_add, vec_out;
    const float* slope;
    const float* dloss;
    float scale;
    const void* add;
    int64_t add_ld;
    void* dlogits;
    int64_t dld;
};

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

// dl = factor * s (slope - <slope, s>), for sigmoid scores times 1 - sigmoid(l), and
// `add` more.  One pass; 65536 x 256 in fp32 with `add` 31.1 us, 6.5 TB/s: HBM.
template <bool BF16, int L, int C>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
    constexpr int N = 4 * C, ROWS = 256 / L;
    const int lane = threadIdx.x & (L - 1), r = threadIdx.x / L;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS + r;
    const bool live = row0 < a.tokens;
    const int64_t row = live ? row0 : a.tokens - 1;
    float v[N], f[N], rest[N], g[N];
    load_row<BF16, L, C>(a.logits, row * a.ld, a.experts, a.vec, lane, v);
    load_row<false, L, C>(a.slope, 0, a.experts, a.vec_slope, lane, f, 0.0f);
    if (a.add) load_row<BF16, L, C>(a.add, row * a.add_ld, a.experts, a.vec_add, lane, g, 0.0f);
    const float factor = a.dloss ? a.scale * *a.dloss : a.scale;
    row_scores<L, N, true>(v, a.score == MX_SOFTMAX, rest);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) dot = __builtin_fmaf(f[i], v[i], dot);
    dot = row_reduce<L>(dot, AddF());
    if (!live) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = 4 * (lane + L * c);
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * c + i;
            o[i] = v[n] == 0.0f ? 0.0f : factor * (v[n] * (f[n] - dot) * rest[n]);
            if (a.add) o[i] += g[n];
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

template <bool B, int L, int C>
void launch(const BalanceArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((balance_kernel<B, L, C>), dim3(a.blocks), dim3(THREADS), 0, s, a);
}
template <bool B, int L, int C>
void launch(const BalanceBwdArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((balance_bwd_kernel<B, L, C>), dim3((uint32_t)ceil_div(a.tokens, 256 / L)), dim3(256), 0, s, a);
}
// The lanes that share a row and the chunks of four experts each holds.  With
// many tokens half as many lanes take a row of the backward pass, as in the
// router; the forward's workgroups walk over rows and keep a sum for every
// element, for which fewer registers are faster than fewer lanes.
constexpr int64_t MANY_TOKENS = 8192;
template <bool B, bool MANY, class A>
void dispatch(const A& a, hipStream_t s) {
    const int e = a.experts;
    if (e <= 32) launch<B, 8, 1>(a, s);
    else if (e <= 64) launch<B, MANY ? 8 : 16, MANY ? 2 : 1>(a, s);
    else if (e <= 128) launch<B, MANY ? 8 : 16, MANY ? 4 : 2>(a, s);
    else if (e <= 256) launch<B, MANY ? 8 : 16, MANY ? 8 : 4>(a, s);
    else if (e <= 512) launch<B, 32, 4>(a, s);
    else launch<B, 64, 4>(a, s);
}

mx_status check_balance(mx_dtype lt, int64_t tokens, int32_t experts, int64_t ld, mx_score score) {
    if (lt != MX_F32 && lt != MX_BF16) return MX_ERR_DTYPE;
    if (score != MX_SOFTMAX && score != MX_SIGMOID) return MX_ERR_UNSUPPORTED;
    if (tokens < 0 || tokens > ((int64_t)1 << 24) || experts < 1 || experts > MAX_EXPERTS) return MX_ERR_SHAPE;
    return ld && ld < experts ? MX_ERR_SHAPE : MX_OK;
}

int blocks_of(int64_t tokens) { return (int)lesser(ceil_div(tokens, 64), MAX_BLOCKS); }

}  // namespace

extern "C" {

int64_t mx_balance_workspace(int64_t tokens, int32_t experts) {
    if (tokens <= 0 || experts < 1 || experts > MAX_EXPERTS) return 0;
    return blocks_of(tokens) * (2 * (int64_t)experts + 1) * 4;
}

mx_status mx_balance(const void* logits, mx_dtype lt, int64_t tokens, int32_t experts, int64_t logits_ld,
                     mx_score score, const int32_t* ids, int32_t top_k, int32_t* counts, float* slope, float* loss,
                     void* workspace, mx_stream stream) {
    const mx_status bad = check_balance(lt, tokens, experts, logits_ld, score);
    if (bad != MX_OK) return bad;
    if (top_k < 1 || top_k > MAX_IDS || tokens > (int64_t)INT32_MAX / top_k) return MX_ERR_SHAPE;
    if (!counts || !slope || !loss || (tokens > 0 && (!logits || !ids || !workspace))) return MX_ERR_NULL;
    if (!aligned_to(logits, type_bytes(lt)) || !aligned_to(ids, 4) || !aligned_to(counts, 4) || !aligned_to(slope, 4) ||
        !aligned_to(loss, 4) || !aligned_to(workspace, 16))
        return MX_ERR_ALIGN;
    const int blocks = tokens > 0 ? blocks_of(tokens) : 0;
    BalanceArgs a{logits, tokens, logits_ld ? logits_ld : experts, experts, score, 0, ids, tokens * top_k, top_k,
                  (float*)workspace, (int32_t*)workspace + (int64_t)blocks * experts, blocks};
    a.vec = experts % 4 == 0 && a.ld % 4 == 0 && aligned_to(logits, 4 * type_bytes(lt));
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (blocks > 0) {
        if (lt == MX_BF16) dispatch<true, false>(a, s);
        else dispatch<false, false>(a, s);
    }
    int lanes_log2 = 0;
    while (1 << lanes_log2 < experts) ++lanes_log2;
    hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(THREADS), 0, s, a.sums, a.counts, blocks, experts, lanes_log2,
                       counts, slope, loss);
    return launch_status();
}

mx_status mx_balance_bwd(const void* logits, mx_dtype lt, int64_t tokens, int32_t experts, int64_t logits_ld,
                         mx_score score, const float* slope, const float* dloss, float scale, const void* add,
                         int64_t add_ld, void* dlogits, int64_t dlogits_ld, mx_stream stream) {
    const mx_status bad = check_balance(lt, tokens, experts, logits_ld, score);
    if (bad != MX_OK) return bad;
    if ((add_ld && add_ld < experts) || (dlogits_ld && dlogits_ld < experts) || !(scale - scale == 0.0f))
        return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!logits || !slope || !dlogits) return MX_ERR_NULL;
    if (!aligned_to(logits, type_bytes(lt)) || !aligned_to(slope, 4) || !aligned_to(dloss, 4) ||
        !aligned_to(add, type_bytes(lt)) || !aligned_to(dlogits, type_bytes(lt)))
        return MX_ERR_ALIGN;
    BalanceBwdArgs a{logits, tokens, logits_ld ? logits_ld : experts, experts, score, 0, 0, 0, 0, slope, dloss, scale,
                     add, add_ld ? add_ld : experts, dlogits, dlogits_ld ? dlogits_ld : experts};
    const size_t four = 4 * type_bytes(lt);
    a.vec = experts % 4 == 0 && a.ld % 4 == 0 && aligned_to(logits, four);
    a.vec_slope = experts % 4 == 0 && aligned_to(slope, 16);
    a.vec_add = experts % 4 == 0 && a.add_ld % 4 == 0 && aligned_to(add, four);
    a.vec_out = experts % 4 == 0 && a.dld % 4 == 0 && aligned_to(dlogits, four);
    (void)hipGetLastError();
    hipStream_t s = (hipStream_t)stream;
    const bool many = tokens >= MANY_TOKENS;
    if (lt == MX_BF16) many ? dispatch<true, true>(a, s) : dispatch<true, false>(a, s);
    else many ? dispatch<false, true>(a, s) : dispatch<false, false>(a, s);
    return launch_status();
}

}  // extern "C"
