// mx_combine.hip -- the weighted sum of the experts' rows for each token, and
// its gradient (gfx950).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_device.h"
#include "mx_host.h"

namespace {

using namespace mx;

struct CombineArgs {
    const void* y;            // [rows x cols], pitch y_ld
    int64_t rows, cols, y_ld;
    const int32_t* slot;      // [tokens x top_k]
    const float* weights;     // [tokens x top_k] or null
    int64_t tokens;
    int top_k;
    const void* residual;     // [tokens x cols] or null
    int64_t res_ld;
    void* out;
    int64_t out_ld;
    int64_t chunks;           // waves that share a row
};

// Pieces of 8 and 16 bytes at any element's address: global memory takes them
// at any alignment, so rows need none beyond their elements'.
typedef unsigned int u32x2v __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned int u32x4v __attribute__((ext_vector_type(4), aligned(2)));

// STREAM: past the caches (non-temporal).  Stores always are: no dirty lines
// are left to write back when the kernel ends (the gradient of 1024 tokens of
// 4 rows of 2880 took 12.1 us without, 10.0 with them; never slower).
template <bool STREAM, class T>
__device__ __forceinline__ T load_piece(const void* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load((const T*)p);
    else return *(const T*)p;
}
template <class T>
__device__ __forceinline__ void store_piece(void* p, T v) {
    __builtin_nontemporal_store(v, (T*)p);
}

// V consecutive elements of a row, as they are in memory.
template <bool BF16, int V>
struct Piece {
    uint32_t u[BF16 ? V / 2 : V];

    // Without FULL the row ends after `left` of them (then element by element,
    // and 0 past it).
    template <bool FULL, bool STREAM>
    __device__ __forceinline__ void load(const void* p, int64_t at, int64_t left) {
        constexpr int W = BF16 ? V / 2 : V;
        const char* q = (const char*)p + at * (BF16 ? 2 : 4);
        if constexpr (!FULL) {
#pragma unroll
            for (int i = 0; i < W; ++i) u[i] = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i >= left) continue;
                if constexpr (BF16) u[i / 2] |= (uint32_t)((const uint16_t*)q)[i] << (i % 2 * 16);
                else u[i] = ((const uint32_t*)q)[i];
            }
        } else if constexpr (W == 2) {
            const u32x2v w = load_piece<STREAM, u32x2v>(q);
            u[0] = w.x; u[1] = w.y;
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const u32x4v w = load_piece<STREAM, u32x4v>(q + 4 * i);
                u[i] = w.x; u[i + 1] = w.y; u[i + 2] = w.z; u[i + 3] = w.w;
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (BF16) return i % 2 ? bf16hi(u[i / 2]) : bf16lo(u[i / 2]);
        else return __uint_as_float(u[i]);
    }
};

template <bool BF16, int V, bool FULL>
__device__ __forceinline__ void store_v(void* p, int64_t at, int64_t left, const float* f) {
    if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= left) continue;
            if constexpr (BF16) ((uint16_t*)p)[at + i] = (uint16_t)f32_to_bf16_rne(f[i]);
            else ((float*)p)[at + i] = f[i];
        }
    } else if constexpr (BF16) {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) u[i] = f32_to_bf16_rne(f[2 * i]) | f32_to_bf16_rne(f[2 * i + 1]) << 16;
        if constexpr (V == 8) store_piece((uint16_t*)p + at, (u32x4v){u[0], u[1], u[2], u[3]});
        else store_piece((uint16_t*)p + at, (u32x2v){u[0], u[1]});
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            store_piece((float*)p + at + i, (u32x4v){__float_as_uint(f[i]), __float_as_uint(f[i + 1]),
                                                             __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3])});
    }
}

// Up to FLIGHT assignments of a token, whose rows are read at once.  All of
// them arrive after one round trip, as scalars; the loads of the rows are then
// issued without waiting for each other, and widened only when all are under
// way.  A slot past top_k or outside [0, rows) becomes -1.
constexpr int FLIGHT = 4;

struct Flight {
    int slot[FLIGHT];
    float weight[FLIGHT];

    // Those from j0 on, for a whole wave (every lane active): lane i fetches
    // one, and the lanes hand them round.
    __device__ __forceinline__ void load_by_lanes(const int32_t* slots, const float* weights, int64_t t, int top_k,
                                                  int j0, int64_t rows) {
        const int j = j0 + (threadIdx.x & (FLIGHT - 1));
        const bool in = j < top_k;
        const int s = in ? slots[t * top_k + j] : -1;
        const float w = in && weights ? weights[t * top_k + j] : 1.0f;
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            slot[i] = __builtin_amdgcn_readlane(s, i);
            slot[i] = slot[i] < rows ? slot[i] : -1;
            weight[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), i));
        }
    }

    // The same from addresses that are uniform in the wave: whichever lanes are
    // active have loaded what they use themselves.  (As the only way it costs
    // combine_kernel 84.9 us against 80.3 at the size named there.)
    __device__ __forceinline__ void load_uniform(const int32_t* slots, const float* weights, int64_t t, int top_k,
                                                 int j0, int64_t rows) {
        const int64_t first = t * top_k;
        const int32_t* factors = weights ? (const int32_t*)weights : slots;     // (no branch among the loads)
        int f[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            const int64_t at = first + min(j0 + i, top_k - 1);
            slot[i] = __builtin_amdgcn_readfirstlane(slots[at]);
            f[i] = __builtin_amdgcn_readfirstlane(factors[at]);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            slot[i] = j0 + i < top_k && slot[i] < rows ? slot[i] : -1;
            weight[i] = weights ? __int_as_float(f[i]) : 1.0f;
        }
    }
};

// out[t] = residual[t] + sum_j w_tj y[slot_tj].  Bound by memory: each row of
// y is read once, each token written once.
// One wave: 64 V columns of one token; a row's waves follow one another, so
// the waves of a workgroup read neighbouring pieces of the same rows.  One
// wave for a whole token was slower (117 against 107 us at the size below).
// 16384 tokens of 4 rows, 2880 bf16 columns, with a residual: 77-80 us, 7.1 to
// 7.3 TB/s (a copy of that size: 5.5); of 8 rows 138 us, 6.8 TB/s.
template <bool YB, bool OB, bool STREAM, bool FULL>
__device__ __forceinline__ void combine_piece(const CombineArgs& a, int64_t t, int64_t col, Flight& n) {
    constexpr int V = YB ? 8 : 4;
    const int64_t left = a.cols - col;
    float acc[V];
    Piece<OB, V> r;
    if (a.residual) r.template load<FULL, false>(a.residual, t * a.res_ld + col, left);
    for (int j0 = 0;;) {
        Piece<YB, V> f[FLIGHT];
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j)
            if (n.slot[j] >= 0) f[j].template load<FULL, STREAM>(a.y, n.slot[j] * a.y_ld + col, left);
        if (j0 == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = a.residual ? r[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
            if (n.slot[j] < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(n.weight[j], f[j][i], acc[i]);
        }
        j0 += FLIGHT;
        if (j0 >= a.top_k) break;
        // (lanes past the row's end, or on its other side of FULL, are not here)
        n.load_uniform(a.slot, a.weights, t, a.top_k, j0, a.rows);
    }
    store_v<OB, V, FULL>(a.out, t * a.out_ld + col, left, acc);
}

template <bool YB, bool OB, bool STREAM>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    constexpr int V = YB ? 8 : 4;
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = w / a.chunks;
    if (t >= a.tokens) return;
    Flight n;
    n.load_by_lanes(a.slot, a.weights, t, a.top_k, 0, a.rows);
    const int64_t col = (w % a.chunks * 64 + (threadIdx.x & 63)) * V;
    if (col >= a.cols) return;
    if (a.cols - col >= V) combine_piece<YB, OB, STREAM, true>(a, t, col, n);
    else combine_piece<YB, OB, STREAM, false>(a, t, col, n);
}

struct CombineBwdArgs {
    const void* dout;
    int64_t dout_ld;
    const void* y;
    int64_t rows, cols, y_ld;
    const int32_t* slot;
    const float* weights;
    int64_t tokens;
    int top_k;
    const int32_t* used_rows;
    void* dy;
    int64_t dy_ld;
    float* dweights;
};

// dy[slot_tj] = w_tj dout[t] and dw_tj = <dout[t], y[slot_tj]> from one read of
// dout and y.  Bound by memory.
// One workgroup: one token, its waves side by side along the columns (one wave
// a token: 5% slower at the size below).  Beyond the tokens the workgroups
// clear the rows of dy past the used ones.  16384 tokens of 4 rows, 2880 bf16
// columns: 141 us, 6.0 TB/s; of 8 rows 288 us, 5.6 TB/s.
constexpr int MAX_WAVES = 8;

// The sums over a wave of FLIGHT values, in a fixed order: lanes 16 j .. 16 j + 15
// get that of value j.  In each of the first two steps a lane hands on the half
// of the values that it does not keep.
__device__ __forceinline__ float wave_sums(const float (&v)[FLIGHT]) {
    static_assert(FLIGHT == 4, "two halvings");
    const bool b5 = threadIdx.x & 32, b4 = threadIdx.x & 16;
    const float x = (b5 ? v[2] : v[0]) + __shfl_xor(b5 ? v[0] : v[2], 32);
    const float y = (b5 ? v[3] : v[1]) + __shfl_xor(b5 ? v[1] : v[3], 32);
    float s = (b4 ? y : x) + __shfl_xor(b4 ? x : y, 16);
    s += quad_xor1(s);
    s += quad_xor2(s);
    s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0x141, 0xF, 0xF, false));   // other quad
    s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0x140, 0xF, 0xF, false));   // other eight
    return s;
}

template <bool DB, bool YB, bool STREAM, bool FULL>
__device__ __forceinline__ void bwd_piece(const CombineBwdArgs& a, int64_t t, int64_t col, const Flight& n,
                                          float* dot) {
    constexpr int V = YB ? 8 : 4;
    const int64_t left = a.cols - col;
    Piece<DB, V> d;
    Piece<YB, V> f[FLIGHT];
    d.template load<FULL, false>(a.dout, t * a.dout_ld + col, left);
    if (a.dweights) {
        // (before any store: dy may be y)
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j)
            if (n.slot[j] >= 0) f[j].template load<FULL, STREAM>(a.y, n.slot[j] * a.y_ld + col, left);
    }
    float g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = d[i];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
        if (n.slot[j] < 0) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = n.weight[j] * g[i];
        store_v<YB, V, FULL>(a.dy, n.slot[j] * a.dy_ld + col, left, v);
    }
    if (a.dweights) {
#pragma unroll
        for (int j = 0; j < FLIGHT; ++j) {
            if (n.slot[j] < 0) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = __builtin_fmaf(g[i], f[j][i], dot[j]);
        }
    }
}

template <bool DB, bool YB, bool STREAM>
__global__ __launch_bounds__(64 * MAX_WAVES) void combine_bwd_kernel(CombineBwdArgs a) {
    constexpr int V = YB ? 8 : 4;
    __shared__ float part[MAX_WAVES][FLIGHT];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int64_t used = a.used_rows ? min(max((int64_t)*a.used_rows, (int64_t)0), a.rows) : a.rows;
    if ((int64_t)blockIdx.x >= a.tokens) {
        const float zero[V] = {};
        for (int64_t r = used + blockIdx.x - a.tokens; r < a.rows; r += gridDim.x - a.tokens)
            for (int64_t col = tid * V; col < a.cols; col += threads * V) {
                if (a.cols - col >= V) store_v<YB, V, true>(a.dy, r * a.dy_ld + col, V, zero);
                else store_v<YB, V, false>(a.dy, r * a.dy_ld + col, a.cols - col, zero);
            }
        return;
    }
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < a.top_k; j0 += FLIGHT) {
        Flight n;
        n.load_by_lanes(a.slot, a.weights, t, a.top_k, j0, used);
        float dot[FLIGHT] = {};
        int64_t col = tid * V;
        for (; col <= a.cols - V; col += threads * V) bwd_piece<DB, YB, STREAM, true>(a, t, col, n, dot);
        if (col < a.cols) bwd_piece<DB, YB, STREAM, false>(a, t, col, n, dot);
        if (!a.dweights) continue;
        const float sum = wave_sums(dot);
        __syncthreads();
        if ((tid & 15) == 0) part[tid >> 6][(tid >> 4) & 3] = sum;
        __syncthreads();
        if (tid < FLIGHT && j0 + tid < a.top_k) {
            float total = 0.0f;
            for (int w = 0; w < threads / 64; ++w) total += part[w][tid];
            a.dweights[t * a.top_k + j0 + tid] = total;
        }
    }
}

mx_status check_combine(mx_dtype yt, mx_dtype ot, int64_t rows, int64_t cols, int64_t y_ld, int64_t tokens,
                        int32_t top_k) {
    if ((yt != MX_F32 && yt != MX_BF16) || (ot != MX_F32 && ot != MX_BF16)) return MX_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX || cols < 1 || tokens < 0 || top_k < 1) return MX_ERR_SHAPE;
    if (tokens > (int64_t)INT32_MAX / top_k) return MX_ERR_SHAPE;
    if (y_ld && y_ld < cols) return MX_ERR_SHAPE;
    return MX_OK;
}

// Whether the experts' rows are more than half of the 256 MB Infinity Cache:
// they are then read past the caches, which could not keep them for a
// neighbouring call.  Measured on bf16 rows of 2880, 4 a token, cached / past
// the caches: forward 10.7 / 11.4 us at 47 MB of rows, 19.6 / 20.6 at 94,
// 31.6 / 29.5 at 142, 107 / 86 at 377; gradient 19.8 / 21.9, 37.4 / 39.5,
// 55.9 / 56.0, 163 / 147.
bool streams(int64_t rows, int64_t cols, mx_dtype yt) {
    return (double)rows * (double)cols * (double)type_bytes(yt) > 128e6;
}

}  // namespace

extern "C" {

mx_status mx_combine(const void* y, mx_dtype yt, int64_t rows, int64_t cols, int64_t y_ld, const int32_t* slot,
                     const float* weights, int64_t tokens, int32_t top_k, const void* residual, int64_t residual_ld,
                     void* out, mx_dtype ot, int64_t out_ld, mx_stream stream) {
    const mx_status bad = check_combine(yt, ot, rows, cols, y_ld, tokens, top_k);
    if (bad != MX_OK) return bad;
    if ((residual_ld && residual_ld < cols) || (out_ld && out_ld < cols)) return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if ((!y && rows > 0) || !slot || !out) return MX_ERR_NULL;
    if (!aligned_to(y, type_bytes(yt)) || !aligned_to(slot, 4) || !aligned_to(weights, 4) ||
        !aligned_to(residual, type_bytes(ot)) || !aligned_to(out, type_bytes(ot)))
        return MX_ERR_ALIGN;
    CombineArgs a{y, rows, cols, y_ld ? y_ld : cols, slot, weights, tokens, top_k, residual,
                  residual_ld ? residual_ld : cols, out, out_ld ? out_ld : cols, 0};
    const int v = yt == MX_BF16 ? 8 : 4;
    a.chunks = ceil_div(cols, 64 * v);
    if (a.chunks > ((int64_t)1 << 25) / tokens) return MX_ERR_SHAPE;    // 2^31 threads at most
    const dim3 grid((uint32_t)ceil_div(tokens * a.chunks, 4));
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    const bool through = streams(tokens * top_k, cols, yt);
#define MX_COMBINE(YB, OB)                                                                                  \
    do {                                                                                                    \
        if (through) hipLaunchKernelGGL((combine_kernel<YB, OB, true>), grid, dim3(256), 0, s, a);          \
        else hipLaunchKernelGGL((combine_kernel<YB, OB, false>), grid, dim3(256), 0, s, a);                 \
    } while (0)
    if (yt == MX_BF16) {
        if (ot == MX_BF16) MX_COMBINE(true, true);
        else MX_COMBINE(true, false);
    } else {
        if (ot == MX_BF16) MX_COMBINE(false, true);
        else MX_COMBINE(false, false);
    }
#undef MX_COMBINE
    return launch_status();
}

mx_status mx_combine_bwd(const void* dout, mx_dtype dt, int64_t dout_ld, const void* y, mx_dtype yt, int64_t rows,
                         int64_t cols, int64_t y_ld, const int32_t* slot, const float* weights, int64_t tokens,
                         int32_t top_k, const int32_t* used_rows, void* dy, int64_t dy_ld, float* dweights,
                         mx_stream stream) {
    const mx_status bad = check_combine(yt, dt, rows, cols, y_ld, tokens, top_k);
    if (bad != MX_OK) return bad;
    if ((dout_ld && dout_ld < cols) || (dy_ld && dy_ld < cols)) return MX_ERR_SHAPE;
    if (tokens > 0 && (!dout || !slot)) return MX_ERR_NULL;
    if (rows > 0 && (!dy || (dweights && !y))) return MX_ERR_NULL;
    if (!aligned_to(dout, type_bytes(dt)) || !aligned_to(y, type_bytes(yt)) || !aligned_to(dy, type_bytes(yt)) ||
        !aligned_to(slot, 4) || !aligned_to(weights, 4) || !aligned_to(used_rows, 4) || !aligned_to(dweights, 4))
        return MX_ERR_ALIGN;
    CombineBwdArgs a{dout, dout_ld ? dout_ld : cols, y, rows, cols, y_ld ? y_ld : cols, slot, weights, tokens, top_k,
                     used_rows, dy, dy_ld ? dy_ld : cols, dweights};
    const int v = yt == MX_BF16 ? 8 : 4;
    const int64_t clear = used_rows && rows > 0 ? min(rows, (int64_t)1024) : 0;
    if (tokens + clear == 0) return MX_OK;
    // (more than 512 tokens: at most 256 threads a workgroup, so with the clearing ones fewer than 2^32)
    if (tokens >= ((int64_t)1 << 23)) return MX_ERR_SHAPE;
    // as few passes over the columns as the waves allow, and as few waves as these passes need; more waves
    // where there are few tokens (three / six for rows of 2880 bf16: 64 tokens 5.9 / 4.9 us, 256 6.4 / 5.4,
    // 1024 9.3 / 10.3, 16384 141 / 141)
    const int64_t most = tokens <= 512 ? MAX_WAVES : 4;
    const int64_t chunks = ceil_div(cols, 64 * v), waves = ceil_div(chunks, ceil_div(chunks, most));
    const dim3 grid((uint32_t)(tokens + clear)), block((uint32_t)(64 * waves));
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    const bool through = streams(tokens * top_k, cols, yt);
#define MX_COMBINE_BWD(DB, YB)                                                                              \
    do {                                                                                                    \
        if (through) hipLaunchKernelGGL((combine_bwd_kernel<DB, YB, true>), grid, block, 0, s, a);          \
        else hipLaunchKernelGGL((combine_bwd_kernel<DB, YB, false>), grid, block, 0, s, a);                 \
    } while (0)
    if (dt == MX_BF16) {
        if (yt == MX_BF16) MX_COMBINE_BWD(true, true);
        else MX_COMBINE_BWD(true, false);
    } else {
        if (yt == MX_BF16) MX_COMBINE_BWD(false, true);
        else MX_COMBINE_BWD(false, false);
    }
#undef MX_COMBINE_BWD
    return launch_status();
}

}  // extern "C"
