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
    int chunks;               // waves that share a row
};

// V consecutive elements of a row as fp32.  VEC: one aligned load (16 bytes
// at the most); otherwise element by element, those past the end 0.
template <bool BF16, int V, bool VEC>
__device__ __forceinline__ void load_v(const void* p, int64_t at, int64_t left, float* f) {
    if constexpr (VEC) {
        if constexpr (BF16 && V == 8) {
            const uint4 w = *(const uint4*)((const uint16_t*)p + at);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16lo(u[i]);
                f[2 * i + 1] = bf16hi(u[i]);
            }
        } else if constexpr (BF16) {
            const uint2 w = *(const uint2*)((const uint16_t*)p + at);
            f[0] = bf16lo(w.x); f[1] = bf16hi(w.x);
            f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 w = *(const float4*)((const float*)p + at + i);
                f[i] = w.x; f[i + 1] = w.y; f[i + 2] = w.z; f[i + 3] = w.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = 0.0f;
            if (i < left)
                f[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[at + i] << 16) : ((const float*)p)[at + i];
        }
    }
}

template <bool BF16, int V, bool VEC>
__device__ __forceinline__ void store_v(void* p, int64_t at, int64_t left, const float* f) {
    if constexpr (VEC) {
        if constexpr (BF16) {
            uint32_t u[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) u[i] = f32_to_bf16_rne(f[2 * i]) | f32_to_bf16_rne(f[2 * i + 1]) << 16;
            if constexpr (V == 8) *(uint4*)((uint16_t*)p + at) = make_uint4(u[0], u[1], u[2], u[3]);
            else *(uint2*)((uint16_t*)p + at) = make_uint2(u[0], u[1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *(float4*)((float*)p + at + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= left) continue;
            if constexpr (BF16) ((uint16_t*)p)[at + i] = (uint16_t)f32_to_bf16_rne(f[i]);
            else ((float*)p)[at + i] = f[i];
        }
    }
}

// One wave: 64 V columns of one token.
template <bool YB, bool OB, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    constexpr int V = YB ? 8 : 4;
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = w / a.chunks;
    const int64_t col = (w % a.chunks * 64 + (threadIdx.x & 63)) * V;
    if (t >= a.tokens || col >= a.cols) return;
    const int64_t left = a.cols - col;
    float acc[V];
    if (a.residual) {
        load_v<OB, V, VEC>(a.residual, t * a.res_ld + col, left, acc);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    }
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t s = a.slot[t * a.top_k + j];
        if (s < 0 || s >= a.rows) continue;
        const float wt = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
        float f[V];
        load_v<YB, V, VEC>(a.y, s * a.y_ld + col, left, f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(wt, f[i], acc[i]);
    }
    store_v<OB, V, VEC>(a.out, t * a.out_ld + col, left, acc);
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

// One workgroup of two waves: one token.  Beyond the tokens the workgroups
// clear the rows of dy past the used ones.
constexpr int BWD_THREADS = 128;

template <bool DB, bool YB, bool VEC>
__global__ __launch_bounds__(BWD_THREADS) void combine_bwd_kernel(CombineBwdArgs a) {
    constexpr int V = YB ? 8 : 4;
    __shared__ float part[BWD_THREADS / 64];
    const int tid = threadIdx.x;
    const int64_t used = a.used_rows ? min(max((int64_t)*a.used_rows, (int64_t)0), a.rows) : a.rows;
    if ((int64_t)blockIdx.x >= a.tokens) {
        const float zero[V] = {};
        for (int64_t r = used + blockIdx.x - a.tokens; r < a.rows; r += gridDim.x - a.tokens)
            for (int64_t col = tid * V; col < a.cols; col += BWD_THREADS * V)
                store_v<YB, V, VEC>(a.dy, r * a.dy_ld + col, a.cols - col, zero);
        return;
    }
    const int64_t t = blockIdx.x;
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t s = a.slot[t * a.top_k + j];
        const bool there = s >= 0 && s < used;
        float dot = 0.0f;
        if (there) {
            const float wt = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
            for (int64_t col = tid * V; col < a.cols; col += BWD_THREADS * V) {
                const int64_t left = a.cols - col;
                float g[V], f[V];
                load_v<DB, V, VEC>(a.dout, t * a.dout_ld + col, left, g);
                if (a.dweights) {
                    load_v<YB, V, VEC>(a.y, s * a.y_ld + col, left, f);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot = __builtin_fmaf(g[i], f[i], dot);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = wt * g[i];
                store_v<YB, V, VEC>(a.dy, s * a.dy_ld + col, left, f);
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
        __syncthreads();
        if ((tid & 63) == 0) part[tid >> 6] = dot;
        __syncthreads();
        if (tid == 0) a.dweights[t * a.top_k + j] = there ? part[0] + part[1] : 0.0f;
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

// Rows that start at whole 16-byte (or, for the narrower of two types, 8-byte)
// pieces and hold a whole number of them.
bool vector_rows(const void* p, mx_dtype t, int64_t ld, int v) {
    return ld % v == 0 && aligned_to(p, v * type_bytes(t));
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
    if (cols > (int64_t)INT32_MAX * 64) return MX_ERR_SHAPE;
    a.chunks = (int)ceil_div(cols, 64 * v);
    const int64_t blocks = ceil_div(tokens * a.chunks, 4);
    if (blocks > ((int64_t)1 << 24) - 1) return MX_ERR_SHAPE;
    const bool vec = cols % v == 0 && vector_rows(y, yt, a.y_ld, v) && vector_rows(out, ot, a.out_ld, v) &&
                     (!residual || vector_rows(residual, ot, a.res_ld, v));
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
#define MX_COMBINE(YB, OB)                                                                                    \
    do {                                                                                                      \
        if (vec) hipLaunchKernelGGL((combine_kernel<YB, OB, true>), dim3((uint32_t)blocks), dim3(256), 0, s, a);   \
        else hipLaunchKernelGGL((combine_kernel<YB, OB, false>), dim3((uint32_t)blocks), dim3(256), 0, s, a);      \
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
    if (tokens + clear > ((int64_t)1 << 24)) return MX_ERR_SHAPE;
    const bool vec = cols % v == 0 && vector_rows(dout, dt, a.dout_ld, v) && vector_rows(dy, yt, a.dy_ld, v) &&
                     (!dweights || vector_rows(y, yt, a.y_ld, v));
    const dim3 grid((uint32_t)(tokens + clear));
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
#define MX_COMBINE_BWD(DB, YB)                                                                                  \
    do {                                                                                                        \
        if (vec) hipLaunchKernelGGL((combine_bwd_kernel<DB, YB, true>), grid, dim3(BWD_THREADS), 0, s, a);      \
        else hipLaunchKernelGGL((combine_bwd_kernel<DB, YB, false>), grid, dim3(BWD_THREADS), 0, s, a);         \
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
