// mx_grad.hip -- the L2 norm over many gradient tensors, and clipping by it
// (gfx950).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_device.h"
#include "mx_host.h"

namespace {

using namespace mx;

// Tensors of one launch: their table travels in the kernel's arguments (no
// copy to the device, nothing kept between calls).
constexpr int TABLE = 96;
constexpr int THREADS = 256;
constexpr int FLIGHT = 4;                   // 16-byte pieces a thread reads at once
constexpr int CHUNK_BYTES = 16 * THREADS * FLIGHT;      // of one tensor, a workgroup's unit of work
constexpr int MAX_PARTIALS = 2048;          // workgroups of a launch

struct GradTable {
    const void* src[TABLE];
    void* dst[TABLE];
    int64_t numel[TABLE];
    int32_t first[TABLE + 1];               // first chunk of each tensor
    uint32_t bf16[(TABLE + 31) / 32];       // a bit a tensor
    int count;
};

__device__ __forceinline__ int tensor_of(const GradTable& g, int chunk) {
    int lo = 0, hi = g.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Squares are summed in fp64: none over- or underflows, and a sum over any
// number of elements is good to fp32's last place.
__device__ __forceinline__ void add_square(double& s, float x) {
    const double d = (double)x;
    s = __builtin_fma(d, d, s);
}

// The sum over a workgroup in a fixed order; every thread gets it.
template <int N>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[N / 64];
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < N / 64; ++i) v += part[i];
    return v;
}

__global__ __launch_bounds__(THREADS) void square_kernel(GradTable g, int chunks, double* partials) {
    double s = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(g, c);
        const bool bf = (g.bf16[t >> 5] >> (t & 31)) & 1;
        const int64_t per = CHUNK_BYTES / (bf ? 2 : 4);
        const int64_t begin = (int64_t)(c - g.first[t]) * per, n = min(per, g.numel[t] - begin);
        const int v = bf ? 8 : 4;
        const char* p = (const char*)g.src[t] + begin * (bf ? 2 : 4);
        const int whole = ((uintptr_t)p & 15) ? 0 : (int)(n / v);
        uint4 w[FLIGHT];
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            const int i = k * THREADS + (int)threadIdx.x;
            w[k] = i < whole ? ((const uint4*)p)[i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (bf) {
                    add_square(s, bf16lo(u[m]));
                    add_square(s, bf16hi(u[m]));
                } else {
                    add_square(s, __uint_as_float(u[m]));
                }
            }
        }
        for (int64_t i = (int64_t)whole * v + threadIdx.x; i < n; i += THREADS)
            add_square(s, bf ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i]);
    }
    s = block_sum<THREADS>(s);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ __forceinline__ double sum_partials(const double* partials, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) s += partials[i];
    return block_sum<THREADS>(s);
}

__global__ __launch_bounds__(THREADS) void norm_kernel(const double* partials, int n, float* norm) {
    const double s = sum_partials(partials, n);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ __launch_bounds__(THREADS) void scale_kernel(GradTable g, int chunks, const double* partials, int n,
                                                        float max_norm, float* norm) {
    const double total = sqrt(sum_partials(partials, n));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const double ratio = (double)max_norm / (total + 1e-6);
    // a norm that is not finite leaves the gradients as they are
    const float coef = total - total == 0.0 && ratio < 1.0 ? (float)ratio : 1.0f;
    // from the end back: what the norm pass read last is still in the cache
    for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const int t = tensor_of(g, c);
        if (coef == 1.0f && g.src[t] == g.dst[t]) continue;
        const bool bf = (g.bf16[t >> 5] >> (t & 31)) & 1;
        const int size = bf ? 2 : 4;
        const int64_t per = CHUNK_BYTES / size;
        const int64_t begin = (int64_t)(c - g.first[t]) * per, n_el = min(per, g.numel[t] - begin);
        const int v = bf ? 8 : 4;
        const char* p = (const char*)g.src[t] + begin * size;
        char* q = (char*)g.dst[t] + begin * size;
        const int whole = (((uintptr_t)p | (uintptr_t)q) & 15) ? 0 : (int)(n_el / v);
        uint4 w[FLIGHT];
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            const int i = k * THREADS + (int)threadIdx.x;
            if (i < whole) w[k] = ((const uint4*)p)[i];
        }
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            const int i = k * THREADS + (int)threadIdx.x;
            if (i >= whole) continue;
            uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
                u[m] = bf ? f32_to_bf16_rne(coef * bf16lo(u[m])) | f32_to_bf16_rne(coef * bf16hi(u[m])) << 16
                          : __float_as_uint(coef * __uint_as_float(u[m]));
            ((uint4*)q)[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        for (int64_t i = (int64_t)whole * v + threadIdx.x; i < n_el; i += THREADS) {
            if (bf) ((uint16_t*)q)[i] = (uint16_t)f32_to_bf16_rne(coef * __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16));
            else ((float*)q)[i] = coef * ((const float*)p)[i];
        }
    }
}

int64_t chunks_of(mx_dtype t, int64_t numel) { return ceil_div(numel * (int64_t)type_bytes(t), CHUNK_BYTES); }

mx_status check_grads(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                      void* const* outs) {
    if (count < 0) return MX_ERR_SHAPE;
    if (count == 0) return MX_OK;
    if (!grads || !types || !numels) return MX_ERR_NULL;
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        if (types[i] != MX_F32 && types[i] != MX_BF16) return MX_ERR_DTYPE;
        // at most 2^40 elements in all: a launch's chunks then fit in 32 bits
        if (numels[i] < 0 || numels[i] > ((int64_t)1 << 40) - total) return MX_ERR_SHAPE;
        total += numels[i];
        if (numels[i] == 0) continue;
        if (!grads[i] || (outs && !outs[i])) return MX_ERR_NULL;
        if (!aligned_to(grads[i], type_bytes(types[i])) || (outs && !aligned_to(outs[i], type_bytes(types[i]))))
            return MX_ERR_ALIGN;
    }
    return MX_OK;
}

// Fills the table with the next tensors of the list from `at` on (empty ones
// left out); returns its chunks.
int fill_table(GradTable& g, int32_t& at, const void* const* grads, const mx_dtype* types, const int64_t* numels,
               int32_t count, void* const* outs) {
    int64_t chunks = 0;
    g.count = 0;
    for (uint32_t& b : g.bf16) b = 0;
    for (; at < count && g.count < TABLE; ++at) {
        if (numels[at] == 0) continue;
        const int i = g.count++;
        g.src[i] = grads[at];
        g.dst[i] = outs ? outs[at] : const_cast<void*>(grads[at]);
        g.numel[i] = numels[at];
        g.first[i] = (int32_t)chunks;
        if (types[at] == MX_BF16) g.bf16[i >> 5] |= 1u << (i & 31);
        chunks += chunks_of(types[at], numels[at]);
    }
    g.first[g.count] = (int32_t)chunks;
    return (int)chunks;
}

// The norm pass; returns how many partial sums it leaves.
int launch_squares(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                   double* partials, hipStream_t s) {
    GradTable g;
    int n = 0;
    for (int32_t at = 0; at < count;) {
        const int chunks = fill_table(g, at, grads, types, numels, count, nullptr);
        if (!chunks) continue;
        const int grid = min(chunks, MAX_PARTIALS);
        hipLaunchKernelGGL(square_kernel, dim3(grid), dim3(THREADS), 0, s, g, chunks, partials + n);
        n += grid;
    }
    return n;
}

}  // namespace

extern "C" {

int64_t mx_grad_workspace(int32_t count) {
    return count <= 0 ? 0 : ceil_div(count, TABLE) * MAX_PARTIALS * (int64_t)sizeof(double);
}

mx_status mx_grad_norm(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                       double* workspace, float* norm, mx_stream stream) {
    const mx_status bad = check_grads(grads, types, numels, count, nullptr);
    if (bad != MX_OK) return bad;
    if (!norm || (count > 0 && !workspace)) return MX_ERR_NULL;
    if (!aligned_to(norm, 4) || !aligned_to(workspace, 8)) return MX_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    const int n = launch_squares(grads, types, numels, count, workspace, s);
    hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(THREADS), 0, s, workspace, n, norm);
    return launch_status();
}

mx_status mx_grad_clip(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                       void* const* outs, float max_norm, double* workspace, float* norm, mx_stream stream) {
    const mx_status bad = check_grads(grads, types, numels, count, outs);
    if (bad != MX_OK) return bad;
    if (!(max_norm >= 0.0f)) return MX_ERR_SHAPE;
    if (!norm || (count > 0 && !workspace)) return MX_ERR_NULL;
    if (!aligned_to(norm, 4) || !aligned_to(workspace, 8)) return MX_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    const int n = launch_squares(grads, types, numels, count, workspace, s);
    if (n == 0) {
        hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(THREADS), 0, s, workspace, n, norm);
        return launch_status();
    }
    GradTable g;
    float* out = norm;
    for (int32_t at = 0; at < count;) {
        const int chunks = fill_table(g, at, grads, types, numels, count, outs);
        if (!chunks) continue;
        const int grid = min(chunks, MAX_PARTIALS);
        hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(THREADS), 0, s, g, chunks, workspace, n, max_norm, out);
        out = nullptr;      // the first launch writes it
    }
    return launch_status();
}

}  // extern "C"
