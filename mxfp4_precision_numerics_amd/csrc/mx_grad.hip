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
constexpr int FLIGHT = 2;                   // 16-byte pieces a thread reads at once
constexpr int CHUNK_BYTES = 16 * THREADS * FLIGHT;      // of one tensor, a workgroup's unit of work
constexpr int MAX_PARTIALS = 2048;          // partial sums that a launch leaves
constexpr int64_t MAX_CHUNKS = 1 << 23;     // of a launch (64 GB): its threads fit in 32 bits
constexpr int64_t MAX_ELEMENTS = (int64_t)1 << 37;      // of all tensors
// Launches beyond one for each TABLE tensors: two neighbours hold more than
// MAX_CHUNKS together.
constexpr int MORE_LAUNCHES = (int)(2 * MAX_ELEMENTS * 4 / CHUNK_BYTES / MAX_CHUNKS);
// Partial sums that every workgroup of the scale pass adds up itself, which
// saves a launch while there are not too many workgroups (16 MB: 12.9 us, with
// the launch 14.4; 32 MB: 22.5 both).
constexpr int FEW_PARTIALS = 2 * MAX_PARTIALS;
// Lists larger than this go past the caches: their end would push out what a
// neighbouring kernel left there, and the two passes cannot share it anyway.
// Measured, clipping fp32 into other buffers, cached / past the caches:
// 24.3 / 26.4 us at 32 MB, 43.3 / 41.9 at 64, 81 / 70 at 128, 1655 / 1512 at
// 3185.
constexpr int64_t STREAM_BYTES = 50'000'000;

struct GradTable {
    const void* src[TABLE];
    void* dst[TABLE];
    int64_t numel[TABLE];
    int32_t first[TABLE + 1];               // first chunk of each tensor
    uint32_t bf16[(TABLE + 31) / 32];       // a bit a tensor
    int count;
};

// 16 bytes at any element's address (global memory takes them at any alignment).
typedef unsigned int u32x4v __attribute__((ext_vector_type(4), aligned(2)));

// STREAM: non-temporal, past the caches.
template <bool STREAM>
__device__ __forceinline__ u32x4v load_piece(const void* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load((const u32x4v*)p);
    else return *(const u32x4v*)p;
}
template <bool STREAM>
__device__ __forceinline__ void store_piece(void* p, u32x4v v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, (u32x4v*)p);
    else *(u32x4v*)p = v;
}

// The i-th workgroup's chunk of n: workgroups go to the eight XCDs in turn, and
// each XCD gets a stretch of its own (clipping 3.2 GB: 1504 us without, 1468
// with).
__device__ __forceinline__ int xcd_order(int i, int n) {
    const int per = n / 8;
    return i < per * 8 ? (i & 7) * per + (i >> 3) : i;
}

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

// A chunk's pieces: its place in its tensor.
struct Chunk {
    const char* p;
    char* q;
    int n, whole;             // elements; whole 16-byte pieces
    bool bf;

    __device__ __forceinline__ Chunk(const GradTable& g, int t, int c) {
        bf = (g.bf16[t >> 5] >> (t & 31)) & 1;
        const int size = bf ? 2 : 4, per = CHUNK_BYTES / size;
        const int64_t begin = (int64_t)(c - g.first[t]) * per;
        n = (int)min((int64_t)per, g.numel[t] - begin);
        p = (const char*)g.src[t] + begin * size;
        q = (char*)g.dst[t] + begin * size;
        whole = n * size / 16;
    }
};

template <bool STREAM>
__device__ __forceinline__ void square_chunk(const Chunk& k, double& s) {
    u32x4v w[FLIGHT];
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
        const int i = f * THREADS + (int)threadIdx.x;
        w[f] = (u32x4v){0, 0, 0, 0};
        if (i < k.whole) w[f] = load_piece<STREAM>(k.p + 16 * i);
    }
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
        const uint32_t u[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (k.bf) {
                add_square(s, bf16lo(u[m]));
                add_square(s, bf16hi(u[m]));
            } else {
                add_square(s, __uint_as_float(u[m]));
            }
        }
    }
    for (int i = k.whole * (k.bf ? 8 : 4) + (int)threadIdx.x; i < k.n; i += THREADS)
        add_square(s, k.bf ? __uint_as_float((uint32_t)((const uint16_t*)k.p)[i] << 16) : ((const float*)k.p)[i]);
}

// Bound by memory: 3.2 GB of fp32 in 455-475 us, 6.7-7.0 TB/s.
template <bool STREAM>
__global__ __launch_bounds__(THREADS) void square_kernel(GradTable g, int chunks, double* partials) {
    double s = 0.0;
    for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
        const int c = xcd_order(i, chunks);
        square_chunk<STREAM>(Chunk(g, tensor_of(g, c), c), s);
    }
    s = block_sum<THREADS>(s);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ __forceinline__ double sum_partials(const double* partials, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) s += partials[i];
    return block_sum<THREADS>(s);
}

// The whole sum into partials[n] (when it is asked for), the norm from it.
__global__ __launch_bounds__(THREADS) void norm_kernel(double* partials, int n, float* norm, bool keep) {
    const double s = sum_partials(partials, n);
    if (threadIdx.x == 0) {
        *norm = (float)sqrt(s);
        if (keep) partials[n] = s;
    }
}

template <bool STREAM>
__device__ __forceinline__ void scale_chunk(const Chunk& k, float coef) {
    u32x4v w[FLIGHT];
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
        const int i = f * THREADS + (int)threadIdx.x;
        if (i < k.whole) w[f] = load_piece<STREAM>(k.p + 16 * i);
    }
#pragma unroll
    for (int f = 0; f < FLIGHT; ++f) {
        const int i = f * THREADS + (int)threadIdx.x;
        if (i >= k.whole) continue;
        uint32_t u[4] = {w[f].x, w[f].y, w[f].z, w[f].w};
#pragma unroll
        for (int m = 0; m < 4; ++m)
            u[m] = k.bf ? f32_to_bf16_rne(coef * bf16lo(u[m])) | f32_to_bf16_rne(coef * bf16hi(u[m])) << 16
                        : __float_as_uint(coef * __uint_as_float(u[m]));
        store_piece<STREAM>(k.q + 16 * i, (u32x4v){u[0], u[1], u[2], u[3]});
    }
    for (int i = k.whole * (k.bf ? 8 : 4) + (int)threadIdx.x; i < k.n; i += THREADS) {
        if (k.bf)
            ((uint16_t*)k.q)[i] =
                (uint16_t)f32_to_bf16_rne(coef * __uint_as_float((uint32_t)((const uint16_t*)k.p)[i] << 16));
        else
            ((float*)k.q)[i] = coef * ((const float*)k.p)[i];
    }
}

// Bound by memory: 3.2 GB of fp32 into another 3.2 GB in 1000-1015 us, 6.3
// TB/s.
// One workgroup a chunk: 8 KB each way.  Fewer workgroups that go on to
// further chunks were slower (both passes of that size 1854 us with 1024 of
// them, 1671 with 4096, 1525 so), and so were chunks of 4 KB (1787) or 16 KB
// (1559).
template <bool STREAM>
__global__ __launch_bounds__(THREADS) void scale_kernel(GradTable g, const double* partials, int n,
                                                        float max_norm, float* norm) {
    const double total = sqrt(sum_partials(partials, n));
    const float seen = (float)total;        // the norm that the caller gets
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = seen;
    const double ratio = (double)max_norm / (total + 1e-6);
    // a norm that is not finite in fp32 leaves the gradients as they are
    const float coef = seen - seen == 0.0f && ratio < 1.0 ? (float)ratio : 1.0f;
    const int c = xcd_order(blockIdx.x, gridDim.x), t = tensor_of(g, c);
    if (coef == 1.0f && g.src[t] == g.dst[t]) return;
    scale_chunk<STREAM>(Chunk(g, t, c), coef);
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
        if (numels[i] < 0 || numels[i] > MAX_ELEMENTS - total || chunks_of(types[i], numels[i]) > MAX_CHUNKS)
            return MX_ERR_SHAPE;
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
        const int64_t more = chunks_of(types[at], numels[at]);
        if (chunks + more > MAX_CHUNKS) break;
        const int i = g.count++;
        g.src[i] = grads[at];
        g.dst[i] = outs ? outs[at] : const_cast<void*>(grads[at]);
        g.numel[i] = numels[at];
        g.first[i] = (int32_t)chunks;
        if (types[at] == MX_BF16) g.bf16[i >> 5] |= 1u << (i & 31);
        chunks += more;
    }
    g.first[g.count] = (int32_t)chunks;
    return (int)chunks;
}

bool large(const mx_dtype* types, const int64_t* numels, int32_t count) {
    int64_t bytes = 0;
    for (int i = 0; i < count; ++i) bytes += numels[i] * (int64_t)type_bytes(types[i]);
    return bytes > STREAM_BYTES;
}

// The norm pass; returns how many partial sums it leaves.
int launch_squares(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                   double* partials, bool past, hipStream_t s) {
    GradTable g;
    int n = 0;
    for (int32_t at = 0; at < count;) {
        const int chunks = fill_table(g, at, grads, types, numels, count, nullptr);
        if (!chunks) continue;
        const int grid = min(chunks, MAX_PARTIALS);
        if (past) hipLaunchKernelGGL(square_kernel<true>, dim3(grid), dim3(THREADS), 0, s, g, chunks, partials + n);
        else hipLaunchKernelGGL(square_kernel<false>, dim3(grid), dim3(THREADS), 0, s, g, chunks, partials + n);
        n += grid;
    }
    return n;
}

}  // namespace

extern "C" {

int64_t mx_grad_workspace(int32_t count) {
    return count <= 0 ? 0 : ((ceil_div(count, TABLE) + MORE_LAUNCHES) * MAX_PARTIALS + 1) * (int64_t)sizeof(double);
}

mx_status mx_grad_norm(const void* const* grads, const mx_dtype* types, const int64_t* numels, int32_t count,
                       double* workspace, float* norm, mx_stream stream) {
    const mx_status bad = check_grads(grads, types, numels, count, nullptr);
    if (bad != MX_OK) return bad;
    if (!norm || (count > 0 && !workspace)) return MX_ERR_NULL;
    if (!aligned_to(norm, 4) || !aligned_to(workspace, 8)) return MX_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    const int n = launch_squares(grads, types, numels, count, workspace, large(types, numels, count), s);
    hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(THREADS), 0, s, workspace, n, norm, false);
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
    const bool past = large(types, numels, count);
    const int n = launch_squares(grads, types, numels, count, workspace, past, s);
    const double* sums = workspace;
    float* out = norm;
    int many = n;
    if (n == 0 || past || n > FEW_PARTIALS) {
        hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(THREADS), 0, s, workspace, n, norm, n > 0);
        sums = workspace + n;
        many = 1;
        out = nullptr;
    }
    GradTable g;
    for (int32_t at = 0; at < count;) {
        const int chunks = fill_table(g, at, grads, types, numels, count, outs);
        if (!chunks) continue;
        if (past)
            hipLaunchKernelGGL(scale_kernel<true>, dim3(chunks), dim3(THREADS), 0, s, g, sums, many, max_norm, out);
        else
            hipLaunchKernelGGL(scale_kernel<false>, dim3(chunks), dim3(THREADS), 0, s, g, sums, many, max_norm, out);
        out = nullptr;      // the first launch writes it
    }
    return launch_status();
}

}  // extern "C"
