// mx_cache.hip -- writing keys and values into the MXFP4 cache, and reading
// them back (gfx950).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_cache.h"
#include "mx_device.h"
#include "mx_host.h"

namespace {

using namespace mx;

// Pieces of 16 bytes at any element's address (global memory takes them at any
// alignment).
typedef unsigned int u32x4v __attribute__((ext_vector_type(4), aligned(2)));

struct Rows {                 // [tokens][heads][dim] at any pitches
    void* p[2];               // keys, values
    int64_t ld[2], head_ld[2];
};

struct CacheArgs {
    CacheView cache;
    Rows rows;
    const int32_t* slots;
    int64_t pieces;           // of eight elements: tokens * heads * dim / 8
};

// Where piece i lies: its token, head and first element.
struct Place {
    int64_t token;
    int head, at;
    __device__ __forceinline__ Place(const CacheArgs& a, int64_t i) {
        const int per = a.cache.dim >> 3;
        const int64_t row = i / per;
        at = (int)(i - row * per) * 8;
        token = row / a.cache.heads;
        head = (int)(row - token * a.cache.heads);
    }
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* f) {
    if constexpr (BF16) {
        const u32x4v w = *(const u32x4v*)((const uint16_t*)p + at);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { f[2 * i] = bf16lo(u[i]); f[2 * i + 1] = bf16hi(u[i]); }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4v w = *(const u32x4v*)((const float*)p + at + 4 * i);
            f[4 * i] = __uint_as_float(w.x);
            f[4 * i + 1] = __uint_as_float(w.y);
            f[4 * i + 2] = __uint_as_float(w.z);
            f[4 * i + 3] = __uint_as_float(w.w);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* f) {
    if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16_rne(f[2 * i]) | f32_to_bf16_rne(f[2 * i + 1]) << 16;
        *(u32x4v*)((uint16_t*)p + at) = (u32x4v){u[0], u[1], u[2], u[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *(u32x4v*)((float*)p + at + 4 * i) =
                (u32x4v){__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                         __float_as_uint(f[4 * i + 3])};
    }
}

__device__ __forceinline__ void flip_signs(float* f, uint32_t mask, int q) {
    const uint32_t m = mask >> (8 * q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(__float_as_uint(f[i]) ^ (m >> i << 31));
}

// A thread: eight elements of a token's keys (blockIdx.y = 0) or values (1); a
// block of 32 is a quad of lanes.
template <bool BF16>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.pieces) return;                             // (whole quads: pieces % 4 == 0)
    const Place p(a, i);
    const int64_t slot = a.slots[p.token];
    if (slot < 0 || slot >= (a.cache.pages << a.cache.page_log2)) return;
    const int which = blockIdx.y, q = threadIdx.x & 3;
    float f[8];
    load8<BF16>(a.rows.p[which], p.token * a.rows.ld[which] + p.head * a.rows.head_ld[which] + p.at, f);
    if (a.cache.rht) {
        flip_signs(f, a.cache.mask, q);
        rht32_quad(f, q);
    }
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    const uint32_t byte = scale_byte_from_amax_bits(quad_max_u(most));
    uint32_t codes = cvt8_rne(f, scale_operand(byte));
    if (byte == 0xFFu) codes = 0;                          // non-finite block: codes are 0
    const int64_t page = slot >> a.cache.page_log2;
    const int offset = (int)(slot & ((1 << a.cache.page_log2) - 1));
    *(uint32_t*)(a.cache.codes[which] + a.cache.codes_at(page, p.head, offset) + (p.at >> 1)) = codes;
    if (q == 0)
        a.cache.scales[which][a.cache.scales_at(page, p.head, offset) + ((int64_t)(p.at >> 5) << a.cache.page_log2)] =
            (uint8_t)byte;
}

template <bool BF16>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int which = a.rows.p[0] ? blockIdx.y : 1;
    if (i >= a.pieces) return;
    const Place p(a, i);
    const int64_t slot = a.slots[p.token];
    float f[8] = {};
    if (slot >= 0 && slot < (a.cache.pages << a.cache.page_log2)) {
        const int64_t page = slot >> a.cache.page_log2;
        const int offset = (int)(slot & ((1 << a.cache.page_log2) - 1)), q = threadIdx.x & 3;
        const uint32_t codes =
            *(const uint32_t*)(a.cache.codes[which] + a.cache.codes_at(page, p.head, offset) + (p.at >> 1));
        const uint32_t byte = a.cache.scales[which][a.cache.scales_at(page, p.head, offset) +
                                                    ((int64_t)(p.at >> 5) << a.cache.page_log2)];
        decode8(codes, scale_operand(byte), f);
        if (byte == 0xFFu) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(0x7FC00000u);
        }
        if (a.cache.rht) {
            rht32_quad(f, q);
            flip_signs(f, a.cache.mask, q);
        }
    }
    store8<BF16>(a.rows.p[which], p.token * a.rows.ld[which] + p.head * a.rows.head_ld[which] + p.at, f);
}

mx_status check_rows(const CacheView& c, mx_dtype t, int64_t tokens, int64_t ld, int64_t head_ld) {
    if (t != MX_F32 && t != MX_BF16) return MX_ERR_DTYPE;
    if (tokens < 0 || tokens > ((int64_t)1 << 33) / ((int64_t)c.heads * c.dim)) return MX_ERR_SHAPE;
    if (ld < 0 || head_ld < 0 || (head_ld && head_ld < c.dim) || (ld && ld < c.dim)) return MX_ERR_SHAPE;
    return MX_OK;
}

CacheArgs cache_args(const CacheView& c, void* k, int64_t k_ld, int64_t k_head_ld, void* v, int64_t v_ld,
                     int64_t v_head_ld, int64_t tokens, const int32_t* slots) {
    const int64_t row = (int64_t)c.heads * c.dim;
    return CacheArgs{c,
                     {{k, v}, {k_ld ? k_ld : row, v_ld ? v_ld : row}, {k_head_ld ? k_head_ld : c.dim, v_head_ld ? v_head_ld : c.dim}},
                     slots, tokens * row / 8};
}

}  // namespace

extern "C" {

mx_status mx_cache_write(const mx_cache* cache, const void* k, int64_t k_ld, int64_t k_head_ld, const void* v,
                         int64_t v_ld, int64_t v_head_ld, mx_dtype t, int64_t tokens, const int32_t* slots,
                         mx_stream stream) {
    CacheView c;
    mx_status bad = view_cache(cache, c);
    if (bad == MX_OK) bad = check_rows(c, t, tokens, k_ld, k_head_ld);
    if (bad == MX_OK) bad = check_rows(c, t, tokens, v_ld, v_head_ld);
    if (bad != MX_OK) return bad;
    if (tokens == 0) return MX_OK;
    if (!k || !v || !slots) return MX_ERR_NULL;
    if (!aligned_to(k, type_bytes(t)) || !aligned_to(v, type_bytes(t)) || !aligned_to(slots, 4)) return MX_ERR_ALIGN;
    const CacheArgs a = cache_args(c, const_cast<void*>(k), k_ld, k_head_ld, const_cast<void*>(v), v_ld, v_head_ld,
                                   tokens, slots);
    const dim3 grid((uint32_t)ceil_div(a.pieces, 256), 2);
    (void)hipGetLastError();
    if (t == MX_BF16) hipLaunchKernelGGL(cache_write_kernel<true>, grid, dim3(256), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL(cache_write_kernel<false>, grid, dim3(256), 0, (hipStream_t)stream, a);
    return launch_status();
}

mx_status mx_cache_read(const mx_cache* cache, void* k, int64_t k_ld, int64_t k_head_ld, void* v, int64_t v_ld,
                        int64_t v_head_ld, mx_dtype t, int64_t tokens, const int32_t* slots, mx_stream stream) {
    CacheView c;
    mx_status bad = view_cache(cache, c);
    if (bad == MX_OK) bad = check_rows(c, t, tokens, k_ld, k_head_ld);
    if (bad == MX_OK) bad = check_rows(c, t, tokens, v_ld, v_head_ld);
    if (bad != MX_OK) return bad;
    if (tokens == 0 || (!k && !v)) return MX_OK;
    if (!slots) return MX_ERR_NULL;
    if (!aligned_to(k, type_bytes(t)) || !aligned_to(v, type_bytes(t)) || !aligned_to(slots, 4)) return MX_ERR_ALIGN;
    const CacheArgs a = cache_args(c, k, k_ld, k_head_ld, v, v_ld, v_head_ld, tokens, slots);
    const dim3 grid((uint32_t)ceil_div(a.pieces, 256), k && v ? 2 : 1);
    (void)hipGetLastError();
    if (t == MX_BF16) hipLaunchKernelGGL(cache_read_kernel<true>, grid, dim3(256), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL(cache_read_kernel<false>, grid, dim3(256), 0, (hipStream_t)stream, a);
    return launch_status();
}

}  // extern "C"
