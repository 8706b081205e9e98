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
    int64_t tokens;
    int lanes;                // of a row: dim / 8
    int per;                  // tokens of a workgroup: 256 / lanes
};

// What a thread handles: eight elements of one token's row of one head; four
// lanes hold a block of 32, the lanes after them the token's next blocks, then
// the head's next token, so that a wave writes consecutive tokens of a page:
// whole lines of codes, neighbouring scale bytes.
struct Piece {
    int64_t token, slot;      // slot -1: outside the cache, or no such token
    int at;                   // first element
    bool live;                // there is such a token

    __device__ __forceinline__ Piece(const CacheArgs& a, int64_t first) {
        const int t = (int)threadIdx.x / a.lanes;
        at = ((int)threadIdx.x - t * a.lanes) * 8;
        token = first + t;
        live = t < a.per && token < a.tokens;
        slot = live ? a.slots[token] : -1;
        if (slot >= a.cache.pages << a.cache.page_log2) slot = -1;
    }
    __device__ __forceinline__ int64_t page(const CacheArgs& a) const { return slot >> a.cache.page_log2; }
    __device__ __forceinline__ int offset(const CacheArgs& a) const { return (int)slot & ((1 << a.cache.page_log2) - 1); }
    __device__ __forceinline__ int64_t row(const CacheArgs& a, int which, int head) const {
        return token * a.rows.ld[which] + head * a.rows.head_ld[which] + at;
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

// Past the caches: what is read back is far more than they would keep of it.
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* f) {
    if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16_rne(f[2 * i]) | f32_to_bf16_rne(f[2 * i + 1]) << 16;
        __builtin_nontemporal_store((u32x4v){u[0], u[1], u[2], u[3]}, (u32x4v*)((uint16_t*)p + at));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_nontemporal_store((u32x4v){__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                                 __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])},
                                        (u32x4v*)((float*)p + at + 4 * i));
    }
}

__device__ __forceinline__ void flip_signs(float* f, uint32_t mask, int q) {
    const uint32_t m = mask >> (8 * q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(__float_as_uint(f[i]) ^ (m >> i << 31));
}

// The quantizer's rule on 32 elements, four lanes a block; the loads of keys and
// values are under way together.  16384 tokens of 8 heads of 128, bf16,
// transformed: 19.0 us, 4.5 TB/s of HBM traffic (read 66 MB, written 18); its grid
// comes and goes in a few microseconds of that.  (Eight such batches in turn: 22.2 us each,
// 25 with two tokens a thread, whose loads are under way together; 4096 tokens 7.8
// and 9.2.)
template <bool BF16>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs a) {
    const int head = blockIdx.y, q = threadIdx.x & 3;
    const Piece p(a, (int64_t)blockIdx.x * a.per);
    if (p.slot < 0) return;                                // (the four lanes of a block together)
    float f[2][8];
#pragma unroll
    for (int which = 0; which < 2; ++which) load8<BF16>(a.rows.p[which], p.row(a, which, head), f[which]);
    const int64_t codes_at = a.cache.codes_at(p.page(a), head, p.offset(a)) + (p.at >> 1);
    const int64_t scale_at =
        a.cache.scales_at(p.page(a), head, p.offset(a)) + ((int64_t)(p.at >> 5) << a.cache.page_log2);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* v = f[which];
        if (a.cache.rht) {
            flip_signs(v, a.cache.mask, q);
            rht32_quad(v, q);
        }
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        const uint32_t byte = scale_byte_from_amax_bits(quad_max_u(most));
        uint32_t codes = cvt8_rne(v, scale_operand(byte));
        if (byte == 0xFFu) codes = 0;                      // non-finite block: codes are 0
        *(uint32_t*)(a.cache.codes[which] + codes_at) = codes;
        if (q == 0) a.cache.scales[which][scale_at] = (uint8_t)byte;
    }
}

// The same way back (the same tokens: 22.9 us, 3.8 TB/s).
template <bool BF16>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs a) {
    const int head = blockIdx.y, q = threadIdx.x & 3;
    const Piece p(a, (int64_t)blockIdx.x * a.per);
    if (!p.live) return;
    uint32_t codes[2] = {0, 0}, byte[2] = {0, 0};
    if (p.slot >= 0) {
        const int64_t codes_at = a.cache.codes_at(p.page(a), head, p.offset(a)) + (p.at >> 1);
        const int64_t scale_at =
            a.cache.scales_at(p.page(a), head, p.offset(a)) + ((int64_t)(p.at >> 5) << a.cache.page_log2);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            codes[which] = *(const uint32_t*)(a.cache.codes[which] + codes_at);
            byte[which] = a.cache.scales[which][scale_at];
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!a.rows.p[which]) continue;
        float f[8] = {};
        if (p.slot >= 0) {
            decode8(codes[which], scale_operand(byte[which]), f);
            if (byte[which] == 0xFFu) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(0x7FC00000u);
            }
            if (a.cache.rht) {
                rht32_quad(f, q);
                flip_signs(f, a.cache.mask, q);
            }
        }
        store8<BF16>(a.rows.p[which], p.row(a, which, head), f);
    }
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
                     slots, tokens, c.dim / 8, 256 / (c.dim / 8)};
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
    const dim3 grid((uint32_t)ceil_div(tokens, a.per), c.heads);
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (t == MX_BF16) hipLaunchKernelGGL(cache_write_kernel<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(cache_write_kernel<false>, grid, dim3(256), 0, s, a);
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
    const dim3 grid((uint32_t)ceil_div(tokens, a.per), c.heads);
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (t == MX_BF16) hipLaunchKernelGGL(cache_read_kernel<true>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(cache_read_kernel<false>, grid, dim3(256), 0, s, a);
    return launch_status();
}

}  // extern "C"
