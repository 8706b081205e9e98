// mx_cache.h -- the key/value cache as the kernels see it, and the host checks
// of its description (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_host.h"

namespace mx {

struct CacheView {
    uint8_t* codes[2];        // keys, values
    uint8_t* scales[2];
    int64_t pages;
    int heads, page_log2, dim, rht;
    uint32_t mask;            // of the RHT's signs, 0 without

    // A token's codes (dim / 2 bytes), and its scale of block 0 (block b's is
    // b << page_log2 bytes further).
    __device__ __forceinline__ int64_t codes_at(int64_t page, int head, int offset) const {
        return (((page * heads + head) << page_log2) + offset) * (dim >> 1);
    }
    __device__ __forceinline__ int64_t scales_at(int64_t page, int head, int offset) const {
        return (((page * heads + head) * (dim >> 5)) << page_log2) + offset;
    }
};

inline mx_status view_cache(const mx_cache* c, CacheView& v) {
    if (!c) return MX_ERR_NULL;
    if (c->heads < 1 || c->heads > 1024 || c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32) return MX_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1))) return MX_ERR_SHAPE;
    if (c->pages < 0 || c->pages > INT32_MAX / c->page_size) return MX_ERR_SHAPE;
    if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return MX_ERR_NULL;
    if (!aligned_to(c->k_codes, 16) || !aligned_to(c->k_scales, 16) || !aligned_to(c->v_codes, 16) ||
        !aligned_to(c->v_scales, 16))
        return MX_ERR_ALIGN;
    v = CacheView{{c->k_codes, c->v_codes}, {c->k_scales, c->v_scales}, c->pages, c->heads, __builtin_ctz(c->page_size),
                  c->head_dim, c->use_rht != 0, c->use_rht ? c->sign_mask : 0u};
    return MX_OK;
}

}  // namespace mx
