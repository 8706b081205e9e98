// mx_attention.hip -- attention over the MXFP4 key/value cache (gfx950).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mx.h"
#include "mx_cache.h"
#include "mx_device.h"
#include "mx_host.h"

namespace {

using namespace mx;

struct AttentionArgs {
    CacheView cache;
    const void* q;
    int64_t tokens, q_ld, q_head_ld;
    int q_heads;
    const int32_t* q_offsets;     // or null: one row a sequence
    int seqs;
    const int32_t* table;
    int64_t table_ld;
    int64_t capacity;             // tokens that a sequence's table entries hold
    const int32_t* lengths;
    float scale;                  // times log2(e)
    int causal, window;
    const float* sinks;
    void* out;
    int64_t out_ld, out_head_ld;
    float* lse;
};

constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f;

// One wave: one query row of one head.  Lanes share the keys 64 at a time for
// the scores, and the row's elements for the sum.
template <bool BF16>
__global__ __launch_bounds__(64) void attention_kernel(AttentionArgs a) {
    __shared__ float q[256], p[64];
    __shared__ int64_t page_of[64];
    const int lane = threadIdx.x, dim = a.cache.dim, head = blockIdx.y;
    const int64_t row = blockIdx.x;
    const int kv = head / (a.q_heads / a.cache.heads);
    int seq = (int)row;
    int64_t first = row, rows = 1;
    if (a.q_offsets) {
        int lo = 0, hi = a.seqs;                           // the last sequence that starts at or before the row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (mid < a.seqs ? a.q_offsets[mid] <= row : false) lo = mid;
            else hi = mid - 1;
        }
        seq = lo;
        first = a.q_offsets[seq];
        rows = a.q_offsets[seq + 1] - first;
        if (row < first || row >= first + rows) return;
    }
    const int64_t length = min(max((int64_t)a.lengths[seq], (int64_t)0), a.capacity);
    const int64_t pos = length - rows + (row - first);
    const int64_t end = a.causal ? pos + 1 : length, begin = a.window ? max(pos - a.window + 1, (int64_t)0) : 0;

    const int64_t at = row * a.q_ld + head * a.q_head_ld + 8 * lane;
    if (8 * lane < dim) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.q)[at + i] << 16) : ((const float*)a.q)[at + i];
        if (a.cache.rht) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = (a.cache.mask >> (8 * (lane & 3) + i)) & 1 ? -f[i] : f[i];
            rht32_quad(f, lane & 3);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) q[8 * lane + i] = f[i];
    }
    __syncthreads();

    float top = a.sinks ? a.sinks[head] * LOG2E : -__builtin_inff(), sum = a.sinks ? 1.0f : 0.0f;
    float acc[4] = {};                                     // elements 2 lane, 2 lane + 1, and those 128 further
    const int bytes = dim >> 1, shift = a.cache.page_log2;
    for (int64_t base = begin; base < end; base += 64) {
        const int64_t key = base + lane;
        int64_t page = key < end ? a.table[seq * a.table_ld + (key >> shift)] : -1;
        if (page >= a.cache.pages) page = -1;
        const int offset = (int)(key & ((1 << shift) - 1));
        float s = -__builtin_inff();
        if (page >= 0) {
            const uint8_t* codes = a.cache.codes[0] + a.cache.codes_at(page, kv, offset);
            const uint8_t* scales = a.cache.scales[0] + a.cache.scales_at(page, kv, offset);
            float dot = 0.0f;
            for (int d = 0; d < dim; d += 8) {
                const uint32_t byte = scales[(int64_t)(d >> 5) << shift];
                float f[8];
                decode8(*(const uint32_t*)(codes + (d >> 1)), scale_operand(byte), f);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(q[d + i], byte == 0xFF ? __builtin_nanf("") : f[i], dot);
            }
            s = dot * a.scale;
        }
        float m = s;
#pragma unroll
        for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
        m = fmaxf(m, top);
        const float safe = m == -__builtin_inff() ? 0.0f : m, keep = __builtin_amdgcn_exp2f(top - safe);
        const float w = page < 0 ? 0.0f : __builtin_amdgcn_exp2f(s - safe);
        float total = w;
#pragma unroll
        for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
        sum = sum * keep + total;
        top = m;
        __syncthreads();
        p[lane] = w;
        page_of[lane] = page;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= keep;
        const int n = (int)min((int64_t)64, end - base);
        for (int j = 0; j < n; ++j) {
            if (page_of[j] < 0) continue;
            const int o = (int)((base + j) & ((1 << shift) - 1));
            const int64_t c = a.cache.codes_at(page_of[j], kv, o), sc = a.cache.scales_at(page_of[j], kv, o);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int b = lane + 64 * h;
                if (b >= bytes) continue;
                const uint32_t byte = a.cache.scales[1][sc + ((int64_t)(b >> 4) << shift)];
                const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a.cache.codes[1][c + b], scale_operand(byte), 0);
                acc[2 * h] = __builtin_fmaf(p[j], byte == 0xFF ? __builtin_nanf("") : v[0], acc[2 * h]);
                acc[2 * h + 1] = __builtin_fmaf(p[j], byte == 0xFF ? __builtin_nanf("") : v[1], acc[2 * h + 1]);
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (lane + 64 * h >= bytes) continue;
        q[2 * (lane + 64 * h)] = sum == 0.0f ? 0.0f : acc[2 * h] * inv;
        q[2 * (lane + 64 * h) + 1] = sum == 0.0f ? 0.0f : acc[2 * h + 1] * inv;
    }
    __syncthreads();
    if (8 * lane < dim) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = q[8 * lane + i];
        if (a.cache.rht) {
            rht32_quad(f, lane & 3);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = (a.cache.mask >> (8 * (lane & 3) + i)) & 1 ? -f[i] : f[i];
        }
        const int64_t to = row * a.out_ld + head * a.out_head_ld + 8 * lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (BF16) ((uint16_t*)a.out)[to + i] = (uint16_t)f32_to_bf16_rne(f[i]);
            else ((float*)a.out)[to + i] = f[i];
        }
    }
    if (a.lse && lane == 0)
        a.lse[row * a.q_heads + head] = sum == 0.0f ? -__builtin_inff() : (top + log2f(sum)) * LN2;
}

mx_status check_pitches(int64_t ld, int64_t head_ld, int dim) {
    return ld < 0 || head_ld < 0 || (ld && ld < dim) || (head_ld && head_ld < dim) ? MX_ERR_SHAPE : MX_OK;
}

}  // namespace

extern "C" {

int64_t mx_cache_attention_workspace(const mx_cache* cache, int64_t tokens, int32_t q_heads, int32_t max_queries) {
    return 0;
}

mx_status mx_cache_attention(const mx_cache* cache, const void* q, mx_dtype qt, int64_t tokens, int32_t q_heads,
                             int64_t q_ld, int64_t q_head_ld, const int32_t* q_offsets, int32_t max_queries,
                             int32_t seqs, const int32_t* page_table, int64_t table_ld, int32_t table_pages,
                             const int32_t* lengths, float scale, int causal, int32_t window, const float* sinks,
                             void* out, int64_t out_ld, int64_t out_head_ld, float* lse, void* workspace,
                             mx_stream stream) {
    CacheView c;
    const mx_status bad = view_cache(cache, c);
    if (bad != MX_OK) return bad;
    if (qt != MX_F32 && qt != MX_BF16) return MX_ERR_DTYPE;
    if (tokens < 0 || q_heads < 1 || q_heads % c.heads || tokens > INT32_MAX / q_heads) return MX_ERR_SHAPE;
    if (seqs < 0 || seqs >= 1 << 24 || (tokens > 0 && seqs == 0) || (!q_offsets && tokens != seqs)) return MX_ERR_SHAPE;
    if (table_pages < 0 || table_ld < 0 || (table_ld && table_ld < table_pages) ||
        table_pages > INT32_MAX / cache->page_size)
        return MX_ERR_SHAPE;
    if (max_queries < 0 || window < 0 || (window && !causal) || !(scale > 0.0f) || !(scale - scale == 0.0f))
        return MX_ERR_SHAPE;
    if (check_pitches(q_ld, q_head_ld, c.dim) != MX_OK || check_pitches(out_ld, out_head_ld, c.dim) != MX_OK)
        return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!q || !out || !lengths || (table_pages > 0 && !page_table)) return MX_ERR_NULL;
    if (mx_cache_attention_workspace(cache, tokens, q_heads, max_queries) > 0 && !workspace) return MX_ERR_NULL;
    if (!aligned_to(q, type_bytes(qt)) || !aligned_to(out, type_bytes(qt)) || !aligned_to(q_offsets, 4) ||
        !aligned_to(page_table, 4) || !aligned_to(lengths, 4) || !aligned_to(sinks, 4) || !aligned_to(lse, 4) ||
        !aligned_to(workspace, 16))
        return MX_ERR_ALIGN;
    const int64_t row = (int64_t)q_heads * c.dim;
    AttentionArgs a{};
    a.cache = c;
    a.q = q;
    a.tokens = tokens;
    a.q_ld = q_ld ? q_ld : row;
    a.q_head_ld = q_head_ld ? q_head_ld : c.dim;
    a.q_heads = q_heads;
    a.q_offsets = q_offsets;
    a.seqs = seqs;
    a.table = page_table;
    a.table_ld = table_ld ? table_ld : table_pages;
    a.capacity = (int64_t)table_pages * cache->page_size;
    a.lengths = lengths;
    a.scale = scale * LOG2E;
    a.causal = causal != 0;
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.out_ld = out_ld ? out_ld : row;
    a.out_head_ld = out_head_ld ? out_head_ld : c.dim;
    a.lse = lse;
    hipStream_t s = (hipStream_t)stream;
    const dim3 grid((uint32_t)tokens, (uint32_t)q_heads);
    (void)hipGetLastError();
    if (qt == MX_BF16) hipLaunchKernelGGL(attention_kernel<true>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(attention_kernel<false>, grid, dim3(64), 0, s, a);
    return launch_status();
}

}  // extern "C"
