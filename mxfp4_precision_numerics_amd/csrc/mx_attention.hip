// mx_attention.hip -- attention over the MXFP4 key/value cache (gfx950).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/mx.h"
#include "mx_cache.h"
#include "mx_device.h"
#include "mx_host.h"
#include "mx_line.h"
#include "mx_rows.h"

namespace {

using namespace mx;

struct Cut;

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
    int near, min_units, group, tile_tokens, tile_log2, tile_heads, head_tiles, line_heads;
    uint32_t code_page, scale_page;   // bytes of a page's codes, scales
    float* parts;
    Cut* cuts;                    // one a share
};

constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f, MAX_FLOAT = 3.40282347e38f;
constexpr float MAX_SCALE = 0x1p127f;  // times log2 e still finite
constexpr int WAVES = 4;              // of a workgroup, sharing a tile's keys
constexpr int MIN_UNITS = WAVES;      // of a workgroup's share, at least, where segments are cut
constexpr int WHOLE_UNITS = 16;       // of a segment that is not cut
// The exponentials' reference is kept until a row's largest score has outgrown it
// by 2^GROWTH: any reference serves, as long as nothing overflows (two prompts, 4096
// queries behind 4096 tokens and 517 behind 1685, 32 heads of 128: 568 us; 587 where
// the sums are scaled for each new maximum)
constexpr float GROWTH = 8.0f;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4v __attribute__((ext_vector_type(4), aligned(2)));

// Accesses through pointers that the compiler cannot tell to be ones to global
// memory.  (A flat access makes it wait for every load under way.)
template <class T>
__device__ __forceinline__ T load_global(const void* p) {
    return *(const __attribute__((address_space(1))) T*)p;
}
template <class T>
__device__ __forceinline__ void store_global(void* p, T v) {
    *(__attribute__((address_space(1))) T*)p = v;
}

// ---------------------------------------------------------------------------
// The work and its shares.
//
// A tile: up to 16 NT rows of one sequence and cache head: `tile_tokens`
// consecutive queries (a power of two) times `tile_heads` of the group's query
// heads.  A segment: a tile and the keys that its rows see, in units of 64.
// All segments' units, in the order sequence, cache head (and part of its
// group), tile, key, are one long line that the workgroups cut into equal
// shares, whatever the lengths are: every workgroup finds its share from the
// lengths themselves.  A segment that lies in one share, or is short, is
// finished there; of one that is cut every share leaves its part (sums, maxima)
// in the workspace, two parts a workgroup at most, and a second launch joins
// them.
// ---------------------------------------------------------------------------
// A value that every lane has, for the scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

__device__ __forceinline__ Seq load_seq(const AttentionArgs& a, int s) {
    Seq q;
    int64_t b = s, e = s + 1;
    if (a.q_offsets) {
        b = min(max((int64_t)load_global<int32_t>(a.q_offsets + s), (int64_t)0), a.tokens);
        e = min(max((int64_t)load_global<int32_t>(a.q_offsets + s + 1), b), a.tokens);
    }
    q.row0 = b;
    q.n = (int)(e - b);
    q.len = (int)min(max((int64_t)load_global<int32_t>(a.lengths + s), (int64_t)0), a.capacity);
    return q;
}

// The line's length, and where one unit of it lies: each thread has a stretch
// of sequences.
struct Line {
    int64_t wave_units[WAVES], total;
    int64_t from;             // units before the stretch that holds it
    int stretch;
};

struct Segment {
    Seq seq;
    int s, head, tile;        // sequence, cache head * head_tiles + part of its group, tile
    int begin, end;           // its units (of keys)
    int64_t start;            // its first unit's place in the line

    // Whether it is done by the share in which it starts: cutting a short one
    // and joining it takes longer than its last steps.
    __device__ __forceinline__ bool whole() const { return end - begin <= WHOLE_UNITS; }
};

// What a share leaves about the segment that it began and did not finish:
// count parts, the first one `slot`, then the even slots of the shares after.
struct Cut {
    Segment seg;
    int count, pad;           // 0: there is none
    int64_t slot;

    __device__ __forceinline__ void write(Cut* to) const {
        uint32_t w[sizeof(Cut) / 4];
        __builtin_memcpy(w, this, sizeof(Cut));
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Cut) / 4); ++i) store_global((uint32_t*)to + i, w[i]);
    }
};
static_assert(sizeof(Cut) % 16 == 0, "the parts follow the cuts, 16-byte aligned");

// The workgroup's share.  Workgroups go round the 8 XCDs in turn.  Few rows over
// long caches: neighbouring shares, which hold parts of one sequence, are put on
// one XCD (5 rows of 32 sequences of 8192 tokens, 8 heads of 128: 65 us in place
// of 81); else they are spread (prompts of 2048 tokens: 114 in place of 122).
__device__ __forceinline__ int share_id(const AttentionArgs& a) {
    return a.near ? (int)((blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) : (int)blockIdx.x;
}

// Measures the line, and finds the stretch of unit share * (what a share has):
// returns that unit's place, not less than the line's length if there is none.
__device__ __forceinline__ int64_t measure_line(const AttentionArgs& a, Line& line, int64_t& per) {
    const int tid = threadIdx.x, each = (a.seqs + WAVES * 64 - 1) / (WAVES * 64);
    int64_t mine = 0;
    for (int s = tid * each; s < min((tid + 1) * each, a.seqs); ++s) mine += units_of(a, load_seq(a, s));
    mine *= a.line_heads;
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t other = __shfl_up(sum, d);
        if ((tid & 63) >= d) sum += other;
    }
    if ((tid & 63) == 63 && tid < WAVES * 64) line.wave_units[tid >> 6] = sum;      // (a later thread has none)
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int64_t u = line.wave_units[w];
        if (w < tid >> 6) base += u;
        total += u;
    }
    total = uniform(total);
    per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)a.min_units);
    const int64_t at = share_id(a) * per, from = base + sum - mine;
    if (from <= at && at < from + mine) {
        line.from = from;
        line.stretch = tid;
    }
    if (tid == 0) line.total = total;
    __syncthreads();
    return at;
}

__device__ __forceinline__ Seq load_uniform_seq(const AttentionArgs& a, int s) {
    Seq q = load_seq(a, s);
    q.row0 = uniform(q.row0);
    q.n = uniform(q.n);
    q.len = uniform(q.len);
    return q;
}

__device__ __forceinline__ void set_tile(const AttentionArgs& a, Segment& g) {
    g.begin = first_unit(a, g.seq, g.tile);
    g.end = end_unit(a, g.seq, g.tile);
}

// The segment that holds unit `at`, which measure_line found.
__device__ __forceinline__ Segment locate(const AttentionArgs& a, const Line& line, int64_t at) {
    Segment g;
    int lo, hi;
    int64_t from = uniform(line.from), units;
    g.s = uniform(line.stretch) * ((a.seqs + WAVES * 64 - 1) / (WAVES * 64));
    for (;; ++g.s) {
        g.seq = load_uniform_seq(a, g.s);
        units = units_of(a, g.seq);
        if (at < from + units * a.line_heads) break;
        from += units * a.line_heads;
    }
    g.head = (int)((at - from) / units);
    from += g.head * units;
    lo = 0;
    hi = tiles_of(a, g.seq) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (from + units_before(a, g.seq, mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    g.tile = lo;
    g.start = from + units_before(a, g.seq, lo);
    set_tile(a, g);
    return g;
}

__device__ __forceinline__ void next_segment(const AttentionArgs& a, Segment& g) {
    g.start += g.end - g.begin;
    if (++g.tile == tiles_of(a, g.seq)) {
        g.tile = 0;
        if (++g.head == a.line_heads) {
            g.head = 0;
            do g.seq = load_uniform_seq(a, ++g.s);
            while (g.seq.n == 0);
        }
    }
    set_tile(a, g);
}

// The kernel's arguments, read again from where they were passed.  What only
// the begin and the end of a segment need would otherwise hold scalar registers
// through the loop over the keys, which then spills (150 of them, a vector
// instruction each on the way back).
__device__ __forceinline__ AttentionArgs arguments() {
    typedef const __attribute__((address_space(4))) uint32_t Word;
    Word* p = (Word*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    union {
        uint32_t w[sizeof(AttentionArgs) / 4];
        AttentionArgs a;
    } u;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(AttentionArgs) / 4); ++i) u.w[i] = p[i];
    return u.a;
}

// A tile's row c: its query row and head; false where there is none.
struct Row {
    int64_t token;
    int head, query;          // query: its number in the sequence
};
__device__ __forceinline__ bool row_of(const AttentionArgs& a, const Segment& g, int c, Row& r) {
    const int t = c / a.tile_heads, part = g.head / a.head_tiles;
    const int h = (g.head - part * a.head_tiles) * a.tile_heads + c - t * a.tile_heads;
    r.query = (g.tile << a.tile_log2) + t;
    r.token = g.seq.row0 + r.query;
    r.head = part * a.group + h;
    return t < a.tile_tokens && h < a.group && t < g.seq.n - (g.tile << a.tile_log2);
}

// A row's maximum, sum and the factor of its sums with its head's sink logit.
// Times log2 e a sink near the largest fp32, or infinite, is held at that: less a
// finite maximum it is no NaN, and every other p is 0 next to it.
struct Sink {
    float top, sum, factor;

    __device__ __forceinline__ Sink(const AttentionArgs& a, const Row& r, bool live, float t, float s)
        : top(t), sum(s), factor(1.0f) {
        if (!a.sinks) return;
        const float x = live ? load_global<float>(a.sinks + r.head) : 0.0f;
        float sink = x * LOG2E;
        if (__builtin_isinf(sink) && x != -__builtin_inff()) sink = __builtin_copysignf(MAX_FLOAT, x);
        top = fmaxf(t, sink);
        const float safe = top == -__builtin_inff() ? 0.0f : top;
        factor = __builtin_amdgcn_exp2f(t - safe);
        sum = s * factor + __builtin_amdgcn_exp2f(sink - safe);
    }
    __device__ __forceinline__ void store_lse(const AttentionArgs& a, const Row& r) const {
        float l = sum == 0.0f ? -__builtin_inff() : (top + log2f(sum)) * LN2;
        if (a.sinks && fabsf(top) == MAX_FLOAT) l = load_global<float>(a.sinks + r.head);      // (held, and alone)
        store_global(a.lse + r.token * a.q_heads + r.head, l);
    }
};

// ---------------------------------------------------------------------------
// Eight elements of a row from the tile's sums: the sink, the division, the
// transform back, the rounding.  top, sum: the row's maximum (times log2 e) and
// sum; o relative to that maximum.  Four lanes hold a block of 32; all of them
// call.
// ---------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void finish(const AttentionArgs& a, const Row& r, bool live, int d, float* o, float top,
                                       float sum) {
    const Sink all(a, r, live, top, sum);
    if (a.sinks) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= all.factor;
    }
    const float inv = 1.0f / all.sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = all.sum == 0.0f ? 0.0f : o[i] * inv;
    if (a.cache.rht) {
        rht32_quad(o, (d >> 3) & 3);
        const uint32_t m = a.cache.mask >> (d & 31);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(__float_as_uint(o[i]) ^ (m >> i << 31));
    }
    if (!live || d >= a.cache.dim) return;
    const int64_t at = r.token * a.out_ld + r.head * a.out_head_ld + d;
    if constexpr (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16_rne(o[2 * i]) | f32_to_bf16_rne(o[2 * i + 1]) << 16;
        store_global((uint16_t*)a.out + at, (u32x4v){u[0], u[1], u[2], u[3]});
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            store_global((float*)a.out + at + 4 * i,
                         (u32x4v){__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                                  __float_as_uint(o[4 * i + 3])});
    }
    if (a.lse && d == 0) all.store_lse(a, r);
}

// A part in the workspace: sums [rows][32 NB], maxima [rows], sums of p [rows].
template <int NB, int ROWS>
struct Part {
    static constexpr int FLOATS = ROWS * (32 * NB + 2);
    float* p;
    __device__ __forceinline__ Part(const AttentionArgs& a, int64_t i) : p(a.parts + i * FLOATS) {}
    __device__ __forceinline__ float* row(int c) const { return p + c * 32 * NB; }
    __device__ __forceinline__ float* top(int c) const { return p + ROWS * 32 * NB + c; }
    __device__ __forceinline__ float* sum(int c) const { return p + ROWS * 32 * NB + ROWS + c; }
};

__device__ __forceinline__ uint32_t bits(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Two fp32 as bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return bits(v);
}

// The same for the 8 NB consecutive elements of a row that a lane has in
// registers, from d on (a multiple of 8 NB).  Heads of up to 64 elements share a
// block between lanes 16 apart.
template <int NB, bool BF16>
__device__ __forceinline__ void finish_row(const AttentionArgs& a, const Row& r, bool live, int d, float* o, float top,
                                           float sum) {
    constexpr int N = 8 * NB;
    const Sink all(a, r, live, top, sum);
    const float inv = all.factor / all.sum;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = all.sum == 0.0f ? 0.0f : o[i] * inv;
    if (a.cache.rht) {
        constexpr int IN = N < 32 ? N : 32;
#pragma unroll
        for (int b = 0; b < N; b += IN) {
            fwht_inlane<IN>(o + b);
            if constexpr (IN < 32) {
                const float s = threadIdx.x & 16 ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < IN; ++i) o[b + i] = __builtin_fmaf(o[b + i], s, __shfl_xor(o[b + i], 16));
            }
            const float c = __uint_as_float(0x3E3504F3u);  // fp32(2^-2.5)
            const uint32_t m = a.cache.mask >> ((d + b) & 31);
#pragma unroll
            for (int i = 0; i < IN; ++i) o[b + i] = __uint_as_float(__float_as_uint(o[b + i] * c) ^ (m >> i << 31));
        }
    }
    if (!live) return;
    const int64_t at = r.token * a.out_ld + r.head * a.out_head_ld + d;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        if (d + i >= a.cache.dim) continue;
        if constexpr (BF16) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = pack(o[i + 2 * k], o[i + 2 * k + 1]);
            store_global((uint16_t*)a.out + at + i, (u32x4v){u[0], u[1], u[2], u[3]});
        } else {
#pragma unroll
            for (int k = 0; k < 8; k += 4)
                store_global((float*)a.out + at + i + k,
                             (u32x4v){__float_as_uint(o[i + k]), __float_as_uint(o[i + k + 1]), __float_as_uint(o[i + k + 2]),
                                      __float_as_uint(o[i + k + 3])});
        }
    }
    if (a.lse && d == 0) all.store_lse(a, r);
}

// The other value of a row of 16 lanes' neighbour (16 lanes on, then 32): of
// the two results one is the lane's own, the other its partner's.
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
template <class Op>
__device__ __forceinline__ float across(float v, Op op) {
    u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r.x), __uint_as_float(r.y));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(r.x), __uint_as_float(r.y));
}

// Eight codes and their scale as bf16, exactly (E2M1 times a power of two).
__device__ __forceinline__ void widen8(uint32_t w, float scale, uint32_t* u) {
    u[0] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    u[1] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    u[2] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    u[3] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
}
__device__ __forceinline__ uint32_t widen2(uint32_t w, float scale, int byte) {
    switch (byte) {           // (a constant)
    case 0: return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    case 1: return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    case 2: return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    default: return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    }
}
__device__ __forceinline__ float scale_of(uint32_t word, int byte) {       // byte: 0..3
    return scale_operand((word >> (8 * byte)) & 0xFFu);
}

// ---------------------------------------------------------------------------
// The kernel.  A wave takes 64 keys and all rows of its tile:
//   S^T = K Q^T   16x16x32 products, keys down, rows across: K's codes of a
//                 lane are consecutive in memory (8 NB of them), Q comes from
//                 LDS in the same order of elements;
//   softmax       a lane has 4 keys of one row in each product, so maxima and
//                 sums over the keys take two exchanges between lanes;
//   O^T = V^T P^T the lane's own p are what the product wants of it when the
//                 keys go in the order (group of 8, product, number): no p
//                 changes lanes.  V's elements of a lane are 2 NB consecutive
//                 ones of eight keys; converted key by key and paired by two
//                 byte permutations.
// Keys of a wave's 64: 32 j + 8 g + 4 t + i is row 4 g + i of score product
// (j, t).  Lane l: column l & 15, group g = l >> 4.
// NB: blocks of 32 that a row is padded to (2, 4, 8); NT: products of 16 rows.
// QT: terms of q, PT: terms of p, in bf16: one each for bf16 rows, two of q where
// it was transformed (then it is no bf16 any more), three for fp32 rows (with two,
// an output's error is 3.3e-6 of its norm, with three 3e-7).  p's half step of 2^-8
// is that of a bf16 output, whose error against 64 bits it makes 2.1e-3 to 2.3e-3
// of the norm, 1.7e-3 of it the output's own rounding.  Two terms of p leave that
// alone, for 3 to 5% of the time with one query a request, 17% with five, 24% of a
// prompt's; who wants them has them, and more, with fp32 queries.
// Bound by HBM: 64 requests of up to 16384 tokens, 8 heads of 128, 139 us (4.5
// TB/s); one of 262144 tokens 53 us (5.6).  Keys and values go from memory to
// registers to the products, no byte through LDS, and a step's loads are sent
// for during the step before.
// ---------------------------------------------------------------------------
template <int NB, int NT, int QT>
struct Shared {
    static constexpr int PITCH = 32 * NB + 8;              // bf16: rows 4 banks apart
    static constexpr int SIDE = NB == 8 ? 128 : 32 * NB, OUT_PITCH = SIDE + 4;
    static constexpr int Q_BYTES = QT * 16 * NT * PITCH * 2, O_BYTES = WAVES * 16 * OUT_PITCH * 4;
    alignas(16) unsigned char data[Q_BYTES > O_BYTES ? Q_BYTES : O_BYTES];
    float top[WAVES][16 * NT], sum[WAVES][16 * NT];
    Line line;
};

// Where a lane finds its part of a page's first group of eight keys, in page 0:
// K's codes (8 NB of them) and scales of key col & 3, V's codes (2 NB) and
// scales of the first key.
template <int NB, bool EXACT>
struct Lane {
    const uint8_t *k, *ks, *v, *vs;
    bool second;                          // NB = 8: the row reaches the lane's second half

    // What a lane would read past the row's end it reads from its begin instead.
    // Of K that meets elements of q that are 0, and is not finite only where the
    // key's score is not anyway; of V it makes elements that nobody writes.
    __device__ __forceinline__ int half(int h) const { return EXACT || second ? h : 0; }
    __device__ __forceinline__ Lane(const AttentionArgs& a, int head, int col, int g) {
        const int shift = a.cache.page_log2, row_bytes = EXACT ? 16 * NB : a.cache.dim >> 1;
        const int blocks = EXACT ? NB : a.cache.dim >> 5;
        const int c = EXACT || col * NB < row_bytes ? col : 0;
        const int piece = EXACT || 4 * NB * g < row_bytes ? 4 * NB * g : 0;        // bytes into a row
        second = piece + 16 < row_bytes;
        const int64_t codes = ((int64_t)head << shift) * row_bytes, scales = (int64_t)head * blocks << shift;
        k = a.cache.codes[0] + codes + (col & 3) * row_bytes + piece;
        ks = a.cache.scales[0] + scales + ((int64_t)(piece >> 4) << shift);
        v = a.cache.codes[1] + codes + c * NB;
        vs = a.cache.scales[1] + scales + ((int64_t)(c * NB >> 4) << shift);
    }
};

__device__ __forceinline__ const uint8_t* in_page(const uint8_t* p, int page, uint32_t bytes) {
    return p + (uint64_t)(uint32_t)page * bytes;
}

// Values that are not finite as bf16 (or fp32): all of a block with the scale
// byte 0xFF, and with the bytes 253 and 254 (2^126 and 2^127) the codes from 4 and
// from 2 on.  A row's product must not meet those of keys that it does not see,
// for 0 times them is NaN.
// Whether one of eight scale bytes is 253 or more.
__device__ __forceinline__ bool any_odd(uint2 w) {
    const uint32_t x = ((w.x & 0x7F7F7F7Fu) + 0x03030303u) & w.x, y = ((w.y & 0x7F7F7F7Fu) + 0x03030303u) & w.y;
    return ((x | y) & 0x80808080u) != 0;
}
// Of eight keys' scales those become 0 whose codes (the lane's, WORDS each) are
// not all finite; a bit each says which.
template <int WORDS>
__device__ __forceinline__ uint32_t take_out(uint2& scales, const uint32_t (&codes)[8][WORDS]) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t& w = i < 4 ? scales.x : scales.y;
        const uint32_t byte = (w >> (8 * (i & 3))) & 0xFFu;
        uint32_t two = 0, four = 0;                        // magnitudes of 2 or more, of 4 or more
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            two |= codes[i][k] & 0x44444444u;
            four |= codes[i][k] & (codes[i][k] << 1) & 0x44444444u;
        }
        if (byte == 0xFFu || (byte == 0xFEu && two) || (byte == 0xFDu && four)) {
            w &= ~(0xFFu << (8 * (i & 3)));
            out |= 1u << i;
        }
    }
    return out;
}
// Eight bits as an operand: 1 where a bit is set.
__device__ __forceinline__ bf16x8 ones(uint32_t b) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ((b >> (2 * i)) & 1u) * 0x3F80u | ((b >> (2 * i + 1)) & 1u) * 0x3F800000u;
    return operand(w[0], w[1], w[2], w[3]);
}

// Whether a row that sees the keys low .. last sees key from + i.
__device__ __forceinline__ bool sees(int last, int low, int from, int i) { return i <= last - from && i >= low - from; }

// A tile's queries on their way to LDS: eight elements of N rows a thread.
// load() sends for them; store() puts them down as QT terms of bf16,
// transformed where the cache is, 0 where there is no row.  The whole workgroup
// calls.
template <int NB, int ROWS, bool BF16, int QT, int THREADS = WAVES * 64>
struct Queries {
    static constexpr int ITEMS = ROWS * 4 * NB, N = (ITEMS + THREADS - 1) / THREADS;
    u32x4v w[N][BF16 ? 1 : 2];

    __device__ __forceinline__ void load(const AttentionArgs& a, const Segment& seg) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * THREADS, c = i / (4 * NB), d = i % (4 * NB) * 8;
            Row r;
            const bool live = row_of(a, seg, c, r) && d < a.cache.dim && i < ITEMS;
            const int64_t from = r.token * a.q_ld + r.head * a.q_head_ld + d;
#pragma unroll
            for (int e = 0; e < (BF16 ? 1 : 2); ++e) {
                w[k][e] = (u32x4v){0, 0, 0, 0};
                if (live)
                    w[k][e] = BF16 ? load_global<u32x4v>((const uint16_t*)a.q + from)
                                   : load_global<u32x4v>((const float*)a.q + from + 4 * e);
            }
        }
    }
    template <int ONLY = -1>                               // that term alone
    __device__ __forceinline__ void store(const AttentionArgs& a, __bf16* to, int pitch) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * THREADS, c = i / (4 * NB), d = i % (4 * NB) * 8;
            if (i >= ITEMS) break;
            float f[8];
            if constexpr (BF16) {
                const uint32_t u[4] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) { f[2 * e] = bf16lo(u[e]); f[2 * e + 1] = bf16hi(u[e]); }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const u32x4v& x = w[k][BF16 ? 0 : e];
                    f[4 * e] = __uint_as_float(x.x);
                    f[4 * e + 1] = __uint_as_float(x.y);
                    f[4 * e + 2] = __uint_as_float(x.z);
                    f[4 * e + 3] = __uint_as_float(x.w);
                }
            }
            if (a.cache.rht) {
                const uint32_t m = a.cache.mask >> (d & 31);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(__float_as_uint(f[e]) ^ (m >> e << 31));
                rht32_quad(f, (d >> 3) & 3);
            }
#pragma unroll
            for (int y = 0; y < QT; ++y) {
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = pack(f[2 * e], f[2 * e + 1]);
                if (ONLY < 0 || ONLY == y)
                    *(uint4*)(to + ((ONLY < 0 ? y * ROWS : 0) + c) * pitch + d) = make_uint4(u[0], u[1], u[2], u[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {              // what is left (of an infinite element, nothing)
                    const float lo = bf16lo(u[e]), hi = bf16hi(u[e]);
                    f[2 * e] = __builtin_isinf(lo) ? 0.0f : f[2 * e] - lo;
                    f[2 * e + 1] = __builtin_isinf(hi) ? 0.0f : f[2 * e + 1] - hi;
                }
            }
        }
    }
};

template <int NB, int NT, bool EXACT, bool BF16, int QT, int PT>
__global__ __launch_bounds__(WAVES * 64, NT == 1 && NB < 8 ? 3 : 2) void attention_kernel(AttentionArgs a) {
    using Sh = Shared<NB, NT, QT>;
    constexpr int M = 2 * NB;                              // elements of V that a lane has, products of the sum
    constexpr int VW = NB == 8 ? 2 : 1;                    // dwords they take
    __shared__ Sh sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4, q_at = col * Sh::PITCH + 8 * NB * g;
    const int shift = a.cache.page_log2;
    const int row_bytes = EXACT ? 16 * NB : a.cache.dim >> 1;
    const float scale = a.scale;

    int64_t per;
    const int64_t begin = measure_line(a, sh.line, per), total = uniform(sh.line.total), stop = min(begin + per, total);
    if (tid == 0) a.cuts[share_id(a)].count = 0;
    if (begin >= total) return;
    Segment seg = locate(a, sh.line, begin);
    int64_t at = begin;
    if (seg.start < begin && seg.whole()) {                // the share before has all of it
        at = seg.start + seg.end - seg.begin;
        if (at >= stop) return;
        next_segment(a, seg);
    }

    for (;;) {
        const int head = seg.head / a.head_tiles;          // of the cache
        const int rows = min(a.tile_tokens, seg.seq.n - (seg.tile << a.tile_log2)) * a.tile_heads;
        const int unit0 = seg.begin + (int)(at - seg.start);
        const int unit1 = seg.whole() ? seg.end : (int)min((int64_t)seg.end, seg.begin + (stop - seg.start));
        // (a sequence without keys has no pages to look at)
        const int units = seg.seq.len == 0 ? 0 : unit1;
        const int32_t* table = a.table + seg.s * a.table_ld;
        const int last_group = (seg.seq.len - 1) & ~7;

        uint32_t kc[2][2][NB];        // codes of K: [j][t]
        uint2 ks[2][NB == 8 ? 2 : 1]; // eight keys' scales of the lane's blocks
        uint32_t vc[2][8][VW];        // codes of V: [j][key]
        uint2 vs[2];
        const int kg = 8 * (col >> 2);                     // the lane's group of keys in a score product

        // A lane looks up the page of one of a unit's eight groups of keys, -1 if it does not exist; others get it
        // from there.
        auto look_up = [&](int unit) { return table[min(UNIT * unit + 8 * (lane & 7), last_group) >> shift]; };
        auto checked = [&](int page) { return page >= 0 && page < (int)a.cache.pages ? page : -1; };
        auto page_of = [&](int pages, int group) { return __builtin_amdgcn_ds_bpermute(4 * group, pages); };
        const Lane<NB, EXACT> my(a, head, col, g);
        auto load_k = [&](int unit, int j, int page) {
            const int o = min(UNIT * unit + 32 * j + kg, last_group) & ((1 << shift) - 1);
            const uint8_t* codes = in_page(my.k, max(page, 0), a.code_page) + o * row_bytes;
            const uint8_t* scales = in_page(my.ks, max(page, 0), a.scale_page) + o;
            if constexpr (NB == 2) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint2 w = *(const uint2*)(codes + 4 * t * row_bytes);
                    kc[j][t][0] = w.x;
                    kc[j][t][1] = w.y;
                }
                ks[j][0] = *(const uint2*)scales;
            } else {
#pragma unroll
                for (int h = 0; h < NB / 4; ++h) {
                    const int more = my.half(h);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint4 w = *(const uint4*)(codes + 4 * t * row_bytes + 16 * more);
                        kc[j][t][4 * h] = w.x;
                        kc[j][t][4 * h + 1] = w.y;
                        kc[j][t][4 * h + 2] = w.z;
                        kc[j][t][4 * h + 3] = w.w;
                    }
                    ks[j][h] = *(const uint2*)(scales + (more << shift));
                }
            }
        };
        auto load_v = [&](int unit, int j, int page) {
            const int o = min(UNIT * unit + 32 * j + 8 * g, last_group) & ((1 << shift) - 1);
            const uint8_t* codes = in_page(my.v, max(page, 0), a.code_page) + o * row_bytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint8_t* from = codes + i * row_bytes;
                if constexpr (NB == 2) vc[j][i][0] = *(const uint16_t*)from;
                else if constexpr (NB == 4) vc[j][i][0] = *(const uint32_t*)from;
                else {
                    const uint2 w = *(const uint2*)from;
                    vc[j][i][0] = w.x;
                    vc[j][i][VW - 1] = w.y;
                }
            }
            vs[j] = *(const uint2*)(in_page(my.vs, max(page, 0), a.scale_page) + o);
        };

        int unit = unit0 + wave, pages = 0, next_pages = 0;
        // The first keys and the queries are on their way at the same time.  (The loads that the loop needs first come
        // first, so that it waits for them alone.)
        Queries<NB, 16 * NT, BF16, QT> queries;
        if (unit < units) {
            pages = look_up(unit);
            next_pages = look_up(min(unit + WAVES, units - 1));
        }
        queries.load(arguments(), seg);
        __builtin_amdgcn_sched_barrier(0);
        if (unit < units) {
            pages = checked(pages);
#pragma unroll
            for (int j = 0; j < 2; ++j) load_k(unit, j, page_of(pages, 4 * j + (col >> 2)));
        }
        __syncthreads();                                   // (the last segment's rows have been read from the same place)
        queries.store(arguments(), (__bf16*)sh.data, Sh::PITCH);
        __builtin_amdgcn_sched_barrier(0);
        if (unit < units) {
#pragma unroll
            for (int j = 0; j < 2; ++j) load_v(unit, j, page_of(pages, 4 * j + g));
        }
        __syncthreads();

        // the keys that each of the lane's rows sees, and those that all see
        int last[NT], low[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            Row r;
            const bool live = row_of(a, seg, 16 * n + col, r);
            const int pos = position(seg.seq, r.query);
            last[n] = !live ? -1 : a.causal ? pos : seg.seq.len - 1;
            low[n] = first_key(a, pos);
        }
        const int query0 = seg.tile << a.tile_log2;
        const int all_to = a.causal ? position(seg.seq, query0) : seg.seq.len - 1;
        const int all_from = first_key(a, position(seg.seq, query0 + rows / a.tile_heads - 1));

        f32x4 acc[NT][M];
        float top[NT], sum[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n] = -__builtin_inff();
            sum[n] = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) acc[n][m] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }

        for (; unit < units; unit += WAVES) {
            const int key0 = UNIT * unit, ahead = min(unit + WAVES, units - 1);
            const bool whole = key0 + UNIT - 1 <= all_to && key0 >= all_from && !__any(pages < 0);
            next_pages = checked(next_pages);
            const int after = look_up(min(unit + 2 * WAVES, units - 1));
            int q_from = q_at;        // (the queries are read again for every unit: registers do not hold them)
            asm volatile("" : "+v"(q_from));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // scores
                f32x4 s[NT][2];
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    uint32_t kf[2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint2 w = ks[j][NB == 8 ? x >> 2 : 0];
                        widen8(kc[j][t][x], scale_of(t ? w.y : w.x, col & 3), kf[t]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int y = 0; y < QT; ++y) {
                            const bf16x8 q = *(const bf16x8*)((const __bf16*)sh.data + q_from +
                                                              (y * 16 * NT + 16 * n) * Sh::PITCH + 8 * x);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                s[n][t] = mfma(operand(kf[t][0], kf[t][1], kf[t][2], kf[t][3]), q,
                                               x == 0 && y == 0 ? (f32x4){0.0f, 0.0f, 0.0f, 0.0f} : s[n][t]);
                        }
                }
                const bool bad = !whole && page_of(pages, 4 * j + g) < 0;
                __builtin_amdgcn_sched_barrier(0);
                load_k(ahead, j, page_of(next_pages, 4 * j + (col >> 2)));

                // softmax of these 32 keys
                uint32_t p[NT][PT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = s[n][i >> 2][i & 3];
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            x[i] = sees(last[n], low[n], key0 + 32 * j + 8 * g, i) && !bad ? x[i] : -__builtin_inff();
                    }
                    float m = x[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) m = fmaxf(m, x[i]);
                    m = fmaxf(across(m, MaxF()) * scale, top[n]);
                    if (__any(m > top[n] + GROWTH)) {
                        const float f = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top[n] - m);
                        sum[n] *= f;
#pragma unroll
                        for (int k = 0; k < M; ++k) acc[n][k] *= f;
                        top[n] = m;
                    }
                    const float safe = top[n] == -__builtin_inff() ? 0.0f : top[n];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], scale, -safe));
                        sum[n] += x[i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float e0 = x[2 * i], e1 = x[2 * i + 1];
#pragma unroll
                        for (int y = 0; y < PT; ++y) {
                            const uint32_t w = p[n][y][i] = pack(e0, e1);
                            e0 -= bf16lo(w);
                            e1 -= bf16hi(w);
                        }
                    }
                }

                __builtin_amdgcn_sched_barrier(0);
                // sums
                uint2 scales = vs[j];
                if (!whole) {
                    // A value that is not finite reaches the rows that see it, and no others: its scale becomes 0
                    // here, and a product of the marks "not finite" and "seen" says where there was one.
                    if (__any(any_odd(scales))) {
                        const bf16x8 mark = ones(take_out(scales, vc[j]));
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t seen = 0;
                            int from = key0 + 32 * j + 8 * g;
                            asm volatile("" : "+v"(from));     // (the comparisons made above are not kept for this)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (sees(last[n], low[n], from, i) && !bad) seen |= 1u << i;
                            const f32x4 hit = mfma(mark, ones(seen), (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (hit[i] == 0.0f) continue;
#pragma unroll
                                for (int k = 0; k < M; ++k) acc[n][k][i] = __builtin_nanf("");
                            }
                        }
                    }
                }
                float sc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[i] = scale_of(i < 4 ? scales.x : scales.y, i & 3);
#pragma unroll
                for (int k = 0; k < M; k += 2) {
                    uint32_t u[8];                         // elements k and k + 1 of the eight keys
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = widen2(vc[j][i][k >> 3], sc[i], (k >> 1) & 3);
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
                        const bf16x8 v = operand(__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel),
                                                 __builtin_amdgcn_perm(u[5], u[4], sel), __builtin_amdgcn_perm(u[7], u[6], sel));
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int y = 0; y < PT; ++y)
                                acc[n][k + odd] = mfma(v, operand(p[n][y][0], p[n][y][1], p[n][y][2], p[n][y][3]),
                                                       acc[n][k + odd]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                load_v(ahead, j, page_of(next_pages, 4 * j + g));
            }
            pages = next_pages;
            next_pages = after;
        }

        // the waves' maxima and sums, then their rows
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            sum[n] = across(sum[n], AddF());
            if (g == 0) {
                sh.top[wave][16 * n + col] = top[n];
                sh.sum[wave][16 * n + col] = sum[n];
            }
        }
        __syncthreads();                                   // (also: nobody reads the queries any more)
        const AttentionArgs b = arguments();
        const bool complete = at == seg.start && unit1 == seg.end;
        const Part<NB, 16 * NT> part(b, 2 * (int64_t)share_id(b) + (at == begin ? 0 : 1));
        constexpr int SIDES = 32 * NB / Sh::SIDE;
        float* o = (float*)sh.data;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (16 * n >= rows) break;
            float m = sh.top[0][16 * n + col];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) m = fmaxf(m, sh.top[w][16 * n + col]);
            const float f = __builtin_amdgcn_exp2f(top[n] - (m == -__builtin_inff() ? 0.0f : m));
#pragma unroll
            for (int side = 0; side < SIDES; ++side) {
                // the lane's elements of a row are consecutive, 8 NB of them: 32 blocks' worth a side
                float* to = o + (wave * 16 + col) * Sh::OUT_PITCH + g * (Sh::SIDE / 4);
                constexpr int PER = 4 / SIDES;
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int k = 0; k < M; k += 4)
                        *(f32x4*)(to + i * M + k) = (f32x4){acc[n][k][side * PER + i] * f, acc[n][k + 1][side * PER + i] * f,
                                                            acc[n][k + 2][side * PER + i] * f, acc[n][k + 3][side * PER + i] * f};
                __syncthreads();
                for (int i = tid; i < 16 * Sh::SIDE / 8; i += WAVES * 64) {
                    const int c = i / (Sh::SIDE / 8), e = i % (Sh::SIDE / 8) * 8;
                    const int d = SIDES == 1 ? e : (e >> 5) * 64 + side * 32 + (e & 31);
                    float most = sh.top[0][16 * n + c];
#pragma unroll
                    for (int w = 1; w < WAVES; ++w) most = fmaxf(most, sh.top[w][16 * n + c]);
                    const float safe = most == -__builtin_inff() ? 0.0f : most;
                    float all = 0.0f, v[8] = {};
#pragma unroll
                    for (int w = 0; w < WAVES; ++w) {
                        all += sh.sum[w][16 * n + c] * __builtin_amdgcn_exp2f(sh.top[w][16 * n + c] - safe);
                        const float* from = o + (w * 16 + c) * Sh::OUT_PITCH + e;
#pragma unroll
                        for (int y = 0; y < 8; ++y) v[y] += from[y];
                    }
                    Row r;
                    const bool live = row_of(b, seg, 16 * n + c, r);
                    if (complete) {
                        finish<BF16>(b, r, live, d, v, most, all);
                    } else if (live) {
                        float* to_part = part.row(16 * n + c) + d;
                        store_global(to_part, (f32x4){v[0], v[1], v[2], v[3]});
                        store_global(to_part + 4, (f32x4){v[4], v[5], v[6], v[7]});
                        if (d == 0) {
                            store_global(part.top(16 * n + c), most);
                            store_global(part.sum(16 * n + c), all);
                        }
                    }
                }
                __syncthreads();
            }
        }
        const int64_t next = seg.start + (seg.end - seg.begin);
        if (unit1 < seg.end && seg.start >= begin && tid == 0) {
            Cut cut;
            cut.seg = seg;
            cut.slot = 2 * (int64_t)share_id(b) + (at == begin ? 0 : 1);
            cut.count = (int)((next - 1) / per) - share_id(b) + 1;
            cut.pad = 0;
            cut.write(b.cuts + share_id(b));
        }
        at = next;
        if (at >= stop) return;
        next_segment(b, seg);
    }
}

// ---------------------------------------------------------------------------
// Many rows of a sequence: prompts, drafts of many heads.
//
// A tile has 128 rows; a wave takes 32 of them (16 where more do not fit the
// registers) and every key.  The workgroup brings in 64 keys at a time, each wave
// its part: it widens K and V to bf16 operands, once for all waves, and puts them
// into LDS lane by lane as the products read them (no bank conflicts).  Two
// buffers; the next unit's is filled while this one's is read.  Products as in
// attention_kernel.  Bound by the vector instructions (exponentials, sums,
// widening) beside the products: two prompts, 4096 queries behind 4096 tokens and
// 517 behind 1685, 32 heads of 128, 533 us and 21 for the join, 774 TFLOP/s; two of
// 4096 behind 4096, 976 us, 845 TFLOP/s; two of 2048 behind 2048, 32 heads of 256,
// 543 us, 760 TFLOP/s (1125 us with 32 rows a wave, whose registers spill).
//
// (K's codes could enter a block-scaled product as they are, with q as a sum of
// e4m3 terms.  Within 16 elements that product aligns its terms to the largest
// and drops what is below 2^-13 of it, so the scores would not be sums in fp32.)
// ---------------------------------------------------------------------------
constexpr int ROWS_TILE = 128;
constexpr int rows_waves(int nb, int qt) { return nb == 8 || (nb == 4 && qt == 3) ? 8 : 4; }

template <int I>
struct Int { static constexpr int value = I; };

template <int NB, int QT>
struct RowsShared {
    static constexpr int M = 2 * NB, V_PARTS = rows_waves(NB, QT) / 2;
    typedef std::conditional_t<V_PARTS == 2, int, int64_t> Odd;    // of a buffer, a byte each
    static constexpr int PITCH = 32 * NB + 8;                  // of q, in bf16
    static constexpr int K_BYTES = 4 * NB * 1024, V_BYTES = 2 * M * 1024;
    union {
        alignas(16) __bf16 q[ROWS_TILE][PITCH];            // one term at a time
        struct {
            alignas(16) unsigned char k[2][K_BYTES], v[2][V_BYTES];
            // values that are not finite: of each wave that brought some in, a lane's keys as bits; whether there are any
            unsigned char marks[2][2][V_PARTS][64];
            alignas(8) unsigned char odd[2][2][V_PARTS];
        } work;
    };
    Line line;
};

template <int NB, bool EXACT, bool BF16, int QT, int PT>
__global__ __launch_bounds__(rows_waves(NB, QT) * 64, rows_waves(NB, QT) == 8 ? 1 : 2) void attention_rows_kernel(AttentionArgs a) {
    using Sh = RowsShared<NB, QT>;
    constexpr int PARTS = rows_waves(NB, QT) / 4, ROWS_WAVE = ROWS_TILE / rows_waves(NB, QT), M = Sh::M, NT = ROWS_WAVE / 16;
    constexpr int KX = NB / PARTS, KV = NB / (2 * PARTS);          // what a lane loads of a key: dwords of K, bytes of V
    __shared__ Sh sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int shift = a.cache.page_log2;
    const int row_bytes = EXACT ? 16 * NB : a.cache.dim >> 1;
    const float scale = a.scale;

    int64_t per;
    const int64_t begin = measure_line(a, sh.line, per), total = uniform(sh.line.total), stop = min(begin + per, total);
    if (tid == 0) a.cuts[share_id(a)].count = 0;
    if (begin >= total) return;
    Segment seg = locate(a, sh.line, begin);
    int64_t at = begin;
    if (seg.start < begin && seg.whole()) {                // the share before has all of it
        at = seg.start + seg.end - seg.begin;
        if (at >= stop) return;
        next_segment(a, seg);
    }

    for (;;) {
        const int head = seg.head / a.head_tiles;
        const int tokens = min(a.tile_tokens, seg.seq.n - (seg.tile << a.tile_log2));
        const int rows = tokens * a.tile_heads;
        bf16x8 qf[QT][NT][NB];
        {
            const AttentionArgs b = arguments();
            Queries<NB, ROWS_TILE, BF16, QT, rows_waves(NB, QT) * 64> queries;
            queries.load(b, seg);
            auto term = [&](auto y) {
                constexpr int Y = decltype(y)::value;
                __syncthreads();
                queries.template store<Y>(b, &sh.q[0][0], Sh::PITCH);
                __syncthreads();
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < NB; ++x)
                        qf[Y][n][x] = *(const bf16x8*)&sh.q[wave * ROWS_WAVE + 16 * n + col][8 * NB * g + 8 * x];
            };
            term(Int<0>());
            if constexpr (QT > 1) term(Int<1>());
            if constexpr (QT > 2) term(Int<2>());
        }

        // the keys that each of the lane's rows sees; those that all of the wave's see, and that any does
        int last[NT], low[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            Row r;
            const bool live = row_of(a, seg, wave * ROWS_WAVE + 16 * n + col, r);
            const int pos = position(seg.seq, r.query);
            last[n] = !live ? -1 : a.causal ? pos : seg.seq.len - 1;
            low[n] = first_key(a, pos);
        }
        const int query0 = seg.tile << a.tile_log2;
        const int first_token = wave * ROWS_WAVE / a.tile_heads;
        const int last_token = min((wave * ROWS_WAVE + ROWS_WAVE - 1) / a.tile_heads, tokens - 1);
        const bool idle = first_token >= tokens;
        const int pos_first = position(seg.seq, query0 + min(first_token, tokens - 1));
        const int pos_last = position(seg.seq, query0 + last_token);
        const int all_to = a.causal ? pos_first : seg.seq.len - 1;
        const int any_to = idle ? -1 : a.causal ? pos_last : seg.seq.len - 1;
        const int all_from = first_key(a, pos_last), any_from = first_key(a, pos_first);

        f32x4 acc[NT][M];
        float top[NT], sum[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n] = -__builtin_inff();
            sum[n] = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) acc[n][m] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        }

        const int unit0 = seg.begin + (int)(at - seg.start);
        const int unit1 = seg.whole() ? seg.end : (int)min((int64_t)seg.end, seg.begin + (stop - seg.start));
        const int units = seg.seq.len == 0 ? unit0 : unit1;
        const int32_t* table = a.table + seg.s * a.table_ld;
        const int last_group = (seg.seq.len - 1) & ~7;
        auto look_up = [&](int unit) { return table[min(UNIT * unit + 8 * (lane & 7), last_group) >> shift]; };
        auto checked = [&](int page) { return page >= 0 && page < (int)a.cache.pages ? page : -1; };
        auto page_of = [&](int pages, int group) { return __builtin_amdgcn_ds_bpermute(4 * group, pages); };

        // what this wave brings in: of K the scores' product k_in of the unit's four, all of each lane's elements or
        // half of them (k_part), and of V 32 keys, a half or a quarter of each lane's elements
        const int k_in = wave / PARTS, k_part = wave % PARTS, j_in = k_in >> 1, t_in = k_in & 1;
        const int v_part = wave % (2 * PARTS);
        uint32_t kc[KX], vc[8][1];
        int kb;
        uint2 vs;
        const Lane<NB, EXACT> my(a, head, col, g);
        auto load = [&](int unit, int pages) {
            const int ok = min(UNIT * unit + 32 * j_in + 8 * (col >> 2), last_group) & ((1 << shift) - 1);
            const int page_k = max(page_of(pages, 4 * j_in + (col >> 2)), 0);
            const uint8_t* codes = in_page(my.k, page_k, a.code_page) + (ok + 4 * t_in) * row_bytes;
            const uint8_t* scales = in_page(my.ks, page_k, a.scale_page) + ok + 4 * t_in + (col & 3);
            if constexpr (KX == 2) {
                const uint2 w = *(const uint2*)(codes + 8 * k_part);
                kc[0] = w.x;
                kc[1] = w.y;
                kb = *scales;
            } else {
                const int more = NB == 8 ? my.half(k_part) : 0;
                const uint4 w = *(const uint4*)(codes + 16 * more);
                kc[0] = w.x;
                kc[1] = w.y;
                kc[2] = w.z;
                kc[3] = w.w;
                kb = scales[more << shift];
            }
            const int ov = min(UNIT * unit + 32 * j_in + 8 * g, last_group) & ((1 << shift) - 1);
            const int page_v = max(page_of(pages, 4 * j_in + g), 0);
            const uint8_t* from = in_page(my.v, page_v, a.code_page) + ov * row_bytes + v_part * KV;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (KV == 1) vc[i][0] = from[i * row_bytes];
                else if constexpr (KV == 2) vc[i][0] = *(const uint16_t*)(from + i * row_bytes);
                else vc[i][0] = *(const uint32_t*)(from + i * row_bytes);
            }
            vs = *(const uint2*)(in_page(my.vs, page_v, a.scale_page) + ov);
        };
        auto store = [&](int buf) {
#pragma unroll
            for (int x = 0; x < KX; ++x) {
                uint32_t u[4];
                widen8(kc[x], scale_operand((uint32_t)kb), u);
                *(uint4*)&sh.work.k[buf][((k_in * NB + k_part * KX + x) * 64 + lane) * 16] = make_uint4(u[0], u[1], u[2], u[3]);
            }
            // values that are not finite: their scale becomes 0, and a mark says where they were
            const bool any = __any(any_odd(vs));
            if (any) {
                const uint32_t out = take_out(vs, vc);
                sh.work.marks[buf][j_in][v_part][lane] = (unsigned char)out;
            }
            if (lane == 0) sh.work.odd[buf][j_in][v_part] = any;
            float sc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sc[i] = scale_of(i < 4 ? vs.x : vs.y, i & 3);
#pragma unroll
            for (int b = 0; b < KV; ++b) {
                uint32_t u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = widen2(vc[i][0], sc[i], b);
#pragma unroll
                for (int second = 0; second < 2; ++second) {
                    const uint32_t sel = second ? 0x07060302u : 0x05040100u;
                    const int k = 2 * (v_part * KV + b) + second;
                    *(uint4*)&sh.work.v[buf][((j_in * M + k) * 64 + lane) * 16] =
                        make_uint4(__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel),
                                   __builtin_amdgcn_perm(u[5], u[4], sel), __builtin_amdgcn_perm(u[7], u[6], sel));
                }
            }
        };

        __syncthreads();                                   // the queries are in registers: their place is free
        int pages = 0, pages1 = 0, pages2 = 0;             // of this unit, the next, the one after
        if (unit0 < units) {
            pages = look_up(unit0);
            pages1 = look_up(min(unit0 + 1, units - 1));
            pages2 = look_up(min(unit0 + 2, units - 1));
            pages = checked(pages);
            pages1 = checked(pages1);
            load(unit0, pages);
            store(unit0 & 1);
            load(min(unit0 + 1, units - 1), pages1);
        }
        for (int unit = unit0; unit < units; ++unit) {
            const int buf = unit & 1, key0 = UNIT * unit;
            __syncthreads();                               // this unit's operands are there, the last one's are read
            pages2 = checked(pages2);
            const int pages3 = look_up(min(unit + 3, units - 1));
            if (unit + 1 < units) store(buf ^ 1);
            load(min(unit + 2, units - 1), pages2);
            __builtin_amdgcn_sched_barrier(0);
            if (key0 <= any_to && key0 + UNIT - 1 >= any_from) {
                const bool whole = key0 + UNIT - 1 <= all_to && key0 >= all_from && !__any(pages < 0);
                // (operands are read AHEAD steps before their products, for a read takes as long as several: the two
                // prompts above took 650 us in place of 702)
                constexpr int AHEAD = 2;
                bf16x8 ring[AHEAD + 1];
                f32x4 s[NT][4];
                auto read_k = [&](int i) { ring[i % (AHEAD + 1)] = *(const bf16x8*)&sh.work.k[buf][(i * 64 + lane) * 16]; };
                auto read_v = [&](int i) { ring[i % (AHEAD + 1)] = *(const bf16x8*)&sh.work.v[buf][(i * 64 + lane) * 16]; };
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) read_k(i);
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i) {
                    const int t = i / NB, x = i % NB;
                    if (i + AHEAD < 4 * NB) read_k(i + AHEAD);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int y = 0; y < QT; ++y)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            s[n][t] = mfma(ring[i % (AHEAD + 1)], qf[y][n][x],
                                           x == 0 && y == 0 ? (f32x4){0.0f, 0.0f, 0.0f, 0.0f} : s[n][t]);
                }
                uint32_t p[NT][2][PT][4];
                bool bad[2] = {false, false};
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) bad[j] = page_of(pages, 4 * j + g) < 0;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = s[n][i >> 2][i & 3];
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = sees(last[n], low[n], key0 + 8 * g, 32 * (i >> 3) + (i & 7)) && !bad[i >> 3]
                                       ? x[i] : -__builtin_inff();
                    }
                    float m = x[0];
#pragma unroll
                    for (int i = 1; i < 16; ++i) m = fmaxf(m, x[i]);
                    m = fmaxf(across(m, MaxF()) * scale, top[n]);
                    if (__any(m > top[n] + GROWTH)) {
                        const float f = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top[n] - m);
                        sum[n] *= f;
#pragma unroll
                        for (int k = 0; k < M; ++k) acc[n][k] *= f;
                        top[n] = m;
                    }
                    const float safe = top[n] == -__builtin_inff() ? 0.0f : top[n];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i], scale, -safe));
                        float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i + 1], scale, -safe));
                        sum[n] += e0 + e1;
#pragma unroll
                        for (int y = 0; y < PT; ++y) {
                            const uint32_t w = p[n][i >> 2][y][i & 3] = pack(e0, e1);
                            e0 -= bf16lo(w);
                            e1 -= bf16hi(w);
                        }
                    }
                }
                typedef typename Sh::Odd Odd;
                const Odd odd = uniform(*(const Odd*)&sh.work.odd[buf][0][0]);
                if (odd) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int part = 0; part < Sh::V_PARTS; ++part) {
                            if (!((odd >> (8 * (j * Sh::V_PARTS + part))) & 1)) continue;
                            const bf16x8 mark = ones(sh.work.marks[buf][j][part][lane]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t seen = 0;
                                int from = key0 + 32 * j + 8 * g;
                                asm volatile("" : "+v"(from)); // (the comparisons made above are not kept for this)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (sees(last[n], low[n], from, i) && !bad[j]) seen |= 1u << i;
                                const f32x4 hit = mfma(mark, ones(seen), (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll
                                    for (int k = 2 * KV * part; k < 2 * KV * (part + 1); ++k)
                                        acc[n][k][i] = hit[i] == 0.0f ? acc[n][k][i] : __builtin_nanf("");
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) read_v(i);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int k = 0; k < M; ++k) {
                        const int i = j * M + k;
                        if (i + AHEAD < 2 * M) read_v(i + AHEAD);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int y = 0; y < PT; ++y)
                                acc[n][k] = mfma(ring[i % (AHEAD + 1)],
                                                 operand(p[n][j][y][0], p[n][j][y][1], p[n][j][y][2], p[n][j][y][3]), acc[n][k]);
                    }
                }
            }
            pages = pages1;
            pages1 = pages2;
            pages2 = pages3;
        }

        const AttentionArgs b = arguments();
        const bool complete = at == seg.start && unit1 == seg.end;
        const Part<NB, ROWS_TILE> part(b, 2 * (int64_t)share_id(b) + (at == begin ? 0 : 1));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = wave * ROWS_WAVE + 16 * n + col;
            Row r;
            const bool live = row_of(b, seg, c, r) && c < rows;
            sum[n] = across(sum[n], AddF());
            // the lane's elements of the row, 8 NB consecutive ones from 8 NB g on
            float o[8 * NB];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < M; ++k) o[M * i + k] = acc[n][k][i];
            if (complete) {
                finish_row<NB, BF16>(b, r, live, 8 * NB * g, o, top[n], sum[n]);
            } else if (live) {
                float* to = part.row(c) + 8 * NB * g;
#pragma unroll
                for (int i = 0; i < 8 * NB; i += 4) store_global(to + i, (f32x4){o[i], o[i + 1], o[i + 2], o[i + 3]});
                if (g == 0) {
                    store_global(part.top(c), top[n]);
                    store_global(part.sum(c), sum[n]);
                }
            }
        }
        const int64_t next = seg.start + (seg.end - seg.begin);
        if (unit1 < seg.end && seg.start >= begin && tid == 0) {
            Cut cut;
            cut.seg = seg;
            cut.slot = 2 * (int64_t)share_id(b) + (at == begin ? 0 : 1);
            cut.count = (int)((next - 1) / per) - share_id(b) + 1;
            cut.pad = 0;
            cut.write(b.cuts + share_id(b));
        }
        at = next;
        if (at >= stop) return;
        next_segment(b, seg);
    }
}

// Joins the parts of the segments that were cut.  Workgroup x: the segment
// that share x began and did not finish, if there is one.  A group of threads
// joins two rows, up to AHEAD parts under way at once.  Where there are no more
// parts than that every group takes rows of its own (512 segments of 128 rows in
// two parts: 17 us less than shared), else workgroup y's groups share two rows.
template <int NB, int NT, bool BF16>
__global__ __launch_bounds__(WAVES * 64) void attention_join_kernel(AttentionArgs a) {
    constexpr int PIECES = 4 * NB, ITEMS = 2 * PIECES, GROUPS = WAVES * 64 / ITEMS, AHEAD = 4;
    __shared__ float o[GROUPS][ITEMS][8 + 1], sums[GROUPS][2], tops[GROUPS][2];
    const Cut cut = a.cuts[blockIdx.x];
    if (cut.count == 0) return;
    const Segment& seg = cut.seg;
    const int rows = min(a.tile_tokens, seg.seq.n - (seg.tile << a.tile_log2)) * a.tile_heads;
    const bool share = cut.count > AHEAD;
    if (2 * (int)blockIdx.y * (share ? 1 : GROUPS) >= rows) return;
    const int item = threadIdx.x % ITEMS, group = threadIdx.x / ITEMS;
    const int pair = share ? blockIdx.y : blockIdx.y * GROUPS + group;
    const int c = 2 * min(pair, 8 * NT - 1) + item / PIECES, d = item % PIECES * 8;
    const int first = share ? group : 0, step = share ? GROUPS : 1;
    float top = -__builtin_inff(), sum = 0.0f, v[8] = {};
    for (int i0 = first; i0 < cut.count; i0 += AHEAD * step) {
        float t[AHEAD], l[AHEAD];
        f32x4 x[AHEAD], y[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = min(i0 + k * step, cut.count - 1);
            const Part<NB, 16 * NT> part(a, i == 0 ? cut.slot : 2 * (int64_t)(blockIdx.x + i));
            t[k] = *part.top(c);                           // (rows that do not exist hold anything and go nowhere)
            l[k] = *part.sum(c);
            x[k] = *(const f32x4*)(part.row(c) + d);
            y[k] = *(const f32x4*)(part.row(c) + d + 4);
        }
        float m = top;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i0 + k * step >= cut.count) t[k] = -__builtin_inff();
            m = fmaxf(m, t[k]);
        }
        const float safe = m == -__builtin_inff() ? 0.0f : m, f = __builtin_amdgcn_exp2f(top - safe);
        sum *= f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= f;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i0 + k * step >= cut.count) continue;
            const float e = __builtin_amdgcn_exp2f(t[k] - safe);
            sum += l[k] * e;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                v[z] += x[k][z] * e;
                v[4 + z] += y[k][z] * e;
            }
        }
        top = m;
    }
    Row r;
    const bool live = row_of(a, seg, c, r) && c < rows;
    if (!share) {
        finish<BF16>(a, r, live && pair < 8 * NT, d, v, top, sum);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) o[group][item][k] = v[k];
    if (d == 0) {
        tops[group][item / PIECES] = top;
        sums[group][item / PIECES] = sum;
    }
    __syncthreads();
    if (group != 0) return;
    const int r2 = item / PIECES;
    float most = tops[0][r2];
#pragma unroll
    for (int w = 1; w < GROUPS; ++w) most = fmaxf(most, tops[w][r2]);
    const float safe = most == -__builtin_inff() ? 0.0f : most;
    float all = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < GROUPS; ++w) {
        const float e = __builtin_amdgcn_exp2f(tops[w][r2] - safe);
        all += sums[w][r2] * e;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += o[w][item][k] * e;
    }
    finish<BF16>(a, r, live, d, v, most, all);
}

// Which kernel, by the rows of a sequence and a head.  Tiles of 16 or 32 rows read
// the cache once each and split the keys over a workgroup's waves; a tile of 128
// reads it once, and every wave passes over all keys.  32 sequences of 8192
// tokens, 8 heads of 128: 36 rows take 108 us in tiles of 32, 171 in one of 128;
// 96 rows 164 and 182; 128 rows 218 and 196.  Heads of 256, tiles of 16: 20 rows
// 140 and 275, 36 rows 306 and 278.
// Few tiles of 128 do not fill the chip, unless their caches are long: 2 heads of
// 800 rows over 1000 tokens take 20 us in tiles of 32, 40 in tiles of 128; 8 heads
// of 1024 rows over 256 tokens 33 and 30.
constexpr int64_t FEW_TILES = 64, FEW_UNITS = 8192;

// What the host chooses from the sizes it knows.
struct Shape {
    int nb, nt, tile_tokens, tile_heads, head_tiles;     // nt 0: attention_rows_kernel
    int64_t shares, part_floats;
};

// capacity: of a sequence, -1 if it is not known: then the shape that needs the larger workspace.
Shape shape_of(const CacheView& c, int64_t tokens, int q_heads, int max_queries, int64_t capacity) {
    Shape s;
    const int group = q_heads / c.heads;
    const int64_t most = max_queries > 0 ? lesser(max_queries, tokens) : tokens;
    s.nb = c.dim <= 64 ? 2 : c.dim <= 128 ? 4 : 8;
    const int64_t rows = most * group;
    const int64_t tiles = tokens * q_heads / ROWS_TILE;
    const bool few = capacity >= 0 && tiles < FEW_TILES && tiles * (capacity / UNIT) < FEW_UNITS;
    if (s.nb < 8) s.nt = rows <= 16 ? 1 : rows <= 96 || few ? 2 : 0;
    else s.nt = rows <= 32 || few ? 1 : 0;                 // (32 rows of 256 elements do not fit the registers)
    const int r = s.nt ? 16 * s.nt : ROWS_TILE;
    s.tile_heads = min(group, r);
    s.head_tiles = (group + r - 1) / r;
    s.tile_tokens = 1;
    while (2 * s.tile_tokens * s.tile_heads <= r) s.tile_tokens *= 2;
    s.shares = s.nt == 1 && s.nb < 8 ? 768 : 512;          // the workgroups that the chip holds at once: 3 or 2 a CU
    s.part_floats = (int64_t)r * (32 * s.nb + 2);
    return s;
}

template <int NB, int NT, bool EXACT>
void launch_main(const AttentionArgs& a, bool bf16, dim3 grid, hipStream_t s) {
    const dim3 block(WAVES * 64);
    if (!bf16) hipLaunchKernelGGL((attention_kernel<NB, NT, EXACT, false, 3, 3>), grid, block, 0, s, a);
    else if (a.cache.rht) hipLaunchKernelGGL((attention_kernel<NB, NT, EXACT, true, 2, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<NB, NT, EXACT, true, 1, 1>), grid, block, 0, s, a);
}

template <int NB, bool EXACT>
void launch_rows(const AttentionArgs& a, bool bf16, dim3 grid, hipStream_t s) {
    const dim3 block(rows_waves(NB, 1) * 64);
    if (!bf16) hipLaunchKernelGGL((attention_rows_kernel<NB, EXACT, false, 3, 3>), grid, dim3(rows_waves(NB, 3) * 64), 0, s, a);
    else if (a.cache.rht) hipLaunchKernelGGL((attention_rows_kernel<NB, EXACT, true, 2, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attention_rows_kernel<NB, EXACT, true, 1, 1>), grid, block, 0, s, a);
}

template <int NB, int NT>     // NT 0: attention_rows_kernel
void launch(const AttentionArgs& a, bool bf16, int shares, bool joined, hipStream_t s) {
    constexpr int ROWS = NT ? 16 * NT : ROWS_TILE;
    const dim3 block(WAVES * 64), grid(shares), join(shares, ROWS / 2);
    const bool exact = a.cache.dim == 32 * NB;
    if constexpr (NT == 0) {
        if (exact) launch_rows<NB, true>(a, bf16, grid, s);
        else launch_rows<NB, false>(a, bf16, grid, s);
    } else {
        if (exact) launch_main<NB, NT, true>(a, bf16, grid, s);
        else launch_main<NB, NT, false>(a, bf16, grid, s);
    }
    if (!joined) return;
    if (bf16) hipLaunchKernelGGL((attention_join_kernel<NB, ROWS / 16, true>), join, block, 0, s, a);
    else hipLaunchKernelGGL((attention_join_kernel<NB, ROWS / 16, false>), join, block, 0, s, a);
}

template <int NB>
void launch(const AttentionArgs& a, int nt, bool bf16, int shares, bool joined, hipStream_t s) {
    if (nt == 0) launch<NB, 0>(a, bf16, shares, joined, s);
    else if (nt == 1) launch<NB, 1>(a, bf16, shares, joined, s);
    else if constexpr (NB < 8) launch<NB, 2>(a, bf16, shares, joined, s);
}

mx_status check_pitches(int64_t ld, int64_t head_ld, int dim) {
    return ld < 0 || head_ld < 0 || (ld && ld < dim) || (head_ld && head_ld < dim) ? MX_ERR_SHAPE : MX_OK;
}

}  // namespace

extern "C" {

int64_t mx_cache_attention_workspace(const mx_cache* cache, mx_dtype qt, int64_t tokens, int32_t q_heads,
                                     int32_t max_queries) {
    CacheView c;
    if (view_cache(cache, c) != MX_OK || q_heads < 1 || q_heads % c.heads || max_queries < 0) return 0;
    if (tokens < 1 || tokens > INT32_MAX / q_heads || (qt != MX_F32 && qt != MX_BF16)) return 0;
    const Shape s = shape_of(c, tokens, q_heads, max_queries, -1);
    return s.shares * (2 * s.part_floats * (int64_t)sizeof(float) + (int64_t)sizeof(Cut));
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
    if (max_queries < 0 || window < 0 || (window && !causal) || !(scale > 0.0f) || !(scale <= MAX_SCALE))
        return MX_ERR_SHAPE;
    if (check_pitches(q_ld, q_head_ld, c.dim) != MX_OK || check_pitches(out_ld, out_head_ld, c.dim) != MX_OK)
        return MX_ERR_SHAPE;
    if (tokens == 0) return MX_OK;
    if (!q || !out || !lengths || (table_pages > 0 && !page_table)) return MX_ERR_NULL;
    if (!workspace) return MX_ERR_NULL;
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
    a.capacity = c.pages ? (int64_t)table_pages * cache->page_size : 0;
    a.lengths = lengths;
    a.scale = scale * LOG2E;
    a.causal = causal != 0;
    // (a window of all that a sequence can hold hides nothing, and costs no masks)
    a.window = window < a.capacity ? window : 0;
    a.sinks = sinks;
    a.out = out;
    a.out_ld = out_ld ? out_ld : row;
    a.out_head_ld = out_head_ld ? out_head_ld : c.dim;
    a.lse = lse;
    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = qt == MX_BF16;
    const Shape shape = shape_of(c, tokens, q_heads, max_queries, a.capacity);
    a.group = q_heads / c.heads;
    a.tile_tokens = shape.tile_tokens;
    a.tile_log2 = __builtin_ctz(shape.tile_tokens);
    a.tile_heads = shape.tile_heads;
    a.head_tiles = shape.head_tiles;
    a.line_heads = c.heads * shape.head_tiles;
    a.code_page = (uint32_t)(c.heads * cache->page_size * (c.dim / 2));
    a.scale_page = (uint32_t)(c.heads * cache->page_size * (c.dim / 32));
    a.cuts = (Cut*)workspace;
    a.parts = (float*)(a.cuts + shape.shares);
    // no more workgroups than there can be work for, and no join where no segment can be long enough to be cut
    const int64_t tiles = (tokens / shape.tile_tokens + lesser(tokens, seqs)) * a.line_heads;
    int64_t longest = greater(ceil_div(a.capacity, UNIT), 1);
    if (a.window) longest = lesser(longest, ((int64_t)a.window + shape.tile_tokens) / UNIT + 2);
    const bool join = longest > WHOLE_UNITS;
    // (short segments go to workgroups of their own as long as there are any: 32 heads of a prompt of 128 tokens take
    // 13 us, 30 with four units a share)
    a.min_units = (int)lesser(greater(longest / 4, 1), MIN_UNITS);
    a.near = join && shape.nt;
    const int shares = shares_of(shape.shares, tiles, longest, a.min_units);
    (void)hipGetLastError();
    if (shape.nb == 2) launch<2>(a, shape.nt, bf16, shares, join, s);
    else if (shape.nb == 4) launch<4>(a, shape.nt, bf16, shares, join, s);
    else launch<8>(a, shape.nt, bf16, shares, join, s);
    return launch_status();
}

}  // extern "C"
