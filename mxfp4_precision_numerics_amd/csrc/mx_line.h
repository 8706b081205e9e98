// mx_line.h -- the attention's work as one line of units: which keys a tile of
// queries sees, and how many units lie before it (gfx950; the same arithmetic
// on the host, for the tests).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_host.h"

namespace mx {

constexpr int UNIT = 64;              // keys that a wave takes at a time

struct Seq {
    int64_t row0;             // its first query row
    int n, len;               // queries, keys
};

// The position of a sequence's i-th query (one past the last: the last key's),
// -1 for all that stand before the first key.  All 32-bit sums here stay within
// 32 bits for any lengths, queries, windows from 0 to 2^31 - 1.
__host__ __device__ __forceinline__ int position(const Seq& q, int i) { return max(q.len - max(q.n - i, 1), -1); }

// A below is what has causal, window, tile_tokens (a power of two) and
// tile_log2.
// The first key that a query at this position (-1 or more) sees.
template <class A>
__host__ __device__ __forceinline__ int first_key(const A& a, int pos) {
    return a.window ? max(pos - a.window + 1, 0) : 0;
}
// Of a sequence's tile i: the first unit that its rows see, and the one after
// the last (a tile whose rows see nothing still has one).
template <class A>
__host__ __device__ __forceinline__ int first_unit(const A& a, const Seq& q, int i) {
    return first_key(a, position(q, i * a.tile_tokens)) / UNIT;
}
template <class A>
__host__ __device__ __forceinline__ int end_unit(const A& a, const Seq& q, int i) {
    const int hi = a.causal ? q.len - max(q.n - i * a.tile_tokens - a.tile_tokens, 0) : q.len;
    return (max(hi, 1) - 1) / UNIT + 1;
}
template <class A>
__host__ __device__ __forceinline__ int tiles_of(const A& a, const Seq& q) {
    return (int)(((uint32_t)q.n + a.tile_tokens - 1) >> a.tile_log2);
}

// Units of a sequence's first x tiles, all of them full ones: sums over the
// tiles of their ends less their begins.  With t tokens a tile, t <= 64 and Q =
// 64 / t, tile i ends at ceil((b + i + 1) / Q) and begins at floor((c + i) / Q)
// for b and c made of the sequence's lengths; with t = 64 C at A + (i + 1) C and
// B + i C.  Ends are 1 at least, begins 0.
__host__ __device__ __forceinline__ int64_t sum_ceil(int64_t y, int q_log2) {       // over j = 1 .. y
    const int64_t w = y >> q_log2, r = y - (w << q_log2);
    return ((w * (w + 1) >> 1) << q_log2) + r * (w + 1);
}
__host__ __device__ __forceinline__ int64_t sum_floor(int64_t y, int q_log2) {      // over j = 0 .. y - 1
    const int64_t w = y >> q_log2, r = y - (w << q_log2);
    return ((w * (w - 1) >> 1) << q_log2) + r * w;
}
template <class A>
__host__ __device__ __forceinline__ int64_t units_before(const A& a, const Seq& q, int x) {
    if (x == 0) return 0;
    if (!a.causal) return (int64_t)x * end_unit(a, q, 0);
    const int64_t at = q.len - q.n, low = at - a.window + 1;
    int64_t units;
    if (a.tile_log2 <= 6) {
        const int q_log2 = 6 - a.tile_log2;
        const int64_t b = (at + a.tile_tokens - 1) >> a.tile_log2;
        units = lesser(x, greater(-b, 0));                      // tiles before the first key: one each
        units += sum_ceil(greater(b + x, 0), q_log2) - sum_ceil(greater(b, 0), q_log2);
        if (a.window) {
            const int64_t c = low >> a.tile_log2;
            units -= sum_floor(greater(c + x, 0), q_log2) - sum_floor(greater(c, 0), q_log2);
        }
    } else {
        const int c_log2 = a.tile_log2 - 6;
        const int64_t n = x, end0 = (at + UNIT - 1) >> 6;
        const int64_t ones = lesser(n, greater((1 - end0) >> c_log2, 0));
        units = ones + (n - ones) * end0 + (((n * (n + 1) - ones * (ones + 1)) >> 1) << c_log2);
        if (a.window) {
            const int64_t begin0 = low >> 6;
            const int64_t none = lesser(n, greater((-begin0 + (1 << c_log2) - 1) >> c_log2, 0));
            units -= (n - none) * begin0 + (((n * (n - 1) - none * (none - 1)) >> 1) << c_log2);
        }
    }
    return units;
}
template <class A>
__host__ __device__ __forceinline__ int64_t units_of(const A& a, const Seq& q) {
    const int tiles = tiles_of(a, q);
    if (tiles == 0) return 0;
    return units_before(a, q, tiles - 1) + end_unit(a, q, tiles - 1) - first_unit(a, q, tiles - 1);
}

// Workgroups of a launch, a multiple of 8 (one of the XCDs each): no more than
// there can be work for, at least min_units of `tiles` times up to `longest`
// units each.
inline int shares_of(int64_t most, int64_t tiles, int64_t longest, int min_units) {
    return (int)lesser(most, ceil_div(ceil_div(tiles * longest, min_units), 8) * 8);
}

}  // namespace mx
