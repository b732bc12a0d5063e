// first_keys.cuh -- a sliding window with a few first keys that stay visible.
//
// Row t at position p attends key j iff j <= p (causal) and (j > p - window or
// j < n_first).  For every row of a block this is the union of two intervals
// that lie in two disjoint ranges of keys: [0, n_first) and [kv_begin, s_k),
// kv_begin = max(n_first, first key of row 0's window).  The kernels walk tiles of a
// virtual key axis, the first range rounded up to whole tiles and then the
// second, and each tile meets one interval per row, as without first keys.
//
// The kernels' argument structs say at compile time whether there are first
// keys (kFirst), so that the kernels without them carry none of this.
#pragma once

namespace fmha {

// The first-key part and the window part of one chunk.
struct ChunkRange {
    int f_lo, f_tiles;  // first keys: tiles of `tile` keys from key f_lo on
    int c_lo, c_hi;     // window part: keys [c_lo, c_hi)
};

template <class A>
__device__ __forceinline__ ChunkRange chunk_range(const A& a, int split, int tile) {
    ChunkRange r;
    if constexpr (A::kFirst) {
        const int v_lo = split * a.kv_chunk, v_hi = v_lo + a.kv_chunk;
        r.f_lo = v_lo;
        r.f_tiles = max(0, (min(v_hi, a.first_span) - v_lo) / tile);
        r.c_lo = a.kv_begin + max(0, v_lo - a.first_span);
        r.c_hi = min(a.s_k, a.kv_begin + max(0, v_hi - a.first_span));
    } else {
        r.f_lo = 0;
        r.f_tiles = 0;
        r.c_lo = a.kv_begin + split * a.kv_chunk;
        r.c_hi = min(a.s_k, r.c_lo + a.kv_chunk);
    }
    return r;
}

// First key of tile j of a block whose window part starts at k_lo.
template <class A>
__device__ __forceinline__ int tile_key(const A&, const ChunkRange& r, int k_lo, int j, int tile) {
    if constexpr (A::kFirst)
        if (j < r.f_tiles) return r.f_lo + j * tile;
    return k_lo + (j - (A::kFirst ? r.f_tiles : 0)) * tile;
}

// One past the last key that tile j may load for a reason (index checks).
template <class A>
__device__ __forceinline__ int tile_end(const A& a, const ChunkRange& r, int k_hi, int j) {
    if constexpr (A::kFirst)
        if (j < r.f_tiles) return a.n_first;
    return k_hi;
}

}  // namespace fmha
