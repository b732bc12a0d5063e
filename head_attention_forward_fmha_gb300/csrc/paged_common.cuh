// paged_common.cuh -- pieces shared by the kernels of the KV cache in pages.
//
// Row i of sequence b lies in page table[b, i / page], row i % page; pages hold a power of
// two of rows, 16 at least, so that the 16 keys from a multiple of 16 on (a granule) lie in
// one page.  A block-table entry outside [0, n_pages) is a page that is not there: its rows
// are not written, not read back and not attended.  A row of the pool has the index
// (page * n_kv_h + head) * page rows + row, below 2^31 (checked on the host); offsets are 64-bit.
#pragma once
#include <climits>
#include "internal.h"
#include "ptx.cuh"

namespace fmha {

// Site codes of the checked build (ptx.cuh), 0x9nn: the cache in pages.
enum PagedCheckSite : unsigned {
    kSitePagedSeq = 0x901,   // paged cache: index of a length, a bound, a start or a block-table entry
    kSitePagedRow = 0x902,   // paged cache: row of a page (and its scale byte)
    kSitePagedIo = 0x903,    // paged append and gather: row of new tokens or of the contiguous output
    kSitePagedQ = 0x904,     // paged attention: query row and its place in shared memory
    kSitePagedKv = 0x905,    // paged attention: shared-memory offset of a key row, or box coordinates
    kSitePagedLds = 0x906,   // paged attention: shared-memory operand of an mma.sync
    kSitePagedTmem = 0x907,  // paged attention: tensor-memory columns of S, P and O
    kSitePagedDesc = 0x908,  // paged attention: K and V stages the MMAs read
    kSitePagedComb = 0x909,  // paged attention: combine or staging buffer
    kSitePagedOut = 0x90a,   // paged attention and merge: output or partial row, sink
};

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const void* tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
        : "memory");
}

// Four E4M3 bytes -> two fp16 pairs (bytes 0 and 1, bytes 2 and 3); exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Entry `slot` of sequence b's block table as it stands there, -1 outside it.  What is loaded is not
// looked at here, so that nothing waits for it before paged_page does.
__device__ __forceinline__ int paged_entry(const PagedCache& c, int batch, int b, int slot, unsigned* status) {
    if (slot < 0 || slot >= c.width || !FMHA_IN_BOUNDS(b >= 0 && b < batch, kSitePagedSeq, status)) return -1;
    return __ldg(c.table + (long long)b * c.width + slot);
}

// The page that an entry names, -1 for one that is not there.
__device__ __forceinline__ int paged_page(const PagedCache& c, int entry) { return (unsigned)entry < (unsigned)c.n_pages ? entry : -1; }

// Pool row of the first key of granule `key` (a multiple of 16) under `head`, given its page; -1 for no page.
__device__ __forceinline__ int paged_row(const PagedCache& c, int page, int head, int key) {
    return page < 0 ? -1 : ((page * c.n_kv_h + head) << c.log_page) + (key & (c.page - 1));
}

__device__ __forceinline__ bool paged_row_ok(const PagedCache& c, long long row) {
    return row >= 0 && row < ((long long)c.n_pages * c.n_kv_h << c.log_page);
}

// Sequence b's first token (its row in a ragged tensor; 0 otherwise) and number of tokens.
// Bounds that do not rise or leave the tensor are cut to what does.
__device__ __forceinline__ void paged_tokens(const PagedTokens& t, int b, int& first, int& n, unsigned* status) {
    first = 0;
    n = t.T;
    if (!t.cu) return;
    if (!FMHA_IN_BOUNDS(b >= 0 && b < t.batch, kSitePagedSeq, status)) {
        n = 0;
        return;
    }
    first = min(max(__ldg(t.cu + b), 0), t.total);
    n = max(0, min(__ldg(t.cu + b + 1), t.total) - first);
}

// Two E4M3 codes, bytes 0 and 2 (LO) or 1 and 3 of w, as bf16 of 2^-120 times their value: the
// code's sign, exponent and mantissa at their places in a bf16, whose exponent bias is 120
// larger.  Subnormal codes come out as bf16 subnormals of the same factor.
template <bool LO>
__device__ __forceinline__ uint32_t e4m3x2_raw(uint32_t w) {
    const uint32_t mag = (LO ? w << 4 : w >> 4) & 0x07F007F0u;
    return ((LO ? w << 8 : w) & 0x80008000u) | mag;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^(byte - 127) in fp32; NaN for 255.
__device__ __forceinline__ float paged_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : byte == 0u ? 0x00400000u : byte << 23);
}

// What brings e4m3x2_raw's values to those of a row under its scale byte: the factor 2^(120 + byte - 127), as a bf16 pair.
// Exact: a code has 4 significant bits, and the product is a bf16 (below 2^-133 it is rounded to one).  The factor is a bf16 up
// to byte 134; above, it is applied in two steps.
struct PagedFactor {
    uint32_t first, second;  // bf16 pairs
    bool two;
};
__device__ __forceinline__ PagedFactor paged_factor(uint32_t byte) {
    PagedFactor f;
    f.two = byte > 134u;
    const uint32_t a = f.two ? 0x7B80u : (byte + 120u) << 7, b = byte == 255u ? 0x7FFFu : byte << 7;
    f.first = a | (a << 16);
    f.second = b | (b << 16);
    return f;
}
// The four codes of a word as two bf16 pairs: bytes 0 and 2, bytes 1 and 3.
__device__ __forceinline__ void paged_values4(uint32_t w, const PagedFactor& f, uint32_t& even, uint32_t& odd) {
    even = mul_bf16x2(e4m3x2_raw<true>(w), f.first);
    odd = mul_bf16x2(e4m3x2_raw<false>(w), f.first);
    if (f.two) {
        even = mul_bf16x2(even, f.second);
        odd = mul_bf16x2(odd, f.second);
    }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// A block's query rows: rows [r0, r0 + n) of sequence b under a KV head, row r being token
// r / group, query head kv_head * group + r % group (so a tile of rows holds few tokens, and a
// causal chunk's early tiles end early).
struct PagedTile {
    int b, first, T, len;  // sequence, its first token, tokens, keys
    int r0, n;             // rows
};

// A tile that one warp has left in shared memory, in every lane of the calling one.  (By shuffles: read as it stands there, a ragged
// decode batch in 8 bits took 248 us in place of 198 and a chunk at hd 256 365 in place of 344.)
__device__ __forceinline__ PagedTile paged_tile_from(const PagedTile* s) {
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    return PagedTile{same(s->b), same(s->first), same(s->T), same(s->len), same(s->r0), same(s->n)};
}

// Row tile `idx` of the launch (tiles of `rows` rows, sequences one after another, each
// sequence's last tile first: under a causal mask it has the most keys; ragged ones with empty slots between).  Warp-collective; all lanes get
// the result; n = 0: past the last tile.
__device__ __forceinline__ PagedTile paged_tile(const PagedFwd& f, int idx, int rows, unsigned* status) {
    const int lane = threadIdx.x & 31;
    PagedTile t{0, 0, 0, 0, 0, 0};
    int tiles = 0;
    if (!f.t.cu) {
        tiles = (f.t.T * f.group + rows - 1) / rows;
        t.b = idx / tiles;
        idx -= t.b * tiles;
        if (t.b >= f.t.batch) return t;
        t.T = f.t.T;
    } else {
        // Sequence b's tiles begin at slot first * group / rows + b: it has as many slots as tiles, or one more.
        int lo = 0, hi = f.t.batch;  // the sequence is one of [lo, hi)
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            bool before = false;
            if (at < hi) {
                int first, n;
                paged_tokens(f.t, at, first, n, status);
                before = (int)((long long)first * f.group / rows) + at <= idx;
            }
            const int reached = __popc(__ballot_sync(0xffffffffu, before));
            if (reached == 0) return t;  // (rows before the first sequence)
            lo += (reached - 1) * step;
            hi = min(hi, lo + step);
            if (step == 1) break;
        }
        t.b = lo;
        paged_tokens(f.t, lo, t.first, t.T, status);
        tiles = (int)(((long long)t.T * f.group + rows - 1) / rows);
        idx -= (int)((long long)t.first * f.group / rows) + lo;
        if (idx >= tiles) {
            t.T = 0;
            return t;
        }
    }
    const int most = min((long long)f.s_k, (long long)f.c.width << f.c.log_page);
    if (FMHA_IN_BOUNDS(t.b < f.t.batch, kSitePagedSeq, status)) t.len = min(max(__ldg(f.seq_lens + t.b), 0), most);
    t.r0 = (tiles - 1 - idx) * rows;
    t.n = min(rows, t.T * f.group - t.r0);
    return t;
}

// The same for blocks whose time goes with their keys: tiles in falling order of the keys that they reach, as far as
// eighths of the longest sequence tell them apart, so that no long block begins when the others end
// (with more sequences looking through them costs more than that: 128 at hd 64, one token each, 30 us, 24 without).
// Gains (in the order of the sequences / so: 16 ragged chunks of up to 512 tokens at hd 128 in 8 bits 210 / 168 us, 4 chunks of 512 in
// bf16 over 200 to 8000 keys 133 / 95, 32 decode steps of ragged sequences at hd 64 in two chunks 38 / 30).
template <int ROWS>
__device__ __forceinline__ PagedTile paged_tile_by_keys(const PagedFwd& f, int idx, unsigned* status) {
    static_assert((ROWS & (ROWS - 1)) == 0, "tiles of a power of two of rows");
    if (f.t.batch > kPagedScan || (f.t.batch == 1 && !f.t.cu)) return paged_tile(f, idx, ROWS, status);
    constexpr int K = 8;
    const int lane = threadIdx.x & 31;
    const int most = min((long long)f.s_k, (long long)f.c.width << f.c.log_page);
    auto keys_of = [&](int b) {
        return b < f.t.batch && FMHA_IN_BOUNDS(b >= 0, kSitePagedSeq, status) ? min(max(__ldg(f.seq_lens + b), 0), most) : 0;
    };
    int top = 0;
    for (int b0 = 0; b0 < f.t.batch; b0 += 32) top = max(top, keys_of(b0 + lane));
    const int width = __reduce_max_sync(0xffffffffu, top) / K + 1;
    // Sequence b0 + lane: its tiles, and how many of them reach X keys at most (the first ones: a tile's last row stands
    // at len - T + ceil(rows up to its end / group) with a causal mask, else all of a sequence's tiles reach len).
    int first = 0, n = 0, len = 0, tiles = 0;
    auto take = [&](int b) {
        first = n = 0;
        if (b < f.t.batch) paged_tokens(f.t, b, first, n, status);
        len = keys_of(b);
        tiles = (int)(((long long)n * f.group + ROWS - 1) / ROWS);
    };
    auto upto = [&](int x) {
        if (x >= len) return tiles;
        return f.causal ? max(0, min(tiles - 1, max(x - len + n, 0) * f.group / ROWS)) : 0;
    };
    int sum[K];
#pragma unroll
    for (int y = 0; y < K; ++y) sum[y] = 0;
    for (int b0 = 0; b0 < f.t.batch; b0 += 32) {
        take(b0 + lane);
        int before = tiles;
#pragma unroll
        for (int y = K - 1; y > 0; --y) {
            const int below = upto(y * width);
            sum[y] += before - below;
            before = below;
        }
        sum[0] += before;
    }
    int at = K;  // the eighth in which the tile lies
#pragma unroll
    for (int y = K - 1; y >= 0; --y) {
        const int all = __reduce_add_sync(0xffffffffu, sum[y]);
        if (at == K) {
            if (idx < all)
                at = y;
            else
                idx -= all;
        }
    }
    PagedTile t{0, 0, 0, 0, 0, 0};
    if (at == K) return t;
    for (int b0 = 0; b0 < f.t.batch; b0 += 32) {
        take(b0 + lane);
        const int end = at == K - 1 ? tiles : upto((at + 1) * width), mine = end - (at > 0 ? upto(at * width) : 0);
        int sums = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int other = __shfl_up_sync(0xffffffffu, sums, s);
            if (lane >= s) sums += other;
        }
        const unsigned past = __ballot_sync(0xffffffffu, sums > idx);
        if (past) {
            const int who = __ffs(past) - 1;
            t.b = b0 + who;
            t.first = __shfl_sync(0xffffffffu, first, who);
            t.T = __shfl_sync(0xffffffffu, n, who);
            t.len = __shfl_sync(0xffffffffu, len, who);
            t.r0 = (__shfl_sync(0xffffffffu, end - 1 + sums - mine, who) - idx) * ROWS;
            t.n = min(ROWS, t.T * f.group - t.r0);
            return t;
        }
        idx -= __shfl_sync(0xffffffffu, sums, 31);
    }
    return t;
}

// Element of q at row r (token r / group, head kvh * group + r % group).
__device__ __forceinline__ long long paged_q_at(const PagedFwd& f, const PagedTile& t, int kvh, int r) {
    const int tok = r / f.group, g = r - tok * f.group;
    return (f.t.cu ? 0 : t.b * f.q_strides[0]) + (long long)(t.first + tok) * f.q_strides[1] + (long long)(kvh * f.group + g) * f.q_strides[2];
}

// Row of o and lse at row r, and its query head.
__device__ __forceinline__ long long paged_out_row(const PagedFwd& f, const PagedTile& t, int kvh, int r, int& head) {
    const int tok = r / f.group;
    head = kvh * f.group + r - tok * f.group;
    return f.t.cu ? (long long)(t.first + tok) * f.n_h + head : ((long long)t.b * f.n_h + head) * f.t.T + tok;
}

// A block's keys, as tiles of `tile` keys: n_head tiles over the first keys [0, n_first), then
// tiles from `start` on over the body [lo, hi), lo >= n_first: of each row's keys the head
// tiles hold those below n_first, the others those from max(n_first, its window) on.  start is lo rounded
// down to `align`.  tile0 and n are the tiles of this block's chunk.
struct PagedKeys {
    int n_first, n_head, lo, hi, start;
    int tile0, n;
    __device__ __forceinline__ int key(int j, int tile) const {
        j += tile0;
        return j < n_head ? j * tile : start + (j - n_head) * tile;
    }
    __device__ __forceinline__ bool head(int j) const { return j + tile0 < n_head; }
    // keys of tile j that some row may attend: [from, to)
    __device__ __forceinline__ int from(int j) const { return head(j) ? 0 : lo; }
    __device__ __forceinline__ int to(int j) const { return head(j) ? n_first : hi; }
};

__device__ __forceinline__ PagedKeys paged_keys(const PagedFwd& f, const PagedTile& t, int split, int tile, int align) {
    PagedKeys k;
    const int p0 = t.len - t.T + t.r0 / f.group, p1 = t.len - t.T + (t.r0 + t.n - 1) / f.group;  // first and last row's positions
    k.hi = f.causal ? min(t.len, p1 + 1) : t.len;
    k.hi = max(k.hi, 0);
    k.n_first = f.window > 0 ? min(f.n_first, k.hi) : 0;
    k.lo = f.window > 0 ? max(k.n_first, p0 - f.window + 1) : 0;
    k.lo = min(k.lo, k.hi);
    k.n_head = (k.n_first + tile - 1) / tile;
    k.start = k.lo / align * align;
    const int body = k.hi > k.lo ? (k.hi - k.start + tile - 1) / tile : 0;
    const int all = k.n_head + body;
    k.tile0 = (int)min((long long)all, (long long)split * f.chunk_tiles);
    k.n = split == f.n_splits - 1 ? all - k.tile0 : min(all - k.tile0, f.chunk_tiles);
    return k;
}

// Keys [lo, hi] of the body and [0, fhi] of the head that row r of the tile attends.
__device__ __forceinline__ void paged_row_keys(const PagedFwd& f, const PagedTile& t, const PagedKeys& k, int r, int& lo, int& hi, int& fhi) {
    lo = INT_MAX;
    hi = fhi = -1;
    if (r >= t.r0 + t.n) return;
    const int p = t.len - t.T + r / f.group;
    lo = k.lo;
    hi = k.hi - 1;
    if (f.causal) hi = min(hi, p);
    if (f.window > 0) lo = max(lo, p - f.window + 1);
    fhi = min(hi, k.n_first - 1);
}

// End of a row: finish_row, but where a NaN score has made the sum NaN, so are O and LSE, for
// any number of chunks (-inf would mark an empty chunk).
__device__ __forceinline__ void paged_finish(float m, float l, float sink_l2, float& inv, float& lse) {
    finish_row(m, l, sink_l2, inv, lse);
    if (l != l) inv = lse = l;
}

// Output of a block whose rows attend no key of their chunk: O = 0 and LSE = -inf, or the row's
// sink in a final output.  Of a partial only the LSE is written: the merge reads no O with it.
__device__ __forceinline__ void paged_write_empty(const PagedFwd& f, const PagedTile& t, int kvh, int split, int col0, int ncol) {
    const int per_row = ncol / 8;
    for (int i = threadIdx.x; i < t.n * per_row; i += blockDim.x) {
        const int r = i / per_row, c = i - r * per_row;
        int head;
        const long long row = paged_out_row(f, t, kvh, t.r0 + r, head);
        if (!FMHA_IN_BOUNDS(row >= 0 && row < f.rows && head < f.n_h && split < f.n_splits && col0 + c * 8 + 8 <= f.c.hd, kSitePagedOut, f.status))
            continue;
        if (f.n_splits == 1) *reinterpret_cast<uint4*>(f.o + row * f.c.hd + col0 + c * 8) = make_uint4(0u, 0u, 0u, 0u);
        if (c == 0 && col0 == 0) {
            if (f.n_splits == 1)
                f.lse[row] = f.sink ? __ldg(f.sink + head) : -INFINITY;
            else
                f.lse_part[split * f.rows + row] = -INFINITY;
        }
    }
}

}  // namespace fmha
