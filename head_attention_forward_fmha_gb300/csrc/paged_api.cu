// paged_api.cu -- the C entry points of the KV cache in pages (declared in include/fmha.h):
// checks of the arguments, the attention's plan, launches on the caller's stream.
#include <algorithm>
#include <climits>
#include <cmath>

#include "fmha.h"
#include "internal.h"

namespace {

using namespace fmha;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMost = 1 << 30;  // sizes and positions: differences of two stay within 32 bits

// The pool and its block table, whose pointers check_cache_pointers looks at.
int check_cache(int batch, int n_kv_h, int hd, int page, int n_pages, int width, PagedCache* c) {
    if (hd != 64 && hd != 128 && hd != 256 && hd != 512)
        return fail(FMHA_ERR_HEADDIM, "hd=%d: supported head dims are 64, 128, 256, 512", hd);
    if (n_kv_h < 1) return fail(FMHA_ERR_HEADS, "n_kv_h=%d must be >= 1", n_kv_h);
    if (page < 16 || page > 65536 || (page & (page - 1)))
        return fail(FMHA_ERR_SHAPE, "page=%d must be a power of two from 16 to 65536", page);
    if (batch < 0 || n_pages < 0 || width < 0) return fail(FMHA_ERR_SHAPE, "negative size (batch=%d n_pages=%d table width=%d)", batch, n_pages, width);
    if ((double)n_pages * n_kv_h * page > (double)(INT_MAX - 65536))  // rows are counted in 32 bits, one page past the end too
        return fail(FMHA_ERR_SHAPE, "n_pages * n_kv_h * page = %.0f rows exceed 2^31 - 65537", (double)n_pages * n_kv_h * page);
    c->n_kv_h = n_kv_h;
    c->hd = hd;
    c->page = page;
    c->log_page = 0;
    while (1 << c->log_page < page) ++c->log_page;
    c->n_pages = n_pages;
    c->width = width;
    return FMHA_OK;
}

int check_cache_pointers(const PagedCache& c) {
    if (!c.k_pages || !c.v_pages || !c.table) return fail(FMHA_ERR_NULL, "pages and block table must be non-NULL");
    if ((c.k_scales == nullptr) != (c.v_scales == nullptr)) return fail(FMHA_ERR_NULL, "k_scales and v_scales are given together or not at all");
    if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.k_scales, 16) || !aligned(c.v_scales, 16) || !aligned(c.table, 4))
        return fail(FMHA_ERR_ALIGN, "pages and scales must be 16-byte, the block table 4-byte aligned");
    return FMHA_OK;
}

// New tokens: `total` of them with bounds, else T for each sequence.
int check_tokens(int batch, int T, int total, bool ragged, int heads, PagedTokens* t) {
    if (T < 0 || total < 0) return fail(FMHA_ERR_SHAPE, "negative size (T=%d total=%d)", T, total);
    const double tokens = ragged ? (double)total : (double)batch * T;
    if (tokens * heads > kMost) return fail(FMHA_ERR_SHAPE, "%.0f tokens of %d heads are too many rows", tokens, heads);
    t->batch = batch;
    t->T = ragged ? std::min(T, total) : T;  // a sequence has no more than there are
    t->total = ragged ? total : 0;
    return FMHA_OK;
}

int check_strides(const long long* s, const char* name) {
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % 8 != 0)
            return fail(FMHA_ERR_SHAPE, "%s: strides must be multiples of 8 elements, not negative (got %lld)", name, s[i]);
    return FMHA_OK;
}

// Rows per KV head from which on the tensor-core kernel is taken, the decode kernel below.  Measured on
// 8 ragged sequences of up to 8192 keys and 8 KV heads (us, decode kernel / tensor cores):
//   bf16   hd  64   16 rows  21 / 30   24 rows  32 / 32     codes  16 rows   28 / 41   24 rows   48 /  41
//   bf16   hd 128   16 rows  28 / 34   24 rows  43 / 34     codes  16 rows   32 / 47   24 rows   52 /  48
//   bf16   hd 256    8 rows  43 / 50   16 rows  51 / 51     codes  16 rows   64 / 78   24 rows  105 /  81
//   bf16   hd 512    8 rows  95 / 110  10 rows 151 / 111    codes  24 rows  157 / 174  32 rows  195 / 174
// The decode kernel reads the keys once for every 16 rows (8 at hd 512).
int tc_min_rows(int hd, bool codes) { return hd == 512 ? (codes ? 25 : 9) : hd == 256 && !codes ? 9 : 17; }

// Estimated time of a key tile in a block of the tensor-core kernel, `rows` being those of a sequence under a KV head
// (measured: blocks of one and of two row tiles at hd 64 and 128, chunks of 512 tokens and 64 rows at hd 256 and 512).
double tc_tile_us(int hd, bool codes, long long rows) {
    if (hd <= 128) return (rows > 128 ? (hd == 64 ? 1.6 : 1.75) : (hd == 64 ? 1.05 : 1.1)) * (codes ? 1.4 : 1.0);  // tiles of 128 keys
    return hd == 256 ? (codes ? 1.7 : 0.75) : codes ? 2.4 : 1.25;                                                  // of 64
}

// Kernel, row tiles and chunks of an attention call.  f->t.T is the number of new tokens of every
// sequence, or with bounds the most that one has; wanted: the number of chunks asked for, 0 for the library's
// choice.  Nothing is lost if a sequence has more tokens or keys than said here: row tiles are counted by
// the tokens that there are, and a sequence's last chunk takes what the others leave.
struct PagedPlan {
    bool tc;
    int rows;  // query rows per thread block
    long long row_tiles;
};

PagedPlan plan_paged(PagedFwd* f, bool ragged, bool codes, int wanted) {
    PagedPlan p;
    const int hd = f->c.hd;
    const long long most = (long long)f->group * f->t.T;  // rows of a sequence under a KV head
    const int path = kernel_path();
    p.tc = path ? path >= 2 : most >= tc_min_rows(hd, codes);
    p.rows = p.tc ? paged_tc_rows(hd) : paged_decode_rows(hd, most);
    const long long tokens = ragged ? f->t.total : (long long)f->t.batch * f->t.T;
    p.row_tiles = !ragged ? f->t.batch * ((most + p.rows - 1) / p.rows)
                  : f->t.batch > kPagedScan ? tokens * f->group / p.rows + f->t.batch  // slots of paged_tile
                                            : std::min(tokens * f->group, (tokens * f->group + (long long)f->t.batch * (p.rows - 1)) / p.rows);
    f->row_tiles = (int)std::min<long long>(p.row_tiles, INT_MAX);
    const int tile = p.tc ? paged_tc_kv_tile(hd) : paged_decode_kv_tile(hd, codes);
    long long span = f->s_k;
    if (f->window > 0) span = std::min<long long>(span, (long long)f->n_first + f->window + std::min<long long>(f->t.T, p.rows) + 2 * tile);
    const long long tiles = std::max(1LL, (span + tile - 1) / tile);
    long long n = wanted;
    if (n <= 0) {
        // The number of chunks with the least estimated time, over the lengths that a batch may have: sequences of
        // s_k keys each, and (counted more without a window) lengths spread evenly up to it, where a sequence of n chunks
        // fills (n + 1) / 2 blocks with n / 2 blocks' work on average.
        const bool one = p.tc || hd == 512 || (codes && p.rows == 16);  // block per SM
        const double slots = sm_count() * (one ? 1.0 : 2.0);
        const double units = (double)std::max(1LL, p.row_tiles) * f->c.n_kv_h * (p.tc && hd == 512 ? 2 : 1);
        const double row_bytes = codes ? hd + 1.0 : 2.0 * hd;
        // what a decode block takes in at most, bytes a us, and what all of them do
        const double rate1 = codes ? (hd == 64 ? 11e3 : 20e3) : hd == 64 ? 26e3 : 36e3, rates = codes ? 5.6e6 : 6.8e6;
        const double parts_us = (double)f->rows * hd * 8.0 / 8e6;  // one chunk's partials, written and read
        double best = 1e300;
        const long long most_n = std::min<long long>(tiles, 64);
        for (long long c = 1; c <= most_n; c += c < 8 ? 1 : c < 32 ? 2 : 8) {
            const long long mine = (tiles + c - 1) / c;  // tiles of a block
            const double bytes = (double)mine * tile * 2.0 * row_bytes;
            double us[2];
            for (int ragged_lens = 0; ragged_lens < 2; ++ragged_lens) {
                const double blocks = units * (double)(ragged_lens ? c + 1 : 2 * c) / 2.0, ratio = blocks / slots;
                const double fixed = p.tc ? (hd == 512 ? 10.0 : 8.0) : 4.0;
                double body = p.tc ? (double)mine * tc_tile_us(hd, codes, most) : bytes / rate1;
                if (ragged_lens) {
                    const double waits = ratio > 1.0 ? (fixed + body) * 0.2 : 0.0;  // for the last block to end, long ones first
                    double work = ratio * fixed + units / slots * (double)c * body / 2.0;
                    if (!p.tc) work = std::max(work, ratio * 2.0 + fixed + units * (double)c / 2.0 * bytes / rates);
                    us[1] = std::max(fixed + body, work + waits);
                } else {
                    if (!p.tc) body = std::max(body, bytes * std::min(slots, blocks) / rates);
                    us[0] = std::max(1.0, ratio + 0.5 * (std::ceil(ratio) - ratio)) * (fixed + body);
                }
            }
            const double even = f->t.batch == 1 ? 1.0 : f->window > 0 ? 0.8 : 0.25;  // a window makes long sequences alike
            double t = even * us[0] + (1.0 - even) * us[1];
            if (c > 1) t += 3.0 + 0.05 * (double)c + 0.2 * (double)std::max(0LL, c - 16) + parts_us * (double)c;  // the merge
            if (t < best * 0.99) {
                best = t;
                n = c;
            }
        }
    }
    n = std::max(1LL, std::min<long long>({n, tiles, 64}));
    // partials of at most 1 GiB
    while (n > 1 && (double)n * f->rows * (hd + 1) * 4 > (double)(1 << 30)) --n;
    f->chunk_tiles = (int)((tiles + n - 1) / n);
    f->n_splits = (int)((tiles + f->chunk_tiles - 1) / f->chunk_tiles);
    return p;
}

// At most s_k keys; a window that holds them all is none.
void bound_keys(PagedFwd* f, int s_k, int window, int n_first) {
    f->s_k = s_k;
    f->window = window >= s_k ? 0 : window;
    f->n_first = f->window > 0 ? std::min(n_first, s_k) : 0;
}

int check_fwd(int batch, int T, int total, bool ragged, int n_h, int n_kv_h, int hd, int page, int n_pages, int width, int s_k, float scale,
              int window, int n_first, int causal, int n_splits, PagedFwd* f) {
    *f = PagedFwd{};
    int rc = check_cache(batch, n_kv_h, hd, page, n_pages, width, &f->c);
    if (rc) return rc;
    if (n_h < 1 || n_h % n_kv_h != 0)
        return fail(FMHA_ERR_HEADS, "n_h=%d n_kv_h=%d: need n_h, n_kv_h >= 1 and n_h %% n_kv_h == 0", n_h, n_kv_h);
    rc = check_tokens(batch, T, total, ragged, n_h, &f->t);
    if (rc) return rc;
    if (s_k < 0 || s_k > kMost) return fail(FMHA_ERR_SHAPE, "s_k=%d must lie in [0, 2^30]", s_k);
    if (window < 0 || n_first < 0) return fail(FMHA_ERR_SHAPE, "window=%d and n_first=%d must be >= 0", window, n_first);
    if (causal != 0 && causal != 1) return fail(FMHA_ERR_SHAPE, "causal must be 0 or 1 (got %d)", causal);
    if (n_splits < 0) return fail(FMHA_ERR_SHAPE, "n_splits=%d must be >= 0", n_splits);
    f->scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (!std::isfinite(f->scale_log2)) return fail(FMHA_ERR_SHAPE, "scale must be finite");
    f->n_h = n_h;
    f->group = n_h / n_kv_h;
    f->rows = (ragged ? (long long)total : (long long)batch * T) * n_h;
    // keys that there are at most
    bound_keys(f, n_pages == 0 ? 0 : (int)std::min<long long>(s_k, (long long)width * page), window, n_first);
    f->causal = causal;
    return FMHA_OK;
}

}  // namespace

extern "C" {

int fmha_paged_append(const struct fmha_paged_append_args* x) try {
    if (!x) return fail(FMHA_ERR_NULL, "fmha_paged_append: NULL arguments");
    PagedAppend a = {};
    int rc = check_cache(x->batch, x->n_kv_h, x->hd, x->page, x->n_pages, x->table_width, &a.c);
    if (rc) return rc;
    rc = check_tokens(x->batch, x->T, x->total, x->cu_q != nullptr, x->n_kv_h, &a.t);
    if (rc) return rc;
    if ((rc = check_strides(x->k_strides, "k")) || (rc = check_strides(x->v_strides, "v"))) return rc;
    if (x->batch == 0 || (x->cu_q ? x->total : x->T) == 0 || x->n_pages == 0 || x->table_width == 0) return FMHA_OK;
    a.c.k_pages = x->k_pages;
    a.c.v_pages = x->v_pages;
    a.c.k_scales = static_cast<uint8_t*>(x->k_scales);
    a.c.v_scales = static_cast<uint8_t*>(x->v_scales);
    a.c.table = x->block_table;
    if ((rc = check_cache_pointers(a.c))) return rc;
    if (!x->k || !x->v || !x->start) return fail(FMHA_ERR_NULL, "k, v and start must be non-NULL");
    if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(x->start, 4) || !aligned(x->cu_q, 4))
        return fail(FMHA_ERR_ALIGN, "k and v must be 16-byte, start and cu_q 4-byte aligned");
    a.t.cu = x->cu_q;
    a.k = static_cast<const __nv_bfloat16*>(x->k);
    a.v = static_cast<const __nv_bfloat16*>(x->v);
    for (int i = 0; i < 3; ++i) {
        a.k_strides[i] = x->k_strides[i];
        a.v_strides[i] = x->v_strides[i];
    }
    a.start = x->start;
    a.status = device_status_word();
    if (!a.status) return fail(FMHA_ERR_LAUNCH, "cannot resolve the device status word");
    const cudaError_t e = launch_paged_append(a, x->stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged append kernel launch");
    return FMHA_OK;
} catch (...) {
    return fail(FMHA_ERR_LAUNCH, "unexpected host exception in fmha_paged_append");
}

int fmha_paged_gather(const struct fmha_paged_gather_args* x) try {
    if (!x) return fail(FMHA_ERR_NULL, "fmha_paged_gather: NULL arguments");
    PagedGather a = {};
    int rc = check_cache(x->batch, x->n_kv_h, x->hd, x->page, x->n_pages, x->table_width, &a.c);
    if (rc) return rc;
    if (x->rows < 0) return fail(FMHA_ERR_SHAPE, "rows=%d must be >= 0", x->rows);
    if ((double)x->batch * x->n_kv_h * x->rows > kMost) return fail(FMHA_ERR_SHAPE, "too many rows");
    if (x->batch == 0 || x->rows == 0 || x->n_pages == 0 || x->table_width == 0) return FMHA_OK;
    a.c.k_pages = const_cast<void*>(x->k_pages);
    a.c.v_pages = const_cast<void*>(x->v_pages);
    a.c.k_scales = static_cast<uint8_t*>(const_cast<void*>(x->k_scales));
    a.c.v_scales = static_cast<uint8_t*>(const_cast<void*>(x->v_scales));
    a.c.table = x->block_table;
    if ((rc = check_cache_pointers(a.c))) return rc;
    if (!x->seq_lens || !x->k || !x->v) return fail(FMHA_ERR_NULL, "seq_lens, k and v must be non-NULL");
    if (!aligned(x->k, 16) || !aligned(x->v, 16) || !aligned(x->seq_lens, 4) || !aligned(x->start, 4))
        return fail(FMHA_ERR_ALIGN, "k and v must be 16-byte, seq_lens and start 4-byte aligned");
    a.start = x->start;
    a.seq_lens = x->seq_lens;
    a.k = static_cast<__nv_bfloat16*>(x->k);
    a.v = static_cast<__nv_bfloat16*>(x->v);
    a.batch = x->batch;
    a.rows = x->rows;
    a.status = device_status_word();
    if (!a.status) return fail(FMHA_ERR_LAUNCH, "cannot resolve the device status word");
    const cudaError_t e = launch_paged_gather(a, x->stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged gather kernel launch");
    return FMHA_OK;
} catch (...) {
    return fail(FMHA_ERR_LAUNCH, "unexpected host exception in fmha_paged_gather");
}

int fmha_fwd_paged_plan(int batch, int T, int total, int n_h, int n_kv_h, int hd, int page, int s_k, int window, int n_first, int causal,
                        int ragged, int codes, int n_splits) try {
    if ((ragged != 0 && ragged != 1) || (codes != 0 && codes != 1))
        return fail(FMHA_ERR_SHAPE, "ragged and codes must be 0 or 1 (got %d and %d)", ragged, codes);
    PagedFwd f;
    const int width = page > 0 && s_k > 0 ? (int)(((long long)s_k + page - 1) / page) : 1;
    const int rc = check_fwd(batch, T, total, ragged != 0, n_h, n_kv_h, hd, page, 1, width, s_k, 1.f, window, n_first, causal, n_splits, &f);
    if (rc) return rc;
    if (f.rows == 0) return 1;
    plan_paged(&f, ragged != 0, codes != 0, n_splits);
    return f.n_splits;
} catch (...) {
    return fail(FMHA_ERR_LAUNCH, "unexpected host exception in fmha_fwd_paged_plan");
}

int fmha_fwd_paged(const struct fmha_fwd_paged_args* x) try {
    if (!x) return fail(FMHA_ERR_NULL, "fmha_fwd_paged: NULL arguments");
    PagedFwd f;
    const bool ragged = x->cu_q != nullptr;
    int rc = check_fwd(x->batch, x->T, x->total, ragged, x->n_h, x->n_kv_h, x->hd, x->page, x->n_pages, x->table_width, x->s_k, x->scale,
                       x->window, x->n_first, x->causal, x->n_splits, &f);
    if (rc) return rc;
    if ((rc = check_strides(x->q_strides, "q"))) return rc;
    if (f.rows == 0 || x->batch == 0) return FMHA_OK;
    f.c.k_pages = const_cast<void*>(x->k_pages);
    f.c.v_pages = const_cast<void*>(x->v_pages);
    f.c.k_scales = static_cast<uint8_t*>(const_cast<void*>(x->k_scales));
    f.c.v_scales = static_cast<uint8_t*>(const_cast<void*>(x->v_scales));
    f.c.table = x->block_table;
    if (f.s_k > 0 && (rc = check_cache_pointers(f.c))) return rc;
    if (!x->q || !x->seq_lens || !x->o || !x->lse) return fail(FMHA_ERR_NULL, "q, seq_lens, o and lse must be non-NULL");
    if (!aligned(x->q, 16) || !aligned(x->o, 16) || !aligned(x->lse, 4) || !aligned(x->seq_lens, 4) || !aligned(x->cu_q, 4) || !aligned(x->sink, 4))
        return fail(FMHA_ERR_ALIGN, "q and o must be 16-byte, lse, seq_lens, cu_q and sink 4-byte aligned");
    f.t.cu = x->cu_q;
    f.q = static_cast<const __nv_bfloat16*>(x->q);
    for (int i = 0; i < 3; ++i) f.q_strides[i] = x->q_strides[i];
    f.seq_lens = x->seq_lens;
    f.sink = x->sink;
    f.o = static_cast<__nv_bfloat16*>(x->o);
    f.lse = x->lse;
    const bool codes = x->k_scales != nullptr;
    PagedPlan p = plan_paged(&f, ragged, codes, x->n_splits);
    if (f.n_splits > 1 && f.s_k < x->s_k) {
        // The workspace has been sized by fmha_fwd_paged_plan, which does not know how many keys the block table holds:
        // no more chunks than it says for s_k.
        PagedFwd told = f;
        bound_keys(&told, x->s_k, x->window, x->n_first);
        plan_paged(&told, ragged, codes, x->n_splits);
        if (f.n_splits > told.n_splits) p = plan_paged(&f, ragged, codes, told.n_splits);
    }
    if ((double)p.row_tiles * f.c.n_kv_h * 2 > INT_MAX) return fail(FMHA_ERR_SHAPE, "too many query rows");
    if (f.n_splits > 1) {
        const size_t need = (size_t)f.n_splits * f.rows * (f.c.hd + 1) * 4;
        if (!x->workspace || x->workspace_bytes < need)
            return fail(FMHA_ERR_WORKSPACE, "fmha_fwd_paged: %zu bytes of workspace needed for %d chunks, %zu given", need, f.n_splits,
                        x->workspace ? x->workspace_bytes : (size_t)0);
        if (!aligned(x->workspace, 16)) return fail(FMHA_ERR_ALIGN, "workspace must be 16-byte aligned");
        f.o_part = static_cast<float*>(x->workspace);
        f.lse_part = f.o_part + (size_t)f.n_splits * f.rows * f.c.hd;
    }
    f.status = device_status_word();
    if (!f.status) return fail(FMHA_ERR_LAUNCH, "cannot resolve the device status word");
    cudaError_t e = p.tc ? launch_paged_tc(f, x->stream) : launch_paged_decode(f, p.rows, x->stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged attention kernel launch");
    if (f.n_splits > 1) {
        e = launch_paged_merge(f, x->stream);
        if (e != cudaSuccess) return cuda_fail(e, "paged merge kernel launch");
    }
    return FMHA_OK;
} catch (...) {
    return fail(FMHA_ERR_LAUNCH, "unexpected host exception in fmha_fwd_paged");
}

}  // extern "C"
