// paged_tc_kernel.cu -- attention over a cache in pages for tiles of 128 query rows, on the
// tcgen05 tensor cores.
//
// One thread block owns up to two row tiles A and B of 128 query rows (one at hd 256 and 512) of one
// sequence under one KV head, and one chunk of the sequence's key tiles:
//   S = Q_t K_j^T    tcgen05.mma M = 128, N = BN, K = hd    (both operands from shared memory)
//   O_t += P V_j     tcgen05.mma M = 128, N = hd, K = BN    (P from tensor memory, written over S)
// At hd 512 two blocks share a row tile: each computes all of S and one 256-column half of O, and
// K's single stage is refilled in two column chunks, each as soon as the MMAs have read it.
//
// The work is a chain of units u, a row tile and a key tile each: A(0) B(0) A(1) B(1) ... or, with one row
// tile, A(0) A(1) ....  Unit u's S and P live in slot u % 2 of tensor memory; the MMA warp issues
//   QK(0) QK(1) | PV(0) QK(2) | PV(1) QK(3) | ...
// and PV(u) before QK(u + 2) in one slot is all the order that the slot needs, since MMAs
// complete in order.  While the softmax of one slot runs, the tensor cores work on the other.
//
// Warp roles (13 warps): with two row tiles 0..3 and 4..7 softmax and epilogue of A and B (one row
// per thread), 8 MMA issue and tensor memory, 9..12 loaders; with one 0..3, 4, and 5..12.  The
// loaders look the pages up in the block table, two tiles ahead, and copy bf16 rows into the
// swizzled operand layout (cp.async, 16 bytes each, zeros for keys that no row of the block attends, so that
// nothing stale is multiplied), or load codes, expand them to bf16 (paged_common.cuh) and
// store those.  Expanded columns 1 and 2 of each four change places: Q is stored the same way, and
// O's columns are put right in the epilogue.
//
// Softmax: scores against a reference, the maximum of the first tile in which the row attends a key.  P in
// bf16 and its fp32 sum have the exponent range for what follows, so the reference moves (and O
// is rescaled) only where a tile's sum passes 2^40: no maximum is taken otherwise.
#include <atomic>
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

template <int HD>
struct PTCfg {
    static constexpr int BM = 128;
    static constexpr int NRT = HD <= 128 ? 2 : 1;         // row tiles
    static constexpr int BN = HD <= 128 ? 128 : 64;       // keys per tile
    static constexpr int HDV = HD == 512 ? 256 : HD;      // columns of O per block
    static constexpr int PARTS = HD / HDV;                // blocks per row tile
    static constexpr int STG = HD == 512 ? 1 : 2;         // K and V stages
    static constexpr int NKC = HD == 512 ? 2 : 1;         // column chunks of a K tile, each with barriers of its own
    static constexpr int KCH = HD / NKC;
    static constexpr int SW = 4 * NRT;                    // softmax warps
    static constexpr int LW = 12 - SW;                    // loader warps
    static constexpr int LT = 32 * LW;
    static constexpr int THREADS = 13 * 32;
    static constexpr int Q_TILE = BM * HD * 2;
    static constexpr int Q_BYTES = NRT * Q_TILE;
    static constexpr int K_TILE = BN * HD * 2;
    static constexpr int V_TILE = BN * HDV * 2;
    static constexpr int O_COL = 2 * BN;                  // tensor memory: two S slots, then O of each row tile
    static constexpr int TMEM_COLS = 512;
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + STG * K_TILE;
    static constexpr int OFF_BAR = OFF_V + STG * V_TILE;
    static constexpr int N_BARS = 1 + 2 * STG * NKC + 2 * STG + 6 + 1;
    static constexpr int NEED = 1024 + OFF_BAR + N_BARS * 8 + 16;
    static constexpr int SMEM = NEED < 120000 ? 120000 : NEED;  // one block per SM: each takes all of tensor memory
    static_assert(O_COL + NRT * HDV <= TMEM_COLS, "S and O fit in tensor memory");
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// What a loader thread needs of one key tile: this lane's granule of 16 keys (lane < BN / 16) as a row of the
// pool, -1 if no row attends a key of it or its page is not there; and the range of keys that count.
struct TileRows {
    int row, from, to;  // from, to: relative to the tile's first key
};

// One loader thread's share of a tile of codes: N pieces of 16 columns, PPR per key, going round the LT threads.
template <int N, int PPR, int LT>
struct Codes {
    uint4 codes[N];
    uint32_t scales[N];

    // base: the pool's first row from the tile's first column on; STRIDE bytes a row.
    template <int STRIDE>
    __device__ __forceinline__ void load(int tid, const uint8_t* base, const uint8_t* sc, const TileRows& t, const PagedCache& c,
                                         unsigned* status) {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int idx = p * LT + tid, key = idx / PPR, i = idx % PPR;
            const int first = __shfl_sync(0xffffffffu, t.row, key >> 4), row = first + (key & 15);
            const bool live = first >= 0 && key >= t.from && key < t.to && FMHA_IN_BOUNDS(paged_row_ok(c, row), kSitePagedRow, status);
            codes[p] = live ? __ldg(reinterpret_cast<const uint4*>(base + (long long)row * STRIDE + i * 16)) : make_uint4(0u, 0u, 0u, 0u);
            scales[p] = live ? __ldg(sc + row) : 127u;
        }
    }

    // As bf16 into a tile of 64-column boxes of `rows` 128-byte rows (16-byte chunk c of row r at chunk c ^ (r % 8)).
    // A piece is two chunks; pieces 4 apart (their chunks lie in the same bank group) take theirs in the other order.
    __device__ __forceinline__ void store(int tid, uint8_t* tile, int rows, unsigned* status) const {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int idx = p * LT + tid, key = idx / PPR, i = idx % PPR;
            const PagedFactor f = paged_factor(scales[p]);
            uint32_t r[8];
            paged_values4(codes[p].x, f, r[0], r[1]);
            paged_values4(codes[p].y, f, r[2], r[3]);
            paged_values4(codes[p].z, f, r[4], r[5]);
            paged_values4(codes[p].w, f, r[6], r[7]);
            const bool swap = PPR > 4 && (i & 4);
            const uint4 a = make_uint4(r[0], r[1], r[2], r[3]), b = make_uint4(r[4], r[5], r[6], r[7]);
            const int off = (i >> 2) * rows * 128 + key * 128, c0 = (i & 3) * 2 + (swap ? 1 : 0);
            if (!FMHA_IN_BOUNDS(key < rows && off >= 0 && off + 128 <= rows * ((PPR + 3) / 4) * 128, kSitePagedKv, status)) continue;
            uint4 x = a, y = b;
            if (swap) {
                x = b;
                y = a;
            }
            *reinterpret_cast<uint4*>(tile + off + ((c0 ^ (key & 7)) << 4)) = x;
            *reinterpret_cast<uint4*>(tile + off + (((c0 ^ 1) ^ (key & 7)) << 4)) = y;
        }
    }
};

template <int HD, bool CODES, bool SINK>
__global__ void __launch_bounds__(PTCfg<HD>::THREADS, 1) paged_tc_kernel(const PagedFwd f) {
    using C = PTCfg<HD>;
    constexpr int BM = C::BM, BN = C::BN, STG = C::STG;
    launch_dependents();  // the merge grid may be scheduled now; it waits for this grid's results
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = smem;
    uint8_t* sk = smem + C::OFF_K;
    uint8_t* sv = smem + C::OFF_V;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* q_full = bars;
    uint64_t* k_full = bars + 1;
    uint64_t* k_empty = k_full + STG * C::NKC;  // by stage and chunk
    uint64_t* v_full = k_empty + STG * C::NKC;
    uint64_t* v_empty = v_full + STG;
    uint64_t* s_full = v_empty + STG;  // [2] by slot
    uint64_t* p_ready = s_full + 2;    // [2]
    uint64_t* o_done = p_ready + 2;    // [2]
    uint64_t* mma_drain = o_done + 2;  // every MMA the issuer launched has completed (exit drain)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % C::PARTS, kvh = blockIdx.x / C::PARTS % f.c.n_kv_h, split = blockIdx.y;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 12 * 32);
        for (int s = 0; s < STG * C::NKC; ++s) {
            mbar_init(&k_full[s], C::LT);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < STG; ++s) {
            mbar_init(&v_full[s], C::LT);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(mma_drain, 1);
        mbar_fence_init();
    }
    grid_dependency_wait();  // every global access below follows the preceding kernel
    const PagedTile t = paged_tile(f, blockIdx.x / C::PARTS / f.c.n_kv_h, BM * C::NRT, f.status);
    if (t.n <= 0) return;
    const PagedKeys k = paged_keys(f, t, split, BN, 16);
    if (k.n <= 0) {  // nothing to attend in this chunk: no tensor memory, no Q
        paged_write_empty(f, t, kvh, split, part * C::HDV, C::HDV);
        return;
    }
    if (warp == C::SW) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int n_rt = C::NRT == 2 && t.n > BM ? 2 : 1;
    const int n_units = k.n * n_rt;

    // Q's rows as 64-column boxes of 128 swizzled rows per row tile, zeros behind the last row; of the
    // opposite sign for a negative scale (the softmax takes its magnitude), for codes with columns 1 and 2 of each
    // four exchanged.  All but the MMA warp take part, w = 0 .. 11.
    auto load_q = [&](int w) {
        constexpr int PPR = HD / 8, BATCH = 4;
        const uint32_t sign = f.scale_log2 < 0.f ? 0x80008000u : 0u;
        const int total = n_rt * BM * PPR;
#pragma unroll 1
        for (int base = w * 32 + lane; base < total; base += 12 * 32 * BATCH) {
            uint4 u[BATCH];
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
                const int i = base + y * 12 * 32, r = i / PPR;
                u[y] = make_uint4(0u, 0u, 0u, 0u);
                if (i < total && r < t.n) u[y] = __ldg(reinterpret_cast<const uint4*>(f.q + paged_q_at(f, t, kvh, t.r0 + r) + i % PPR * 8));
            }
#pragma unroll
            for (int y = 0; y < BATCH; ++y) {
                const int i = base + y * 12 * 32, r = i / PPR, c = i % PPR;
                uint4 v = u[y];
                if constexpr (CODES)
                    v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x5410),
                                   __byte_perm(v.z, v.w, 0x7632));
                v = make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign);
                const int at = (r / BM) * C::Q_TILE + (c >> 3) * BM * 128 + (r % BM) * 128 + (((c & 7) ^ (r & 7)) << 4);
                if (i < total && FMHA_IN_BOUNDS(at >= 0 && at + 16 <= C::Q_BYTES, kSitePagedQ, f.status)) *reinterpret_cast<uint4*>(sq + at) = v;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
    };

    if (warp > C::SW) {
        // ------------------------------------------------------------ loaders
        // K_0, K_1, V_0, K_2, V_1, ...: the order in which the MMA warp takes them.
        const int tid = threadIdx.x - (C::SW + 1) * 32;
        // this lane's page of tile j, and with it the tile's rows
        auto page_of = [&](int j) {
            if (j >= k.n || lane >= BN / 16) return -1;
            const int key = k.key(j, BN) + 16 * lane;
            return key < k.to(j) && key + 16 > k.from(j) ? paged_entry(f.c, f.t.batch, t.b, key >> f.c.log_page, f.status) : -1;
        };
        auto rows_of = [&](int j, int page) {
            const int key0 = k.key(j, BN);
            return TileRows{paged_row(f.c, page, kvh, key0 + 16 * lane), k.from(j) - key0, k.to(j) - key0};
        };
        bool ok = true;
        if constexpr (CODES) {
            constexpr int KPPR = C::KCH / 16, VPPR = C::HDV / 16;
            Codes<BN * KPPR / C::LT, KPPR, C::LT> kb[C::NKC];
            Codes<BN * VPPR / C::LT, VPPR, C::LT> vb;
            const uint8_t* const kp = static_cast<const uint8_t*>(f.c.k_pages);
            const uint8_t* const vp = static_cast<const uint8_t*>(f.c.v_pages) + part * C::HDV;
            auto fetch_k = [&](const TileRows& r) {
#pragma unroll
                for (int c = 0; c < C::NKC; ++c) kb[c].template load<HD>(tid, kp + c * C::KCH, f.c.k_scales, r, f.c, f.status);
            };
            int ahead = page_of(1);
            TileRows r_v = rows_of(0, page_of(0));
            fetch_k(r_v);
            vb.template load<HD>(tid, vp, f.c.v_scales, r_v, f.c, f.status);
            load_q(warp - 1);
            // K_j and then V_{j - 1}, for j up to k.n (where there is no K_j)
#pragma unroll 1
            for (int j = 0; ok && j <= k.n; ++j) {
                const int page = ahead;  // of tile j + 1
                ahead = page_of(j + 2);
                const TileRows next = rows_of(j + 1, page);
                if (j < k.n) {
                    const int s = j % STG;
#pragma unroll
                    for (int c = 0; c < C::NKC; ++c) {
                        const int q = s * C::NKC + c;
                        ok = ok && (j < STG || mbar_wait(&k_empty[q], ((j / STG) - 1) & 1, f.status));
                        if (ok) {
                            kb[c].store(tid, sk + s * C::K_TILE + c * (C::K_TILE / C::NKC), BN, f.status);
                            fence_proxy_async_smem();
                            mbar_arrive(&k_full[q]);
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && j + 1 < k.n) fetch_k(next);
                }
                if (ok && j > 0) {
                    const int jv = j - 1, s = jv % STG;
                    ok = jv < STG || mbar_wait(&v_empty[s], ((jv / STG) - 1) & 1, f.status);
                    if (ok) {
                        vb.store(tid, sv + s * C::V_TILE, BN, f.status);
                        fence_proxy_async_smem();
                        mbar_arrive(&v_full[s]);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && j < k.n) vb.template load<HD>(tid, vp, f.c.v_scales, r_v, f.c, f.status);
                }
                r_v = next;
            }
        } else {
            // A copy is announced when the next one has been issued, or when that one has to wait.
            uint64_t* pending = nullptr;
            auto announce = [&]() {
                fence_proxy_async_smem();
                mbar_arrive(pending);
                pending = nullptr;
            };
            auto wait_empty = [&](uint64_t* bar, unsigned parity) {
                if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
                if (pending) {
                    cp_async_wait<0>();
                    announce();
                }
                return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, f.status));
            };
            auto copy = [&](const void* pages, const TileRows& r, int col0, int cols, uint8_t* tile, uint64_t* full) {
                const __nv_bfloat16* const base = static_cast<const __nv_bfloat16*>(pages) + col0;
                const uint32_t dst = smem_u32(tile);
                const int ppr = cols / 8;  // a constant once inlined
#pragma unroll 4
                for (int idx = tid; idx < BN * ppr; idx += C::LT) {
                    const int key = idx / ppr, i = idx % ppr;
                    const int first = __shfl_sync(0xffffffffu, r.row, key >> 4), row = first + (key & 15);
                    const bool live = first >= 0 && key >= r.from && key < r.to && FMHA_IN_BOUNDS(paged_row_ok(f.c, row), kSitePagedRow, f.status);
                    const int off = (i >> 3) * BN * 128 + key * 128 + (((i & 7) ^ (key & 7)) << 4);
                    if (FMHA_IN_BOUNDS(off >= 0 && off + 16 <= BN * cols * 2, kSitePagedKv, f.status))
                        cp_async16(dst + off, base + (live ? (long long)row * HD + i * 8 : 0), live);
                }
                cp_async_commit();
                if (pending) {
                    cp_async_wait<1>();
                    announce();
                }
                pending = full;
            };
            int ahead = page_of(1);
            TileRows r_k = rows_of(0, page_of(0)), r_v = r_k;
#pragma unroll 1
            for (int j = 0; ok && j <= k.n; ++j) {
                const int page = ahead;  // of tile j + 1
                ahead = page_of(j + 2);
                if (j < k.n) {
                    const int s = j % STG;
#pragma unroll
                    for (int c = 0; c < C::NKC; ++c) {
                        const int q = s * C::NKC + c;
                        ok = ok && (j < STG || wait_empty(&k_empty[q], ((j / STG) - 1) & 1));
                        if (ok) copy(f.c.k_pages, r_k, c * C::KCH, C::KCH, sk + s * C::K_TILE + c * (C::K_TILE / C::NKC), &k_full[q]);
                    }
                }
                if (j == 0) load_q(warp - 1);
                if (ok && j > 0) {
                    const int jv = j - 1, s = jv % STG;
                    ok = jv < STG || wait_empty(&v_empty[s], ((jv / STG) - 1) & 1);
                    if (ok) copy(f.c.v_pages, r_v, part * C::HDV, C::HDV, sv + s * C::V_TILE, &v_full[s]);
                }
                r_v = r_k;
                r_k = rows_of(j + 1, page);
            }
            cp_async_wait<0>();  // nothing is in flight when the block exits, whatever the waits said
            if (pending) announce();
        }
    } else if (warp == C::SW) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp walks the loop and one elected lane issues, so that the descriptors stay in
        // uniform registers.
        constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0);
        constexpr uint32_t idesc_o = idesc_bf16_f32(BM, C::HDV, 1);
        // A descriptor's low word holds the address in units of 16 bytes: the operands of a step
        // are a constant distance from the first.
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sq), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sk), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sv), BN * 128, 1024);
        bool ok = mbar_wait(q_full, 0, f.status);
        auto issue_qk = [&](int u) -> bool {
            const int j = n_rt == 2 ? u >> 1 : u, rt = n_rt == 2 ? u & 1 : 0, s = j % STG;
            const uint32_t d = tmem + (u & 1) * BN;
            if (!FMHA_IN_BOUNDS(s >= 0 && C::OFF_K + (s + 1) * C::K_TILE <= C::OFF_V && (rt + 1) * C::Q_TILE <= C::OFF_K, kSitePagedDesc, f.status))
                return false;
            const uint64_t a0 = q_desc + rt * (C::Q_TILE / 16), b0 = k_desc + s * (C::K_TILE / 16);
#pragma unroll 1
            for (int c = 0; c < C::NKC; ++c) {
                if (rt == 0 && !mbar_wait(&k_full[s * C::NKC + c], (j / STG) & 1, f.status)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int y = 0; y < C::KCH / 64; ++y) {  // 64-column boxes
                        const int x = c * (C::KCH / 64) + y;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 16 columns = 32 bytes into the swizzled row
                            tc_mma_f16(d, a0 + x * (BM * 128 / 16) + kk * 2, b0 + x * (BN * 128 / 16) + kk * 2, idesc_s,
                                       (c > 0 || y > 0 || kk > 0) ? 1u : 0u);
                    }
                    if (rt == n_rt - 1) tc_commit(&k_empty[s * C::NKC + c]);
                    if (c == C::NKC - 1) tc_commit(&s_full[u & 1]);
                }
                __syncwarp();
            }
            return true;
        };
        for (int u = 0; ok && u < 2 && u < n_units; ++u) ok = issue_qk(u);
        for (int u = 0; ok && u < n_units; ++u) {
            const int j = n_rt == 2 ? u >> 1 : u, rt = n_rt == 2 ? u & 1 : 0, s = j % STG;
            if (rt == 0 && !mbar_wait(&v_full[s], (j / STG) & 1, f.status)) break;
            if (!mbar_wait(&p_ready[u & 1], (u >> 1) & 1, f.status)) break;
            tc_fence_after();
            const uint64_t b0 = v_desc + s * (C::V_TILE / 16);
            const uint32_t p_col = tmem + (u & 1) * BN, o_col = tmem + C::O_COL + rt * C::HDV;
            if (!FMHA_IN_BOUNDS(s >= 0 && C::OFF_V + (s + 1) * C::V_TILE <= C::OFF_BAR && o_col - tmem + C::HDV <= C::TMEM_COLS, kSitePagedDesc, f.status))
                break;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    tc_mma_f16_ts(o_col, p_col + kk * 8, b0 + kk * (16 * 128 / 16), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                tc_commit(&o_done[u & 1]);
                if (rt == n_rt - 1) tc_commit(&v_empty[s]);
            }
            __syncwarp();
            if (u + 2 < n_units && !issue_qk(u + 2)) break;
        }
        // Exit drain: whatever the loop issued has completed before tensor memory and the operand
        // buffers are released, even if a wait gave up.
        if (elect_one()) tc_commit(mma_drain);
        __syncwarp();
        mbar_wait(mma_drain, 0, f.status);
    } else {
        // ------------------------------------------------------------ softmax and epilogue of row tile rt
        load_q(warp);
        const int rt = warp >> 2, quarter = warp & 3;
        if (rt < n_rt) {
            const int row = rt * BM + quarter * 32 + lane;  // of the block's rows; its TMEM lane is row % 128
            const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
            const uint32_t t_o = t_lane + C::O_COL + rt * C::HDV;
            auto o_addr = [&](int c) {  // columns 32 c .. 32 c + 31 of O
                return t_o + (FMHA_IN_BOUNDS(C::O_COL + rt * C::HDV + c * 32 + 32 <= C::TMEM_COLS, kSitePagedTmem, f.status) ? c * 32 : 0);
            };
            int jlo, jhi, fhi;
            paged_row_keys(f, t, k, t.r0 + row, jlo, jhi, fhi);
            const bool valid = row < t.n, warp_live = __any_sync(0xffffffffu, valid);
            // |scale| log2(e), not 0: a masked -inf times 0 would be a NaN (2^-126 makes all weights equal as it should)
            const float sl2 = fmaxf(fabsf(f.scale_log2), 1.17549435e-38f);
            float m_ref = -INFINITY, l = 0.f;
            // pages of a tile, by granule of 16 keys: looked up one tile ahead
            auto page_there = [&](int j) {
                if (j >= k.n || lane >= BN / 16) return false;
                const int key = k.key(j, BN) + 16 * lane;
                return key < k.to(j) && paged_entry(f.c, f.t.batch, t.b, key >> f.c.log_page, f.status) >= 0;
            };
            bool ahead = page_there(0), ok = true;
#pragma unroll 1
            for (int j = 0; j < k.n; ++j) {
                const int u = j * n_rt + rt, slot = u & 1;
                const unsigned pages = __ballot_sync(0xffffffffu, ahead);
                ahead = page_there(j + 1);
                if (!__all_sync(0xffffffffu, mbar_wait(&s_full[slot], (u >> 1) & 1, f.status))) {
                    ok = false;
                    break;
                }
                if (!warp_live) {  // rows behind the last one: whatever P they have goes nowhere
                    tc_fence_before();
                    mbar_arrive(&p_ready[slot]);
                    continue;
                }
                tc_fence_after();
                const uint32_t s_addr = t_lane + (FMHA_IN_BOUNDS(slot * BN + BN <= C::O_COL, kSitePagedTmem, f.status) ? slot * BN : 0);
                const int key0 = k.key(j, BN);
                const int lo = k.head(j) ? 0 : jlo, hi = k.head(j) ? fhi : jhi;
                const bool full = pages == (1u << (BN / 16)) - 1u && key0 >= lo && key0 + BN - 1 <= hi;
                // the row's scores from column `col` of the tile on, -inf where it attends no key
                auto load_scores = [&](int col, float (&x)[32]) {
                    tmem_ld32(s_addr + col, x);
                    tmem_wait_ld();
                    if (!full) {
                        const int first = key0 + col;
                        const int k0 = max(0, lo - first), k1 = min(31, hi - first);
                        uint32_t in = k1 >= k0 ? (0xffffffffu >> (31 - k1)) & (0xffffffffu << k0) : 0u;
                        const unsigned p = pages >> (col >> 4);
                        in &= (p & 1u ? 0xffffu : 0u) | (p & 2u ? 0xffff0000u : 0u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = (in >> i) & 1u ? x[i] : -INFINITY;
                    }
                };
                float alpha = 1.f, sum;
                uint32_t pk[BN / 2];
                bool move = valid && m_ref == -INFINITY;
#pragma unroll 1
                for (int again = 0;; ++again) {
                    if (__any_sync(0xffffffffu, move)) {
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int col = 0; col < BN; col += 32) {
                            float x[32];
                            load_scores(col, x);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[i], x[i + 1]));
                        }
                        const float mt = mx * sl2;
                        if (mt > m_ref) {
                            if (m_ref != -INFINITY) alpha = ex2_approx(m_ref - mt);  // without a reference O is zero
                            m_ref = mt;
                            l *= alpha;
                        }
                    }
                    const float mu = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t q2 = f32x2(sl2, sl2), mu2 = f32x2(mu, mu);
                    uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                    for (int col = 0; col < BN; col += 32) {
                        float x[32];
                        load_scores(col, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            f32x2_split(fma_f32x2(f32x2(x[2 * i], x[2 * i + 1]), q2, mu2), y0, y1);
                            y0 = ex2_approx(y0);
                            y1 = ex2_approx(y1);
                            pk[col / 2 + i] = pack_bf16x2(y0, y1);
                            s2[i & 1] = add_f32x2(s2[i & 1], f32x2(y0, y1));
                        }
                    }
                    float a0, a1, b0, b1;
                    f32x2_split(s2[0], a0, a1);
                    f32x2_split(s2[1], b0, b1);
                    sum = (a0 + a1) + (b0 + b1);
                    move = sum > 1.0995116e12f;  // 2^40
                    if (again > 0 || !__any_sync(0xffffffffu, move)) break;
                }
                l += sum;
                // O's rescale needs the unit before on this row tile: with two row tiles its PV completed before S did
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    if (n_rt == 1 && !__all_sync(0xffffffffu, mbar_wait(&o_done[(u - 1) & 1], ((u - 1) >> 1) & 1, f.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < C::HDV / 32; ++c) {
                        float ov[32];
                        tmem_ld32(o_addr(c), ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] *= alpha;
                        tmem_st32(o_addr(c), ov);
                    }
                }
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) tmem_st32u(s_addr + c * 32, pk + c * 32);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_ready[slot]);
            }
            // ------------------------------------------------------------ epilogue
            const int last = (k.n - 1) * n_rt + rt;
            if (ok) ok = mbar_wait(&o_done[last & 1], (last >> 1) & 1, f.status);
            ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld below is warp-collective
            tc_fence_after();
            int head = 0;
            const long long orow = valid ? paged_out_row(f, t, kvh, t.r0 + row, head) : 0;
            float inv, lse;
            paged_finish(m_ref, l, (SINK && valid) ? sink_log2_of(f.sink, head, f.n_h, f.status) : -INFINITY, inv, lse);
            const bool store = valid && ok && FMHA_IN_BOUNDS(orow >= 0 && orow < f.rows && split < f.n_splits, kSitePagedOut, f.status);
            const unsigned rows_live = __ballot_sync(0xffffffffu, store);
            // through a 4 KB corner of the row tile's Q per warp (its MMAs are done), so that a
            // store covers whole 64- or 128-byte pieces of rows
            uint8_t* stage = sq + rt * C::Q_TILE + quarter * 4096;
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < C::HDV / 32; ++c) {
                    float ov[32];
                    tmem_ld32(o_addr(c), ov);
                    tmem_wait_ld();
                    if constexpr (CODES) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float x = ov[i + 1];
                            ov[i + 1] = ov[i + 2];
                            ov[i + 2] = x;
                        }
                    }
                    const int col = part * C::HDV + c * 32;
                    if (!FMHA_IN_BOUNDS(col + 32 <= HD && quarter * 4096 + 4096 <= C::Q_TILE, kSitePagedComb, f.status)) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                            make_float4(ov[4 * q] * inv, ov[4 * q + 1] * inv, ov[4 * q + 2] * inv, ov[4 * q + 3] * inv);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // 4 rows of 8 x 16 bytes
                        const int r = i * 4 + (lane >> 3), q = lane & 7;
                        const long long at = __shfl_sync(0xffffffffu, orow, r);
                        if (!((rows_live >> r) & 1u)) continue;
                        const float4 v = *reinterpret_cast<const float4*>(stage + r * 128 + ((q ^ (r & 7)) << 4));
                        if (f.n_splits == 1)
                            *reinterpret_cast<uint2*>(f.o + at * HD + col + q * 4) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(f.o_part + (split * f.rows + at) * HD + col + q * 4) = v;
                    }
                    __syncwarp();
                }
            }
            if (store && part == 0) (f.n_splits == 1 ? f.lse + orow : f.lse_part + split * f.rows + orow)[0] = lse;
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == C::SW) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int HD, bool CODES, bool SINK>
cudaError_t launch_t(const PagedFwd& f, cudaStream_t stream) {
    using C = PTCfg<HD>;
    auto kern = paged_tc_kernel<HD, CODES, SINK>;
    static std::atomic<bool> attr_set[128];  // set once per device; any host thread may set it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 128) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(f.row_tiles * C::PARTS * f.c.n_kv_h), f.n_splits);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, f);
}

template <bool CODES, bool SINK>
cudaError_t launch_s(const PagedFwd& f, cudaStream_t stream) {
    switch (f.c.hd) {
        case 64: return launch_t<64, CODES, SINK>(f, stream);
        case 128: return launch_t<128, CODES, SINK>(f, stream);
        case 256: return launch_t<256, CODES, SINK>(f, stream);
        case 512: return launch_t<512, CODES, SINK>(f, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int paged_tc_kv_tile(int hd) { return hd <= 128 ? PTCfg<128>::BN : PTCfg<256>::BN; }
int paged_tc_rows(int hd) { return hd <= 128 ? 256 : 128; }

cudaError_t launch_paged_tc(const PagedFwd& f, cudaStream_t stream) {
    const bool sink = f.sink && f.n_splits == 1, codes = f.c.k_scales != nullptr;
    if (codes) return sink ? launch_s<true, true>(f, stream) : launch_s<true, false>(f, stream);
    return sink ? launch_s<false, true>(f, stream) : launch_s<false, false>(f, stream);
}

}  // namespace fmha
