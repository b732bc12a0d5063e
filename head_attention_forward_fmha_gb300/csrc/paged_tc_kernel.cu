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
// Warp roles: 4 warps per row tile softmax and epilogue (one row per thread), one warp MMA issue and
// tensor memory, one producer, and for codes the converters.
//   bf16 pages: the producer's lanes look a tile's pages up in the block table, one tile ahead, and load
//     its boxes by TMA into the swizzled operand layout (a page that is not there is a box behind the
//     pool: zeros).  Of a V tile at the end of the keys (or at the start of a window) it then clears the
//     rows that no query row attends, so that nothing stale is multiplied.
//   8-bit pages: bulk copies of the pages' codes into a raw buffer, the scale bytes by cp.async, and the
//     converters expand them to bf16 (paged_common.cuh) into the operand layout.  Expanded columns 1 and 2 of
//     each four change places: Q is stored the same way, and O's columns are put right in the epilogue.
//     (To fp16 by the hardware's conversion it takes half the instructions but, with the units that
//     fp16's range asks for, not less time: 346 us for a chunk that takes 305.)
// At hd 256 and 512 256 of Q's columns lie in tensor memory: QK takes its A operand from there, which at N = 64 is
// faster (32 clocks an MMA, 48 with both operands from shared memory) and leaves room for stages and raw buffers.
//
// Softmax: scores against a reference, the maximum of the first scores that the row attends (so that a row's
// only key has P = 1, which bf16 holds).  Only where a score passes the reference by kPast = 8 (log2 units) does that
// move, by a whole number, and the sum, O and the tile's weights so far are multiplied by the power of two.  So P is at
// most 2^8 and O's fp32 sum holds values of V up to 2^120 over the number of keys.  (P and its own sum would bear 40, but not
// P V: with V of 2^90 O was infinite.  For a chunk of 512 tokens over 4 x 8192 keys both bounds take the same time with scores of
// unit variance; with a deviation of 8, where 40 is never passed, hd 128 takes 276 us and 220 with 40, hd 64 233 and 200, hd 256
// 472 and 416, hd 512 and 8 bits the same.)  (The check comes before a chunk's
// exponentials: found afterwards, with the chunk done again, it cost 254 us where it now takes 222.)
//
// What bounds it (GB300; chunks of 512 tokens over 4 x 8192 keys, 32 query heads on 4): at hd 128 in bf16 a tile of 256 rows
// and 128 keys takes 1.75 us, of which the MMAs need 1.33, the exponentials as long on half of the
// SM's four schedulers' time: 222 us; 1390 TFLOP/s, 73 % of the measured peak, for 8 x 2048 tokens over 8192 keys.  At hd 64 (201 us)
// the softmax, 1.6 us a tile for half the MMAs: stalls on its scores from tensor memory and on fixed latencies, 1.6 each per
// issue, with the tensor pipe at 30 %.  At hd 256 (419 us, 1270 TFLOP/s; 1470 for the 8 x 2048 tokens) and 512 (1234 us, each half of
// O with all of S: a third of the MMAs are done twice) the MMAs.  In 8 bits the converters: 2.4 us a tile at hd 128
// (309 us), 1.7 for 64 keys at 256 (921 us), 2.4 at 512 (2335 us), with 2.5 integer instructions a value; fewer than eight
// warps for it take longer (six 452, four 514 us where eight took 305).  At hd 512 both blocks of a row tile load and convert all of K,
// and load all 512 columns of V's codes, of which each uses its own 256: a quarter of a block's traffic from the pages.
#include <atomic>
#include <type_traits>
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

template <int HD, bool CODES>
struct PTCfg {
    static constexpr int BM = 128;
    static constexpr int NRT = HD <= 128 ? 2 : 1;         // row tiles
    static constexpr int BN = HD <= 128 ? 128 : 64;       // keys per tile
    static constexpr int HDV = HD == 512 ? 256 : HD;      // columns of O per block
    static constexpr int PARTS = HD / HDV;                // blocks per row tile
    static constexpr int QT = HD >= 256 ? 256 : 0;        // columns of Q in tensor memory, the first ones
    static constexpr int KST = HD == 64 ? 4 : HD == 128 ? 2 : HD == 256 ? 3 : CODES ? 1 : 2;  // K stages
    static constexpr int VST = HD == 512 ? 1 : KST;       // V stages
    static constexpr int NKC = HD == 512 ? 2 : 1;         // column chunks of a K tile, each with barriers of its own
    static constexpr int KCH = HD / NKC;
    static constexpr int NB = KCH / 64;                   // 64-column blocks of a K chunk, and of V
    static constexpr int SW = 4 * NRT;                    // softmax warps
    static constexpr int CW = CODES ? 8 : 0;              // converter warps
    static constexpr int CT = 32 * CW;
    static constexpr int HW = HD == 512 && !CODES ? 4 : 0;  // warps that only help to load Q
    static constexpr int QW = QT == HD ? SW : SW + CW + HW;  // warps that load Q
    static constexpr int WARPS = SW + 2 + CW + HW;        // + MMA issuer (warp SW) and producer (SW + 1)
    static constexpr int THREADS = WARPS * 32;
    static constexpr int CH = CODES && NRT == 2 ? 32 : 64;  // scores that a softmax thread holds (18 warps leave it 96 registers)
    static constexpr int K_ARRIVALS = CODES ? CT : 1;     // on a full barrier of K or V
    static constexpr int Q_TILE = BM * (HD - QT) * 2;
    static constexpr int Q_BYTES = NRT * Q_TILE;
    static constexpr int K_TILE = BN * HD * 2;
    static constexpr int V_TILE = BN * HDV * 2;
    static constexpr int O_COL = 2 * BN;                  // tensor memory: two S slots, then O of each row tile, then Q
    static constexpr int Q_COL = O_COL + NRT * HDV;
    static constexpr int TMEM_COLS = 512;
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + KST * K_TILE;
    static constexpr int OFF_RAW = OFF_V + VST * V_TILE;  // codes of K, of V
    static constexpr int RAW_TILE = BN * HD;
    static constexpr int OFF_SC = OFF_RAW + (CODES ? 2 * RAW_TILE : 0);  // scale bytes of K, of V
    static constexpr int OFF_BAR = OFF_SC + (CODES ? 2 * BN : 0);
    static constexpr int N_BARS = 1 + 2 * KST * NKC + 2 * VST + 6 + 1 + 4;
    static constexpr int OFF_TILE = OFF_BAR + N_BARS * 8 + 16;  // (the tensor-memory address before it)
    static constexpr int NEED = 1024 + OFF_TILE + 32;
    static_assert(OFF_TILE % 4 == 0 && sizeof(PagedTile) <= 32, "the block's rows");
    static constexpr int SMEM = NEED < 120000 ? 120000 : NEED;  // one block per SM: each takes all of tensor memory
    static_assert(NB == HDV / 64, "K chunks and V tiles have the same layout");
    static_assert(Q_COL + QT / 2 <= TMEM_COLS, "S, O and Q fit in tensor memory");
    static_assert(QT % KCH == 0 || QT == HD, "a K chunk meets Q in one place");
    static_assert(SMEM <= 232448, "shared memory budget");
};

constexpr float kPast = 8.f;  // by how much a score may pass its row's reference

// Operand layout of a K chunk and of a V tile, NB blocks of 64 columns wide: groups of 8 keys, in each
// the blocks one after another (1024 bytes: 8 rows of 128, 16-byte chunk c of row r at chunk c ^ (r % 8)).
// So the rows of a page lie together, all blocks of them, and one TMA box brings them: a box costs ~50
// clocks and ~2.4 for each 128 bytes (32 KB in boxes of 2 KB 1621 clocks, of 4 KB 1019, of 32 KB 669).
template <int NB>
__device__ __forceinline__ int operand_row(int key, int block) {
    return (key >> 3) * (NB * 1024) + block * 1024 + (key & 7) * 128;
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// One arrival on the barrier when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 packed words times a packed factor, in this thread's TMEM lane.  (32 columns are read, 16 written.)
__device__ __forceinline__ void tmem_scale_pairs(uint32_t taddr, uint32_t factor) {
    float v[32];
    tmem_ld32(taddr, v);
    tmem_wait_ld();
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = mul_bf16x2(__float_as_uint(v[i]), factor);
    tmem_st16u(taddr, w);
}

template <int HD, bool CODES, bool SINK>
__global__ void __launch_bounds__(PTCfg<HD, CODES>::THREADS, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const PagedFwd f) {
    using C = PTCfg<HD, CODES>;
    constexpr int BM = C::BM, BN = C::BN, KST = C::KST, VST = C::VST;
    launch_dependents();  // the merge grid may be scheduled now; it waits for this grid's results
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = smem;
    uint8_t* sk = smem + C::OFF_K;
    uint8_t* sv = smem + C::OFF_V;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* q_full = bars;
    uint64_t* k_full = bars + 1;
    uint64_t* k_empty = k_full + KST * C::NKC;  // by stage and chunk
    uint64_t* v_full = k_empty + KST * C::NKC;
    uint64_t* v_empty = v_full + VST;
    uint64_t* s_full = v_empty + VST;  // [2] by slot
    uint64_t* p_ready = s_full + 2;    // [2]
    uint64_t* o_done = p_ready + 2;    // [2]
    uint64_t* mma_drain = o_done + 2;  // every MMA the issuer launched has completed (exit drain)
    uint64_t* raw_full = mma_drain + 1;   // [2] raw codes and scale bytes of K, of V (bf16: a V tile to be cleared in part)
    uint64_t* raw_empty = raw_full + 2;   // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
    PagedTile* tile = reinterpret_cast<PagedTile*>(smem + C::OFF_TILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % C::PARTS, kvh = blockIdx.x / C::PARTS % f.c.n_kv_h, split = blockIdx.y;
    if (threadIdx.x == 0) {
        mbar_init(q_full, C::QW * 32);
        for (int s = 0; s < KST * C::NKC; ++s) {
            mbar_init(&k_full[s], C::K_ARRIVALS);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < VST; ++s) {
            mbar_init(&v_full[s], C::K_ARRIVALS);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
            mbar_init(&o_done[s], 1);
            mbar_init(&raw_full[s], CODES ? 33 : 1);
            mbar_init(&raw_empty[s], CODES ? C::CT : 1);
        }
        mbar_init(mma_drain, 1);
        mbar_fence_init();
    }
    grid_dependency_wait();  // every global access below follows the preceding kernel
    // One warp reads which rows and keys are the block's, for all: lengths or bounds that another stream changes meanwhile give
    // results of any value, but no warps that disagree on what they wait for.
    const int box_keys = min(f.c.page, BN);  // keys that are copied at once, from a multiple of that on
    if (warp == C::SW) {
        const PagedTile mine = paged_tile_by_keys<BM * C::NRT>(f, blockIdx.x / C::PARTS / f.c.n_kv_h, f.status);
        if (lane == 0) *tile = mine;
        if (mine.n > 0 && paged_keys(f, mine, split, BN, box_keys).n > 0) {
            tmem_alloc(tmem_slot, C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const PagedTile t = paged_tile_from(tile);
    if (t.n <= 0) return;
    const PagedKeys k = paged_keys(f, t, split, BN, box_keys);
    if (k.n <= 0) {  // nothing to attend in this chunk: no tensor memory, no Q
        paged_write_empty(f, t, kvh, split, part * C::HDV, C::HDV);
        return;
    }
    const uint32_t tmem = *tmem_slot;
    const int n_rt = C::NRT == 2 && t.n > BM ? 2 : 1;

    // Q of the opposite sign for a negative scale (the softmax takes its magnitude); for codes with columns 1 and 2 of each
    // four exchanged; zeros behind the last row.
    const uint32_t q_sign = f.scale_log2 < 0.f ? 0x80008000u : 0u;
    auto as_operand = [&](uint4 v) {
        if constexpr (CODES)
            v = make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
        return make_uint4(v.x ^ q_sign, v.y ^ q_sign, v.z ^ q_sign, v.w ^ q_sign);
    };
    // Columns from QT on as 64-column boxes of 128 swizzled rows per row tile, by warps w = 0 .. QW - 1.
    auto load_q = [&](int w) {
        if constexpr (C::QT < HD) {
            constexpr int PPR = (HD - C::QT) / 8, BATCH = 8, QN = C::QW * 32;
            const int total = n_rt * BM * PPR;
#pragma unroll 1
            for (int base = w * 32 + lane; base < total; base += QN * BATCH) {
                uint4 u[BATCH];
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const int i = base + y * QN, r = i / PPR;
                    u[y] = make_uint4(0u, 0u, 0u, 0u);
                    if (i < total && r < t.n) u[y] = __ldg(reinterpret_cast<const uint4*>(f.q + paged_q_at(f, t, kvh, t.r0 + r) + C::QT + i % PPR * 8));
                }
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const int i = base + y * QN, r = i / PPR, c = i % PPR;
                    const int at = (r / BM) * C::Q_TILE + (c >> 3) * BM * 128 + (r % BM) * 128 + (((c & 7) ^ (r & 7)) << 4);
                    if (i < total && FMHA_IN_BOUNDS(at >= 0 && at + 16 <= C::Q_BYTES, kSitePagedQ, f.status)) *reinterpret_cast<uint4*>(sq + at) = as_operand(u[y]);
                }
            }
            fence_proxy_async_smem();
        }
        mbar_arrive(q_full);
    };

    // The block table's entry for this lane's granule of 16 keys (lane < BN / 16) of tile j, -1 where no key is needed.
    auto entry_of = [&](int j) {
        if (j >= k.n || lane >= BN / 16) return -1;
        const int key = k.key(j, BN) + 16 * lane;  // (the copy that it begins may reach into the keys)
        return key < k.to(j) && (key | (box_keys - 1)) >= k.from(j) ? paged_entry(f.c, f.t.batch, t.b, key >> f.c.log_page, f.status) : -1;
    };
    // all lanes of the warp go on or none: collectives follow
    auto wait_all = [&](uint64_t* bar, unsigned parity) { return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, f.status)); };

    if (warp == C::SW + 1) {
        // ------------------------------------------------------------ producer
        // K_0, K_1, V_0, K_2, V_1, ...: the order in which the MMA warp takes them.
        if constexpr (!CODES) {
            if (lane == 0) {
                tma_prefetch_desc(&tmk);
                tma_prefetch_desc(&tmv);
            }
            const int log_box = __ffs(box_keys) - 1, boxes = BN >> log_box;
            // blocks block0 .. block0 + NB - 1 of K or V, all keys of tile j
            auto load = [&](const CUtensorMap* map, int j, int page, int block0, uint8_t* tile, uint64_t* bar) {
                const int key0 = k.key(j, BN);
                if (lane == 0) mbar_arrive_expect_tx(bar, BN * C::NB * 128);
                __syncwarp();
                const int p = __shfl_sync(0xffffffffu, page, lane << (log_box - 4) & 31);
                const int slab = p < 0 ? f.c.n_pages * f.c.n_kv_h : p * f.c.n_kv_h + kvh;  // behind the pool: zeros
                const int row = (key0 + (lane << log_box)) & (f.c.page - 1);
                if (lane < boxes && FMHA_IN_BOUNDS(row + box_keys <= f.c.page && ((lane + 1) << log_box) <= BN, kSitePagedKv, f.status))
                    tma_load_5d(tile + (lane << log_box) * C::NB * 128, map, 0, 0, block0, row >> 3, slab, bar);
            };
            bool ok = true;
            int k_issued = 0, v_issued = 0, cleared = 0, ahead = entry_of(1), page_k = paged_page(f.c, entry_of(0)), page_v = page_k;
#pragma unroll 1
            for (int j = 0; ok && j <= k.n; ++j) {
                const int page = paged_page(f.c, ahead);  // of tile j + 1
                ahead = entry_of(j + 2);
                if (j < k.n) {
                    const int s = j % KST;
#pragma unroll 1
                    for (int c = 0; ok && c < C::NKC; ++c) {
                        ok = j < KST || wait_all(&k_empty[s * C::NKC + c], ((j / KST) - 1) & 1);
                        if (ok) {
                            load(&tmk, j, page_k, c * C::NB, sk + s * C::K_TILE + c * (C::K_TILE / C::NKC), &k_full[s * C::NKC + c]);
                            ++k_issued;
                        }
                    }
                }
                if (ok && j > 0) {
                    const int jv = j - 1, s = jv % VST;
                    ok = jv < VST || wait_all(&v_empty[s], ((jv / VST) - 1) & 1);
                    if (ok) {
                        const int key0 = k.key(jv, BN), from = k.from(jv) - key0, to = k.to(jv) - key0;
                        uint8_t* tile = sv + s * C::V_TILE;
                        if (from <= 0 && to >= BN) {
                            load(&tmv, jv, page_v, part * C::NB, tile, &v_full[s]);
                        } else {
                            load(&tmv, jv, page_v, part * C::NB, tile, &raw_full[0]);
                            ok = wait_all(&raw_full[0], cleared++ & 1);
                            const int lead = max(from, 0), rows = lead + BN - min(to, BN);  // those before `from`, those from `to` on
                            for (int i = lane; ok && i < rows * (C::HDV / 8); i += 32) {
                                const int r = i / (C::HDV / 8), c = i % (C::HDV / 8), row = r < lead ? r : r - lead + to;
                                if (FMHA_IN_BOUNDS(row >= 0 && row < BN, kSitePagedKv, f.status))
                                    *reinterpret_cast<uint4*>(tile + operand_row<C::NB>(row, c >> 3) + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (ok && lane == 0) mbar_arrive(&v_full[s]);
                        }
                        ++v_issued;
                    }
                }
                page_v = page_k;
                page_k = page;
            }
            // Exit drain: what was loaded has landed before the block exits, whatever the waits said.
            drain_ring(k_full, KST * C::NKC, k_issued, f.status);
            drain_ring(v_full, VST, v_issued, f.status);
        } else {
            // One raw buffer each for K and V, filled again as soon as the converters have read it: they go
            // K_0 K_1 V_0 K_2 V_1 ..., so K_{j+2} can be on its way while they are at V_j.
            const uint64_t pol = l2_policy_evict_first();
            bool ok = true;
            int issued[2] = {0, 0};
            const int log_box = __ffs(box_keys) - 1;
            auto load = [&](int x, int j, int page) {
                ok = ok && (issued[x] == 0 || wait_all(&raw_empty[x], (issued[x] - 1) & 1));
                if (!ok) return;
                const int key0 = k.key(j, BN);
                const uint8_t* const pool = static_cast<const uint8_t*>(x ? f.c.v_pages : f.c.k_pages);
                const uint8_t* const sc = x ? f.c.v_scales : f.c.k_scales;
                uint8_t* const raw = smem + C::OFF_RAW + x * C::RAW_TILE;
                // box `lane` begins with granule lane * box_keys / 16
                const int p = __shfl_sync(0xffffffffu, page, lane << (log_box - 4) & 31);
                const int key = key0 + (lane << log_box), row = p < 0 ? -1 : ((p * f.c.n_kv_h + kvh) << f.c.log_page) + (key & (f.c.page - 1));
                const bool there = (lane << log_box) < BN && row >= 0 &&
                                   FMHA_IN_BOUNDS(paged_row_ok(f.c, row + box_keys - 1LL) && ((lane + 1) << log_box) <= BN, kSitePagedRow, f.status);
                const unsigned boxes = __ballot_sync(0xffffffffu, there);
                if (lane == 0) mbar_arrive_expect_tx(&raw_full[x], __popc(boxes) * box_keys * HD);
                __syncwarp();
                if (there) bulk_load_hint(smem_u32(raw + (lane << log_box) * HD), pool + (long long)row * HD, box_keys * HD, &raw_full[x], pol);
                // scale bytes, four keys a lane
                const int first = __shfl_sync(0xffffffffu, paged_row(f.c, page, kvh, key0 + 16 * lane), lane >> 2);
                if (lane < BN / 4) {
                    const bool live = first >= 0 && FMHA_IN_BOUNDS(paged_row_ok(f.c, first + 15LL), kSitePagedRow, f.status);
                    cp_async4(smem + C::OFF_SC + x * BN + lane * 4, sc + (live ? first + (lane & 3) * 4 : 0), live);
                }
                cp_async_arrive(&raw_full[x]);
                ++issued[x];
            };
            int ahead = entry_of(2);
            const int page0 = paged_page(f.c, entry_of(0));
            int page1 = paged_page(f.c, entry_of(1));
            load(0, 0, page0);
            load(1, 0, page0);
            if (k.n > 1) load(0, 1, page1);
#pragma unroll 1
            for (int j = 2; ok && j <= k.n; ++j) {
                const int page2 = paged_page(f.c, ahead);
                ahead = entry_of(j + 1);
                if (j < k.n) load(0, j, page2);
                load(1, j - 1, page1);
                page1 = page2;
            }
            // Exit drain: the last copies have landed (those before them had to, for the buffer to be free).
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (issued[x] > 0) mbar_wait(&raw_full[x], (issued[x] - 1) & 1, f.status);
        }
    } else if (C::HW > 0 && warp > C::SW + 1) {
        load_q(warp - 2);
    } else if (warp > C::SW + 1) {
        // ------------------------------------------------------------ converters
        const int tid = threadIdx.x - (C::SW + 2) * 32;
        bool ok = true;
        if constexpr (C::QT < HD) load_q(warp - 2);
        if constexpr (CODES) {
            // Pieces of 16 columns, PPR per key, going round the threads, four read before they are expanded.
            // Columns from col0 on, as many as a K chunk or V tile has.
            auto convert = [&](int j, int x, int col0, uint8_t* tile) {
                constexpr int PPR = C::KCH / 16, N = BN * PPR / C::CT, STEP = C::CT / PPR;  // keys from one piece of a thread to the next
                const int key0 = k.key(j, BN), from = k.from(j) - key0, to = k.to(j) - key0;
                const uint8_t* const raw = smem + C::OFF_RAW + x * C::RAW_TILE;
                const uint8_t* const sc = smem + C::OFF_SC + x * BN;
                const int i = tid % PPR, first = tid / PPR;
                // a piece is two neighbouring chunks; pieces 4 apart lie in the same banks: they store theirs in the other order
                const int c0 = (i & 3) * 2 ^ (first & 7), flip = PPR > 4 ? (i >> 2) & 1 : 0;
                constexpr int U = N < 4 ? N : 4;
                static_assert(N % U == 0 && STEP % 8 == 0, "pieces in fours, at one place of the swizzle");
#pragma unroll
                for (int n0 = 0; n0 < N; n0 += U) {
                    uint4 u[U];
                    uint32_t byte[U], most = 0u;
#pragma unroll
                    for (int n = 0; n < U; ++n) {
                        const int key = first + (n0 + n) * STEP;
                        u[n] = *reinterpret_cast<const uint4*>(raw + key * HD + col0 + i * 16);
                        byte[n] = sc[key];
                        if (key < from || key >= to) {  // nothing stale is multiplied
                            u[n] = make_uint4(0u, 0u, 0u, 0u);
                            byte[n] = 127u;
                        }
                        most = max(most, byte[n]);
                    }
                    const bool two = __any_sync(0xffffffffu, most > 134u);
#pragma unroll
                    for (int n = 0; n < U; ++n) {
                        const int key = first + (n0 + n) * STEP;
                        uint32_t r[8];
                        const uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
                        if (!two) {  // the factor in one step (paged_common.cuh)
                            const uint32_t fac = (byte[n] + 120u) * 0x00800080u;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                r[2 * y] = mul_bf16x2(e4m3x2_raw<true>(w[y]), fac);
                                r[2 * y + 1] = mul_bf16x2(e4m3x2_raw<false>(w[y]), fac);
                            }
                        } else {
                            const PagedFactor fac = paged_factor(byte[n]);
#pragma unroll
                            for (int y = 0; y < 4; ++y) paged_values4(w[y], fac, r[2 * y], r[2 * y + 1]);
                        }
                        if (!FMHA_IN_BOUNDS(key < BN && (i >> 2) < C::NB, kSitePagedKv, f.status)) continue;
                        uint8_t* const row = tile + operand_row<C::NB>(key, i >> 2);
                        uint4 a = make_uint4(r[0], r[1], r[2], r[3]), b = make_uint4(r[4], r[5], r[6], r[7]);
                        if (flip) {
                            const uint4 y = a;
                            a = b;
                            b = y;
                        }
                        *reinterpret_cast<uint4*>(row + ((c0 ^ flip) << 4)) = a;
                        *reinterpret_cast<uint4*>(row + ((c0 ^ 1 ^ flip) << 4)) = b;
                    }
                }
                fence_proxy_async_smem();
            };
            // K_0, K_1, V_0, K_2, V_1, ...
#pragma unroll 1
            for (int j = 0; ok && j <= k.n; ++j) {
                if (j < k.n) {
                    const int s = j % KST;
                    ok = wait_all(&raw_full[0], j & 1);
#pragma unroll 1
                    for (int c = 0; ok && c < C::NKC; ++c) {
                        ok = j < KST || wait_all(&k_empty[s * C::NKC + c], ((j / KST) - 1) & 1);
                        if (!ok) break;
                        convert(j, 0, c * C::KCH, sk + s * C::K_TILE + c * (C::K_TILE / C::NKC));
                        if (c == C::NKC - 1) mbar_arrive(&raw_empty[0]);
                        mbar_arrive(&k_full[s * C::NKC + c]);
                    }
                }
                if (ok && j > 0) {
                    const int jv = j - 1, s = jv % VST;
                    ok = wait_all(&raw_full[1], jv & 1) && (jv < VST || wait_all(&v_empty[s], ((jv / VST) - 1) & 1));
                    if (ok) {
                        convert(jv, 1, part * C::HDV, sv + s * C::V_TILE);
                        mbar_arrive(&raw_empty[1]);
                        mbar_arrive(&v_full[s]);
                    }
                }
            }
        }
    } else if (warp == C::SW) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp walks the loop, its waits agreed upon by all lanes, and one elected lane issues; the
        // slot and the row tile of a unit are constants of the code: descriptors then stay in uniform registers.
        constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0);
        constexpr uint32_t idesc_o = idesc_bf16_f32(BM, C::HDV, 1);
        // A descriptor's low word holds the address in units of 16 bytes: the operands of a step
        // are a constant distance from the first.
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sq), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_u32(sk), 16, C::NB * 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sv), 1024, C::NB * 1024);
        bool ok = wait_all(q_full, 0);
        auto chain = [&](auto rts) {
            constexpr int NR = decltype(rts)::value;
            // QK(u) of key tile j, for row tile RT, into slot SLOT
            auto issue_qk = [&](int j, auto rt_, auto slot_) -> bool {
                constexpr int RT = decltype(rt_)::value, SLOT = decltype(slot_)::value;
                const int s = j % KST;
                const uint32_t d = tmem + SLOT * BN;
                if (!FMHA_IN_BOUNDS(s >= 0 && C::OFF_K + (s + 1) * C::K_TILE <= C::OFF_V && (RT + 1) * C::Q_TILE <= C::OFF_K, kSitePagedDesc, f.status))
                    return false;
                const uint64_t a0 = q_desc + RT * (C::Q_TILE / 16), b0 = k_desc + s * (C::K_TILE / 16);
#pragma unroll
                for (int c = 0; c < C::NKC; ++c) {
                    if (RT == 0 && !wait_all(&k_full[s * C::NKC + c], (j / KST) & 1)) return false;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int y = 0; y < C::NB; ++y)  // blocks of 64 columns
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {  // 16 columns = 32 bytes into the swizzled row
                                const uint64_t b = b0 + c * (C::K_TILE / C::NKC / 16) + y * 64 + kk * 2;
                                const int col = c * C::KCH + y * 64 + kk * 16;
                                const uint32_t more = col > 0 ? 1u : 0u;
                                if (col < C::QT)
                                    tc_mma_f16_ts(d, tmem + C::Q_COL + col / 2, b, idesc_s, more);
                                else
                                    tc_mma_f16(d, a0 + (col - C::QT) / 64 * (BM * 128 / 16) + kk * 2, b, idesc_s, more);
                            }
                        if (RT == NR - 1) tc_commit(&k_empty[s * C::NKC + c]);
                        if (c == C::NKC - 1) tc_commit(&s_full[SLOT]);
                    }
                    __syncwarp();
                }
                return true;
            };
            // PV(u) for slot SLOT, key tile j, row tile RT; phase: of the slot's barrier
            auto issue_pv = [&](int j, unsigned phase, auto rt_, auto slot_) -> bool {
                constexpr int RT = decltype(rt_)::value, SLOT = decltype(slot_)::value;
                const int s = j % VST;
                if (RT == 0 && !wait_all(&v_full[s], (j / VST) & 1)) return false;
                if (!wait_all(&p_ready[SLOT], phase)) return false;
                tc_fence_after();
                const uint64_t b0 = v_desc + s * (C::V_TILE / 16);
                if (!FMHA_IN_BOUNDS(s >= 0 && C::OFF_V + (s + 1) * C::V_TILE <= C::OFF_RAW && C::O_COL + (RT + 1) * C::HDV <= C::TMEM_COLS, kSitePagedDesc, f.status))
                    return false;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        tc_mma_f16_ts(tmem + C::O_COL + RT * C::HDV, tmem + SLOT * BN + kk * 8, b0 + kk * (C::NB * 128), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&o_done[SLOT]);
                    if (RT == NR - 1) tc_commit(&v_empty[s]);
                }
                __syncwarp();
                return true;
            };
            constexpr std::integral_constant<int, 0> zero{};
            constexpr std::integral_constant<int, 1> one{};
            if constexpr (NR == 2) {
                ok = ok && issue_qk(0, zero, zero) && issue_qk(0, one, one);
#pragma unroll 1
                for (int j = 0; ok && j < k.n; ++j) {
                    ok = issue_pv(j, j & 1, zero, zero) && (j + 1 >= k.n || issue_qk(j + 1, zero, zero)) && issue_pv(j, j & 1, one, one) &&
                         (j + 1 >= k.n || issue_qk(j + 1, one, one));
                }
            } else {
                ok = ok && issue_qk(0, zero, zero) && (k.n < 2 || issue_qk(1, zero, one));
#pragma unroll 1
                for (int j = 0; ok && j < k.n; j += 2) {
                    ok = issue_pv(j, (j >> 1) & 1, zero, zero) && (j + 2 >= k.n || issue_qk(j + 2, zero, zero)) &&
                         (j + 1 >= k.n || issue_pv(j + 1, (j >> 1) & 1, zero, one)) && (j + 3 >= k.n || issue_qk(j + 3, zero, one));
                }
            }
        };
        if (C::NRT == 2 && n_rt == 2)
            chain(std::integral_constant<int, C::NRT>{});
        else
            chain(std::integral_constant<int, 1>{});
        // Exit drain: whatever the loop issued has completed before tensor memory and the operand
        // buffers are released, even if a wait gave up.
        if (elect_one()) tc_commit(mma_drain);
        __syncwarp();
        mbar_wait(mma_drain, 0, f.status);
    } else {
        // ------------------------------------------------------------ softmax and epilogue of row tile rt
        const int rt = warp >> 2, quarter = warp & 3;
        if constexpr (C::QT > 0) {
            // the first columns of this thread's row into tensor memory
            const uint4* const src = reinterpret_cast<const uint4*>(f.q + paged_q_at(f, t, kvh, t.r0 + min(warp * 32 + lane, t.n - 1)));
            const uint32_t t_q = tmem + ((uint32_t)(quarter * 32) << 16) + C::Q_COL;
#pragma unroll 1
            for (int c = 0; c < C::QT / 64; c += 2) {
                uint32_t w[2][32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 v = as_operand(warp * 32 + lane < t.n ? __ldg(src + c * 8 + i) : make_uint4(0u, 0u, 0u, 0u));
                    w[i / 8][i % 8 * 4] = v.x;
                    w[i / 8][i % 8 * 4 + 1] = v.y;
                    w[i / 8][i % 8 * 4 + 2] = v.z;
                    w[i / 8][i % 8 * 4 + 3] = v.w;
                }
                const bool in = FMHA_IN_BOUNDS(C::Q_COL + c * 32 + 64 <= C::TMEM_COLS, kSitePagedTmem, f.status);
                tmem_st32u(t_q + (in ? c * 32 : 0), w[0]);
                tmem_st32u(t_q + (in ? c * 32 + 32 : 0), w[1]);
            }
            tmem_wait_st();
            tc_fence_before();
        }
        load_q(warp);
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
            // |scale| log2(e), not 0: a masked -inf times 0 would be a NaN (the smallest number, 2^-149, makes the weights of any
            // finite scores equal as it should)
            const float sl2 = fmaxf(fabsf(f.scale_log2), 1.40129846e-45f);
            float m_ref = -INFINITY, l = 0.f;
            int ahead = entry_of(0);  // block-table entries of a tile, loaded one tile ahead
            bool ok = true;
#pragma unroll 1
            for (int j = 0; j < k.n; ++j) {
                const int u = j * n_rt + rt, slot = u & 1;
                const unsigned pages = __ballot_sync(0xffffffffu, paged_page(f.c, ahead) >= 0);
                ahead = entry_of(j + 1);
                if (!wait_all(&s_full[slot], (u >> 1) & 1)) {
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
                auto load_scores = [&](int col, float (&x)[C::CH / 32][32]) {
#pragma unroll
                    for (int h = 0; h < C::CH / 32; ++h) tmem_ld32(s_addr + col + h * 32, x[h]);
                    tmem_wait_ld();
                    if (!full) {
#pragma unroll
                        for (int h = 0; h < C::CH / 32; ++h) {
                            const int first = key0 + col + h * 32;
                            const int k0 = max(0, lo - first), k1 = min(31, hi - first);
                            uint32_t in = k1 >= k0 ? (0xffffffffu >> (31 - k1)) & (0xffffffffu << k0) : 0u;
                            const unsigned p = pages >> ((col >> 4) + 2 * h);
                            in &= (p & 1u ? 0xffffu : 0u) | (p & 2u ? 0xffff0000u : 0u);
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[h][i] = (in >> i) & 1u ? x[h][i] : -INFINITY;
                        }
                    }
                };
                auto top_of = [&](const float (&x)[C::CH / 32][32]) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int h = 0; h < C::CH / 32; ++h)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[h][i], x[h][i + 1]));
                    return mx * sl2;
                };
                // The weights of C::CH scores from column col on, as packed pairs; false if a wait gave up.
                auto weights = [&](int col, uint32_t* pk) -> bool {
                    float x[C::CH / 32][32];
                    load_scores(col, x);
                    const float mt = top_of(x);
                    const bool move = mt > m_ref + kPast;  // true without a reference
                    if (__any_sync(0xffffffffu, move)) {
                        float alpha = 1.f;
                        if (move) {
                            if (m_ref == -INFINITY) {  // O and l are zero
                                m_ref = mt;
                            } else {
                                const float d = ceilf(mt - m_ref);
                                alpha = d < 127.f ? __uint_as_float((uint32_t)(127 - (int)d) << 23) : 0.f;
                                m_ref += d;
                                l *= alpha;
                            }
                        }
                        if (__any_sync(0xffffffffu, alpha != 1.f)) {
                            // O's rescale needs the PV before on this row tile; with two row tiles that completed before S did
                            if (j > 0) {
                                if (n_rt == 1 && !wait_all(&o_done[(u - 1) & 1], ((u - 1) >> 1) & 1)) return ok = false;
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
                            tmem_wait_st();
                            const uint32_t a16 = __float_as_uint(alpha) >> 16;
#pragma unroll 1
                            for (int c = 0; c < col / 2; c += 16) tmem_scale_pairs(s_addr + c, a16 | (a16 << 16));
                            tmem_wait_st();
                            load_scores(col, x);  // so that they need not be kept meanwhile
                        }
                    }
                    const float mu = m_ref == -INFINITY ? 0.f : -m_ref;
                    const uint64_t q2 = f32x2(sl2, sl2), mu2 = f32x2(mu, mu);
                    const uint64_t one2 = f32x2(1.f, 1.f);  // (a packed add takes twice as long as a packed fma)
                    uint64_t c2[2] = {0ull, 0ull};
#pragma unroll
                    for (int h = 0; h < C::CH / 32; ++h)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            f32x2_split(fma_f32x2(f32x2(x[h][2 * i], x[h][2 * i + 1]), q2, mu2), y0, y1);
                            y0 = ex2_approx(y0);
                            y1 = ex2_approx(y1);
                            pk[h * 16 + i] = pack_bf16x2(y0, y1);
                            c2[i & 1] = fma_f32x2(f32x2(y0, y1), one2, c2[i & 1]);
                        }
                    float a0, a1, b0, b1;
                    f32x2_split(c2[0], a0, a1);
                    f32x2_split(c2[1], b0, b1);
                    l += (a0 + a1) + (b0 + b1);
                    return true;
                };
                // P over S: columns col / 2 on take the weights of the scores from col on, which have been read
#pragma unroll 1
                for (int col = 0; col < BN; col += C::CH) {
                    uint32_t pk[C::CH / 2];
                    if (!weights(col, pk)) break;
                    if constexpr (C::CH == 64)
                        tmem_st32u(s_addr + col / 2, pk);
                    else
                        tmem_st16u(s_addr + col / 2, pk);
                }
                if (!ok) break;
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
            // through a 4 KB corner of the row tile's Q (or, with Q in tensor memory, of K) per warp, whose MMAs are done, so that a
            // store covers whole 64- or 128-byte pieces of rows
            uint8_t* stage = smem + (C::NRT == 2 ? rt * C::Q_TILE : 0) + quarter * 4096;
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
                    if (!FMHA_IN_BOUNDS(col + 32 <= HD && quarter * 4096 + 4096 <= (C::NRT == 2 ? C::Q_TILE : C::OFF_V), kSitePagedComb, f.status)) continue;
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
    using C = PTCfg<HD, CODES>;
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
    CUtensorMap tmk = {}, tmv = {};  // bf16 pages; without keys nothing is loaded
    if (!CODES && f.s_k > 0) {
        // [pool head][group of 8 rows][block][row of 8][64 columns], the order of the operand layout
        const cuuint64_t row = (cuuint64_t)HD * 2;
        const cuuint64_t dims[5] = {64, 8, HD / 64, (cuuint64_t)f.c.page / 8, (cuuint64_t)f.c.n_pages * f.c.n_kv_h};
        const cuuint64_t strides[4] = {row, 128, row * 8, row * f.c.page};
        const cuuint32_t box[5] = {64, 8, C::NB, (cuuint32_t)(f.c.page < C::BN ? f.c.page : C::BN) / 8, 1};
        if (encode_swizzled_map(&tmk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f.c.k_pages, dims, strides, box, 5) != CUDA_SUCCESS ||
            encode_swizzled_map(&tmv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f.c.v_pages, dims, strides, box, 5) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(f.row_tiles * C::PARTS * f.c.n_kv_h), f.n_splits);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tmk, tmv, f);
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

int paged_tc_kv_tile(int hd) { return hd <= 128 ? PTCfg<128, false>::BN : PTCfg<256, false>::BN; }
int paged_tc_rows(int hd) { return hd <= 128 ? 256 : 128; }

cudaError_t launch_paged_tc(const PagedFwd& f, cudaStream_t stream) {
    const bool sink = f.sink && f.n_splits == 1, codes = f.c.k_scales != nullptr;
    if (codes) return sink ? launch_s<true, true>(f, stream) : launch_s<true, false>(f, stream);
    return sink ? launch_s<false, true>(f, stream) : launch_s<false, false>(f, stream);
}

}  // namespace fmha
