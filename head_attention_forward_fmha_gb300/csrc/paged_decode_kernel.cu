// paged_decode_kernel.cu -- attention over a cache in pages for few query rows per KV head.
//
// One thread block handles RT (8 or 16) query rows of one sequence that share a KV head, and
// one chunk of that sequence's key tiles.  A producer warp streams the tiles from HBM through a ring
// of TMA boxes (128-byte swizzle): its lanes look the tile's pages up in the block table, one
// tile ahead, and issue the boxes of the pages (a page that is not there is a box
// behind the pool, which the TMA fills with zeros).  Four consumer warps, eight for codes, each take 16
// keys of a tile, which lie in one page:
//   S^T = K Q^T     mma.sync m16n8k16, keys as M, so that 8 query rows fill N = 8
//   O^T += V^T P^T  keys as the reduction dimension; P transposed in registers (movmatrix)
// with the online softmax between them, and merge their partial states at the end.
//
// 8-bit pages: the codes become fp16 operands in registers, by the hardware's exact conversion (one
// instruction for two codes; the step to bf16 took 4.5, and the kernel half its rate: 16 sequences of 16384
// keys at hd 128 137 us).  Scales stay outside the MMAs: K's multiply the scores, V's the weights, in
// fp32.  What fp16 asks for in range is kept apart as powers of two: Q's rows are scaled to a largest element in
// [2^14, 2^15) (elements below 2^-28 of it lose bits), P carries a factor 2^12, and V's scales are taken
// relative to the largest that the warp has met, O being kept in units of it (weights whose V lies
// more than 2^26 below that lose bits).  V's operand is loaded by ldmatrix with
// transposition on pairs of codes, so that rows g and g + 8 of the A operand are columns 2 g and 2 g + 1.
//
// What bounds it: bf16 is memory (16 sequences of 16384 keys, 32 query heads on 8 of 128: 161 us, 6.7 TB/s in pages of 16 and 154 in
// pages of 64; a plain copy's rate with a window of 4096 in 32 sequences); a block takes in 36 KB a us at most, so short
// batches are split until there are two blocks for each SM.  In 8 bits (111 us, 4.9 TB/s; pages of 64 103) the ALUs' 44 % and the latencies of
// ldmatrix, conversion and shuffles in turn: eight consumer warps instead of four brought 137 -> 107 us.
// 16 rows for 9 and more: twice the accumulators for the same keys read once (one block per SM for codes); at
// hd 512 they would spill.
#include <atomic>
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

template <int HD, int NB, bool CODES>
struct PDCfg {
    static constexpr int RT = 8 * NB;                  // query rows per block
    static constexpr int NCW = CODES ? 8 : 4;          // consumer warps
    static constexpr int KW = HD <= 128 ? NCW : NCW / 2;  // key groups of 16 keys
    static constexpr int DW = NCW / KW;                // warps that share a key group's columns in P V
    static constexpr int KT = 16 * KW;                 // keys per tile
    static constexpr int HDW = HD / DW;                // columns of O per warp
    static constexpr int THREADS = (NCW + 1) * 32;
    static constexpr int ROW = CODES ? HD : HD * 2;    // bytes of a stored row
    static constexpr int TILE_BYTES = KT * ROW;
    static constexpr int BOX_BYTES = ROW < 128 ? TILE_BYTES : KT * 128;  // 128 bytes wide
    static constexpr int NBOX = TILE_BYTES / BOX_BYTES;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int STAGES = STAGE_BYTES <= 16384 ? 6 : 3;
    static constexpr int Q_STRIDE = HD * 2 + 16;       // padded row
    static constexpr int Q_BYTES = RT * Q_STRIDE;
    static constexpr int SC_BYTES = CODES ? 2 * KT : 0;  // scale bytes of a stage: K's, then V's
    static constexpr int OFF_Q = STAGES * STAGE_BYTES;
    static constexpr int OFF_BAR = OFF_Q + Q_BYTES;
    static constexpr int OFF_LIVE = OFF_BAR + 2 * STAGES * 8;  // per stage: a bit for each 16 keys that are there
    static constexpr int OFF_SC = OFF_LIVE + (STAGES * 4 + 15) / 16 * 16;
    static constexpr int OFF_QE = OFF_SC + STAGES * SC_BYTES;  // codes: power of two of each Q row
    static constexpr int OFF_ML = OFF_QE + (CODES ? RT * 4 : 0);
    static constexpr int OFF_TILE = OFF_ML + KW * RT * 12 + 16;  // (the abort flag's 16 bytes before it)
    static constexpr int SMEM = 1024 + OFF_TILE + 32;
    static_assert(OFF_TILE % 4 == 0 && sizeof(PagedTile) <= 32, "the block's rows");
    static_assert(KW <= 8 && KW * RT * HD * 4 <= STAGES * STAGE_BYTES, "the combine buffer reuses the ring");
};

__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// One arrival on the barrier when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

template <int HD, int NB, bool CODES, bool SINK>
__global__ void __launch_bounds__(PDCfg<HD, NB, CODES>::THREADS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const PagedFwd f) {
    using C = PDCfg<HD, NB, CODES>;
    launch_dependents();  // the merge grid may be scheduled now; it waits for this grid's results
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stages = smem;
    uint8_t* qs = smem + C::OFF_Q;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint32_t* live = reinterpret_cast<uint32_t*>(smem + C::OFF_LIVE);
    uint8_t* scales = smem + C::OFF_SC;
    int* q_exp = reinterpret_cast<int*>(smem + C::OFF_QE);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [KW][RT] (max, sum) per key group
    int* v_exp = reinterpret_cast<int*>(ml + C::KW * C::RT);   // [KW] codes: unit of a group's O
    int* abort_flag = v_exp + C::KW * C::RT;
    PagedTile* tile = reinterpret_cast<PagedTile*>(smem + C::OFF_TILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.x % f.c.n_kv_h, split = blockIdx.y;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], CODES ? 33 : 1);
            mbar_init(&empty[s], C::NCW);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    grid_dependency_wait();  // every global access below follows the preceding kernel
    // One warp reads which rows and keys are the block's, for all: lengths or bounds that another stream changes meanwhile give
    // results of any value, but no two warps that wait for each other at different barriers.
    if (warp == C::NCW) {
        const PagedTile mine = paged_tile_by_keys<C::RT>(f, blockIdx.x / f.c.n_kv_h, f.status);
        if (lane == 0) *tile = mine;
    }
    __syncthreads();
    const PagedTile t = paged_tile_from(tile);
    if (t.n <= 0) return;
    // A tile's boxes: of min(page, KT) keys each, from a multiple of that on.
    const int box_keys = min(f.c.page, C::KT);
    const PagedKeys k = paged_keys(f, t, split, C::KT, box_keys);
    if (k.n <= 0) {
        paged_write_empty(f, t, kvh, split, 0, HD);
        return;
    }

    // ------------------------------------------------------------ producer
    if (warp == C::NCW) {
        const int log_pages = __ffs(C::KT / box_keys) - 1;                 // boxes along a tile's keys (and NBOX across)
        const int box_rows = CODES && HD == 64 ? box_keys / 2 : box_keys;  // rows of 128 bytes (two keys at 64 bytes each)
        if (lane == 0) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
        const uint64_t pol = l2_policy_evict_first();
        // the block table one tile ahead, by 16 keys: granule `lane`
        auto entry = [&](int it) {
            if (it >= k.n || 16 * lane >= C::KT) return -1;
            const int key = k.key(it, C::KT) + 16 * lane;
            return key < k.to(it) ? paged_entry(f.c, f.t.batch, t.b, key >> f.c.log_page, f.status) : -1;
        };
        int issued = 0, ahead = entry(0);
        for (int it = 0; it < k.n; ++it) {
            const int s = it % C::STAGES, page = paged_page(f.c, ahead), key = k.key(it, C::KT);
            ahead = entry(it + 1);
            // (all lanes go on or none: collectives follow)
            if (it >= C::STAGES && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((it / C::STAGES) - 1) & 1, f.status))) break;
            const unsigned there = __ballot_sync(0xffffffffu, page >= 0);
            uint8_t* kst = stages + s * C::STAGE_BYTES;
            if (lane == 0) {
                live[s] = there;
                mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
            }
            __syncwarp();
            // box i: K's and then V's, of each first all pages of the first 128 bytes' columns
            for (int i0 = 0; i0 < 2 * C::NBOX << log_pages; i0 += 32) {
                const int i = i0 + lane, mine = i & ((1 << log_pages) - 1), col = (i >> log_pages) % C::NBOX, v = (i >> log_pages) / C::NBOX;
                const int bp = __shfl_sync(0xffffffffu, page, mine * (box_keys >> 4) & 31);  // the box begins with that granule
                const int slab = bp < 0 ? f.c.n_pages * f.c.n_kv_h : bp * f.c.n_kv_h + kvh;  // behind the pool: zeros
                const int row = ((key + mine * box_keys) & (f.c.page - 1)) / (box_keys / box_rows);
                const int at = v * C::TILE_BYTES + col * C::BOX_BYTES + mine * box_rows * 128;
                if (v < 2 && FMHA_IN_BOUNDS(s < C::STAGES && row >= 0 && row + box_rows <= f.c.page / (box_keys / box_rows) &&
                                                at + box_rows * 128 <= C::STAGE_BYTES,
                                            kSitePagedKv, f.status))
                    tma_load_3d_hint(kst + at, v ? &tmv : &tmk, col * (CODES ? 128 : 64), row, slab, &full[s], pol);
            }
            if constexpr (CODES) {
                // scale bytes, four keys a lane
                const int row = __shfl_sync(0xffffffffu, paged_row(f.c, page, kvh, key + 16 * lane), lane >> 2) + (lane & 3) * 4;
                if (lane < C::KT / 4) {
                    const bool ok = row >= (lane & 3) * 4 && FMHA_IN_BOUNDS(paged_row_ok(f.c, row + 3LL), kSitePagedRow, f.status);
                    cp_async4(scales + s * C::SC_BYTES + lane * 4, f.c.k_scales + (ok ? row : 0), ok);
                    cp_async4(scales + s * C::SC_BYTES + C::KT + lane * 4, f.c.v_scales + (ok ? row : 0), ok);
                }
                cp_async_arrive(&full[s]);
            }
            ++issued;
        }
        // Exit drain: what this warp loaded has landed before the block may exit.
        drain_ring(full, C::STAGES, issued, f.status);
        return;
    }

    // ------------------------------------------------------------ consumers
    const int kw = warp / C::DW, dw = warp - kw * C::DW;

    // Q rows -> shared memory (zero rows past the end); for codes as fp16 times a power of two of the row
    if constexpr (!CODES) {
        for (int i = threadIdx.x; i < C::RT * (HD / 8); i += C::NCW * 32) {
            const int r = i / (HD / 8), c8 = i - r * (HD / 8);
            uint4 val = make_uint4(0, 0, 0, 0);
            if (r < t.n) val = __ldg(reinterpret_cast<const uint4*>(f.q + paged_q_at(f, t, kvh, t.r0 + r) + c8 * 8));
            if (FMHA_IN_BOUNDS(r * C::Q_STRIDE + c8 * 16 + 16 <= C::Q_BYTES, kSitePagedQ, f.status))
                *reinterpret_cast<uint4*>(qs + r * C::Q_STRIDE + c8 * 16) = val;
        }
    } else {
        constexpr int LPR = HD >= 256 ? 32 : HD / 8, VEC = HD / 8 / LPR;  // lanes of a row, 16-byte pieces of a lane
        for (int r0 = warp * (32 / LPR); r0 < C::RT; r0 += C::NCW * (32 / LPR)) {
            const int r = r0 + lane / LPR, lc = lane % LPR;
            uint4 u[VEC];
            uint32_t mx = 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                u[v] = make_uint4(0, 0, 0, 0);
                if (r < t.n) u[v] = __ldg(reinterpret_cast<const uint4*>(f.q + paged_q_at(f, t, kvh, t.r0 + r) + (v * LPR + lc) * 8));
                mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u[v].x & 0x7FFF7FFFu, u[v].y & 0x7FFF7FFFu), __vmaxu2(u[v].z & 0x7FFF7FFFu, u[v].w & 0x7FFF7FFFu)));
            }
            mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
            for (int s = LPR / 2; s > 0; s >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            const int e = (int)(mx >> 7), up = e < 255 ? min(max(14 - (e - 127), -120), 120) : 0;
            const float fac = __uint_as_float((uint32_t)(127 + up) << 23);
            if (lc == 0 && FMHA_IN_BOUNDS(r < C::RT, kSitePagedQ, f.status)) q_exp[r] = up;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const uint32_t x[4] = {u[v].x, u[v].y, u[v].z, u[v].w};
                uint32_t h[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) h[y] = pack_f16x2(bf16_lo(x[y]) * fac, bf16_hi(x[y]) * fac);
                const int at = r * C::Q_STRIDE + (v * LPR + lc) * 16;
                if (FMHA_IN_BOUNDS(r < C::RT && at + 16 <= C::Q_BYTES, kSitePagedQ, f.status)) *reinterpret_cast<uint4*>(qs + at) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }

    // Keys of each accumulator row of this thread (rows nb * 8 + 2 * (lane % 4) + i), and those that every row attends.
    int jlo[NB][2], jhi[NB][2], fhi[NB][2];
    int all_lo = 0, all_hi = INT_MAX, all_f = INT_MAX;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = t.r0 + nb * 8 + 2 * (lane & 3) + i;
            paged_row_keys(f, t, k, r, jlo[nb][i], jhi[nb][i], fhi[nb][i]);
            if (r < t.r0 + t.n) {
                all_lo = max(all_lo, jlo[nb][i]);
                all_hi = min(all_hi, jhi[nb][i]);
                all_f = min(all_f, fhi[nb][i]);
            }
        }
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, s));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, s));
        all_f = min(all_f, __shfl_xor_sync(0xffffffffu, all_f, s));
    }

    float m[NB][2], l[NB][2];
    float o[C::HDW / 16][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
        for (int db = 0; db < C::HDW / 16; ++db) o[db][nb][0] = o[db][nb][1] = o[db][nb][2] = o[db][nb][3] = 0.f;
    }
    named_barrier_sync(1, C::NCW * 32);  // Q staged

    // Codes: the scale's power of two goes with those of the rows of Q and K, so that a score leaves fp32's range only if its value does.
    int scale_exp = 0;
    const float sl2 = CODES ? frexpf(f.scale_log2, &scale_exp) : f.scale_log2;
    int row_exp[NB][2], v_unit = 0;  // codes: power of two of Q's rows over the scale's; unit of O, as a scale byte
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) row_exp[nb][i] = CODES ? q_exp[nb * 8 + 2 * (lane & 3) + i] - scale_exp : 0;
    const uint32_t qs_addr = smem_u32(qs);
    const int g = lane >> 2, t4 = lane & 3;
    constexpr float kBias = CODES ? 12.f : 0.f;  // log2 of the factor that P and its sum carry
    bool ok = true;

    for (int it = 0; it < k.n; ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait(&full[s], (it / C::STAGES) & 1, f.status)) {
            ok = false;
            break;
        }
        const uint32_t kst = smem_u32(stages + s * C::STAGE_BYTES);
        const uint32_t vst = kst + C::TILE_BYTES;
        const int kb = k.key(it, C::KT) + 16 * kw;  // this warp's first key
        const bool there = (live[s] >> kw) & 1u;

        // S^T (16 keys x RT rows) = K Q^T
        float sc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
        if constexpr (!CODES) {
            const int k_row = 16 * kw + (lane & 15), k_c8 = lane >> 4;
            const uint32_t q_addr = qs_addr + ((lane & 7) + (NB >= 2 ? 8 * (lane >> 4) : 0)) * C::Q_STRIDE + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const int d = 16 * kk + 8 * k_c8;
                uint32_t ka = kst + (d >> 6) * C::BOX_BYTES + k_row * 128 + ((((d & 63) >> 3) ^ (k_row & 7)) << 4);
                if (!FMHA_IN_BOUNDS(ka >= kst && ka + 16 <= kst + C::TILE_BYTES, kSitePagedLds, f.status)) ka = kst;
                uint32_t a0, a1, a2, a3;
                ldsm_x4(ka, a0, a1, a2, a3);
                uint32_t qa = q_addr + kk * 32;
                if (!FMHA_IN_BOUNDS(qa >= qs_addr && qa + 16 <= qs_addr + C::Q_BYTES, kSitePagedLds, f.status)) qa = qs_addr;
                uint32_t bq[NB][2];
                if constexpr (NB == 1)
                    ldsm_x2(qa, bq[0][0], bq[0][1]);
                else
                    ldsm_x4(qa, bq[0][0], bq[0][1], bq[1][0], bq[1][1]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(sc[nb], a0, a1, a2, a3, bq[nb][0], bq[nb][1]);
            }
        } else {
            // Thread (g, t4) takes columns 32 kk + 8 t4 .. + 7 of keys g and g + 8, and of query rows g.
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) {
                uint2 w[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int key = 16 * kw + g + 8 * y, d = 32 * kk + 8 * t4;
                    const int row = HD == 64 ? key >> 1 : key, byte = HD == 64 ? (key & 1) * 64 + d : d & 127;
                    uint32_t ka = kst + (HD == 64 ? 0 : d >> 7) * C::BOX_BYTES + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 8);
                    if (!FMHA_IN_BOUNDS(ka >= kst && ka + 8 <= kst + C::TILE_BYTES, kSitePagedLds, f.status)) ka = kst;
                    w[y] = lds64(ka);
                }
                uint32_t a[2][4];  // words 0 and 1 of keys g and g + 8
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    e4m3x4_to_f16(w[y].x, a[0][y], a[0][2 + y]);
                    e4m3x4_to_f16(w[y].y, a[1][y], a[1][2 + y]);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    uint32_t qa = qs_addr + (nb * 8 + g) * C::Q_STRIDE + (32 * kk + 8 * t4) * 2;
                    if (!FMHA_IN_BOUNDS(qa + 16 <= qs_addr + C::Q_BYTES, kSitePagedLds, f.status)) qa = qs_addr;
                    const uint4 q = lds128(qa);
                    mma_f16_16816(sc[nb], a[0][0], a[0][1], a[0][2], a[0][3], q.x, q.y);
                    mma_f16_16816(sc[nb], a[1][0], a[1][1], a[1][2], a[1][3], q.z, q.w);
                }
            }
        }

        // scale, mask, online softmax (log2 domain)
        const bool in_head = k.head(it);
        const int need_lo = in_head ? 0 : all_lo, need_hi = in_head ? all_f : all_hi;
        const bool edge = !there || kb < need_lo || kb + 15 > need_hi;
        const int j0 = kb + g, j1 = j0 + 8;
        uint32_t ke[2] = {127u, 127u};             // scale bytes of K's rows g and g + 8
        float v0 = 1.f, v1 = 1.f, to_unit = 1.f;  // factors of their V rows in units of O, of O so far
        if constexpr (CODES) {
            const uint8_t* ks = scales + s * C::SC_BYTES + 16 * kw + g;
            ke[0] = ks[0];
            ke[1] = ks[8];
            uint32_t b0 = ks[C::KT], b1 = ks[C::KT + 8];
            if (edge) {
                // a key that no row attends has no factor, whatever memory holds there
                if (!there || j0 < k.from(it) || j0 >= k.to(it)) b0 = 0u;
                if (!there || j1 < k.from(it) || j1 >= k.to(it)) b1 = 0u;
            }
            uint32_t top = max(b0 == 255u ? 0u : b0, b1 == 255u ? 0u : b1);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
            const int unit = max(v_unit, (int)top);
            auto power = [](int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + e) << 23); };
            to_unit = power(v_unit - unit);
            v_unit = unit;
            v0 = b0 == 255u ? NAN : power((int)b0 - unit);
            v1 = b1 == 255u ? NAN : power((int)b1 - unit);
        }
        uint32_t pb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float mx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x0 = sc[nb][i] * sl2, x1 = sc[nb][2 + i] * sl2;
                if constexpr (CODES) {
                    // times K's scale, the power of two that undoes Q's, and the attention's scale
                    auto power = [&](uint32_t byte) {
                        return byte == 255u ? NAN : __uint_as_float((uint32_t)min(max((int)byte - row_exp[nb][i], 1), 254) << 23);
                    };
                    x0 = sc[nb][i] * power(ke[0]) * sl2;
                    x1 = sc[nb][2 + i] * power(ke[1]) * sl2;
                }
                if (edge) {
                    const int lo = in_head ? 0 : jlo[nb][i], hi = in_head ? fhi[nb][i] : jhi[nb][i];
                    x0 = (there && j0 >= lo && j0 <= hi) ? x0 : -INFINITY;
                    x1 = (there && j1 >= lo && j1 <= hi) ? x1 : -INFINITY;
                }
                sc[nb][i] = x0;
                sc[nb][2 + i] = x1;
                mx[i] = fmaxf(x0, x1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 4));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 8));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 16));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[nb][i], mx[i]);
                const float mu = (mn == -INFINITY) ? 0.f : mn;
                const float alpha = exp2f(m[nb][i] - mu);
                m[nb][i] = mn;
                const float p0 = exp2f(sc[nb][i] - mu + kBias);
                const float p1 = exp2f(sc[nb][2 + i] - mu + kBias);
                l[nb][i] = l[nb][i] * alpha + p0 + p1;
                sc[nb][i] = CODES ? p0 * v0 : p0;
                sc[nb][2 + i] = CODES ? p1 * v1 : p1;
                const float fac = CODES ? alpha * to_unit : alpha;
#pragma unroll
                for (int db = 0; db < C::HDW / 16; ++db) {
                    o[db][nb][i] *= fac;
                    o[db][nb][2 + i] *= fac;
                }
            }
            pb[nb][0] = movmatrix_t(CODES ? pack_f16x2(sc[nb][0], sc[nb][1]) : pack_bf16x2(sc[nb][0], sc[nb][1]));
            pb[nb][1] = movmatrix_t(CODES ? pack_f16x2(sc[nb][2], sc[nb][3]) : pack_bf16x2(sc[nb][2], sc[nb][3]));
        }

        // O^T (columns x RT rows) += V^T P^T
        // keys 2 t4, 2 t4 + 1 and those 8 further on: which of them V's operand keeps
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (edge) {
            auto pair = [&](int key) {
                const bool a = there && key >= k.from(it) && key < k.to(it), b = there && key + 1 >= k.from(it) && key + 1 < k.to(it);
                return (a ? 0xffffu : 0u) | (b ? 0xffff0000u : 0u);
            };
            keep0 = pair(kb + 2 * t4);
            keep1 = pair(kb + 2 * t4 + 8);
        }
        if constexpr (!CODES) {
            const int v_row = 16 * kw + (lane & 7) + 8 * (lane >> 4), v_c8 = (lane >> 3) & 1;
#pragma unroll
            for (int db = 0; db < C::HDW / 16; ++db) {
                const int d = dw * C::HDW + 16 * db + 8 * v_c8;
                uint32_t va = vst + (d >> 6) * C::BOX_BYTES + v_row * 128 + ((((d & 63) >> 3) ^ (v_row & 7)) << 4);
                if (!FMHA_IN_BOUNDS(va >= vst && va + 16 <= vst + C::TILE_BYTES, kSitePagedLds, f.status)) va = vst;
                uint32_t a0, a1, a2, a3;
                ldsm_x4_t(va, a0, a1, a2, a3);
                if (edge) {
                    a0 &= keep0;
                    a1 &= keep0;
                    a2 &= keep1;
                    a3 &= keep1;
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(o[db][nb], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
            }
        } else {
            // matrices of ldmatrix: keys 0 .. 7 and 8 .. 15, of 16 columns and of the next 16
            const int key = 16 * kw + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
            for (int db = 0; db < C::HDW / 32; ++db) {
                const int d = dw * C::HDW + 32 * db + 16 * (lane >> 4);
                const int row = HD == 64 ? key >> 1 : key, byte = HD == 64 ? (key & 1) * 64 + d : d & 127;
                uint32_t va = vst + (HD == 64 ? 0 : d >> 7) * C::BOX_BYTES + row * 128 + (((byte >> 4) ^ (row & 7)) << 4);
                if (!FMHA_IN_BOUNDS(va >= vst && va + 16 <= vst + C::TILE_BYTES, kSitePagedLds, f.status)) va = vst;
                uint32_t r[4];
                ldsm_x4_t(va, r[0], r[1], r[2], r[3]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    // two keys of column 2 g, then of column 2 g + 1.  (What memory holds at keys that no row
                    // attends may be the codes' NaN: it counts as 0.)
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16(__byte_perm(r[2 * y], 0u, 0x3120), a0, a1);
                    e4m3x4_to_f16(__byte_perm(r[2 * y + 1], 0u, 0x3120), a2, a3);
                    if (edge) {
                        a0 &= keep0;
                        a1 &= keep0;
                        a2 &= keep1;
                        a3 &= keep1;
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_f16_16816(o[2 * db + y][nb], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------------------ epilogue
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 4);
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 8);
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 16);
        }
    if (!ok) atomicOr(abort_flag, 1);
    named_barrier_sync(1, C::NCW * 32);  // every warp is done with the ring
    if (*abort_flag) return;

    if (dw == 0 && lane < 4) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int mi = kw * C::RT + nb * 8 + 2 * lane + i;
                if (FMHA_IN_BOUNDS(mi >= 0 && mi < C::KW * C::RT, kSitePagedComb, f.status)) ml[mi] = make_float2(m[nb][i], l[nb][i]);
            }
        if (CODES && lane == 0) v_exp[kw] = v_unit;
    }
    named_barrier_sync(1, C::NCW * 32);

    // This warp's O, relative to the row's maximum over all key groups
    float* comb = reinterpret_cast<float*>(stages);  // [KW][RT][HD]
    int common = 0;  // codes: the largest of the groups' units, in which the sum is formed
    float to_common = 1.f;
    if constexpr (CODES) {
#pragma unroll
        for (int w = 0; w < C::KW; ++w) common = max(common, v_exp[w]);
        to_common = v_unit - common < -126 ? 0.f : __uint_as_float((uint32_t)(127 + v_unit - common) << 23);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = nb * 8 + 2 * t4 + i;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::KW; ++w) M = fmaxf(M, ml[w * C::RT + r].x);
            float fac = exp2f(m[nb][i] - ((M == -INFINITY) ? 0.f : M));
            if constexpr (CODES) fac *= to_common;
#pragma unroll
            for (int db = 0; db < C::HDW / 16; ++db) {
                // rows g and g + 8 of the operand: columns g and g + 8 of 16, for codes 2 g and 2 g + 1
                const int d = dw * C::HDW + 16 * db + (CODES ? 2 * g : g);
                const int ci = (kw * C::RT + r) * HD + d;
                if (!FMHA_IN_BOUNDS(ci >= 0 && ci + (CODES ? 1 : 8) < C::KW * C::RT * HD, kSitePagedComb, f.status)) continue;
                comb[ci] = o[db][nb][i] * fac;
                comb[ci + (CODES ? 1 : 8)] = o[db][nb][2 + i] * fac;
            }
        }
    named_barrier_sync(1, C::NCW * 32);

    // Sum of the key groups, one divide by the running sum (plus the sink)
    for (int item = threadIdx.x; item < C::RT * (HD / 8); item += C::NCW * 32) {
        const int r = item / (HD / 8), d8 = item - r * (HD / 8);
        if (r >= t.n) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::KW; ++w) M = fmaxf(M, ml[w * C::RT + r].x);
        const float Mu = (M == -INFINITY) ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < C::KW; ++w) L += ml[w * C::RT + r].y * exp2f(ml[w * C::RT + r].x - Mu);
        int head;
        const long long row = paged_out_row(f, t, kvh, t.r0 + r, head);
        float inv, lse;
        paged_finish(M - kBias, L, SINK ? sink_log2_of(f.sink, head, f.n_h, f.status) : -INFINITY, inv, lse);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < C::KW; ++w) {
            const float4* src = reinterpret_cast<const float4*>(comb + (w * C::RT + r) * HD + d8 * 8);
            const float4 u0 = src[0], u1 = src[1];
            acc[0] += u0.x; acc[1] += u0.y; acc[2] += u0.z; acc[3] += u0.w;
            acc[4] += u1.x; acc[5] += u1.y; acc[6] += u1.z; acc[7] += u1.w;
        }
        if constexpr (CODES) {  // out of O's units; the divide first, within fp32's range
            const float unit = paged_scale((uint32_t)common);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = acc[e] * inv * unit;
            inv = 1.f;
        }
        if (!FMHA_IN_BOUNDS(row >= 0 && row < f.rows && split < f.n_splits, kSitePagedOut, f.status)) continue;
        if (f.n_splits == 1) {
            uint4 pk;
            pk.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
            pk.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
            pk.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
            pk.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
            *reinterpret_cast<uint4*>(f.o + row * HD + d8 * 8) = pk;
            if (d8 == 0) f.lse[row] = lse;
        } else {
            const long long prow = split * f.rows + row;
            float4* dst = reinterpret_cast<float4*>(f.o_part + prow * HD + d8 * 8);
            dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
            if (d8 == 0) f.lse_part[prow] = lse;
        }
    }
}

template <int HD, int NB, bool CODES, bool SINK>
cudaError_t launch_t(const PagedFwd& f, cudaStream_t stream) {
    using C = PDCfg<HD, NB, CODES>;
    auto kern = paged_decode_kernel<HD, NB, CODES, SINK>;
    static std::atomic<bool> attr_set[128];  // set once per device; any host thread may set it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 128) attr_set[dev] = true;
    }
    // The pool as rows of 64 bf16 or 128 codes per box; rows of 64 codes in pairs.
    const int box_keys = f.c.page < C::KT ? f.c.page : C::KT, per_row = CODES && HD == 64 ? 2 : 1;
    const cuuint64_t row_bytes = (cuuint64_t)C::ROW * per_row;
    const cuuint64_t dims[3] = {CODES ? row_bytes : (cuuint64_t)HD, (cuuint64_t)(f.c.page / per_row), (cuuint64_t)f.c.n_pages * f.c.n_kv_h};
    const cuuint64_t strides[2] = {row_bytes, (cuuint64_t)f.c.page * C::ROW};
    const cuuint32_t box[3] = {CODES ? 128u : 64u, (cuuint32_t)(box_keys / per_row), 1};
    const CUtensorMapDataType type = CODES ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tmk = {}, tmv = {};  // without keys nothing is loaded
    if (f.s_k > 0 && (encode_swizzled_map(&tmk, type, f.c.k_pages, dims, strides, box, 3) != CUDA_SUCCESS ||
        encode_swizzled_map(&tmv, type, f.c.v_pages, dims, strides, box, 3) != CUDA_SUCCESS))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(f.row_tiles * f.c.n_kv_h), f.n_splits);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tmk, tmv, f);
}

template <bool CODES, bool SINK>
cudaError_t launch_s(const PagedFwd& f, int rows, cudaStream_t stream) {
    switch (f.c.hd) {
        case 64: return rows == 16 ? launch_t<64, 2, CODES, SINK>(f, stream) : launch_t<64, 1, CODES, SINK>(f, stream);
        case 128: return rows == 16 ? launch_t<128, 2, CODES, SINK>(f, stream) : launch_t<128, 1, CODES, SINK>(f, stream);
        case 256: return rows == 16 ? launch_t<256, 2, CODES, SINK>(f, stream) : launch_t<256, 1, CODES, SINK>(f, stream);
        case 512: return launch_t<512, 1, CODES, SINK>(f, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int paged_decode_kv_tile(int hd, bool codes) {
    return codes ? (hd <= 128 ? PDCfg<128, 1, true>::KT : PDCfg<256, 1, true>::KT) : hd <= 128 ? PDCfg<128, 1, false>::KT : PDCfg<256, 1, false>::KT;
}
int paged_decode_rows(int hd, long long rows) { return rows > 8 && hd <= 256 ? 16 : 8; }

cudaError_t launch_paged_decode(const PagedFwd& f, int rows, cudaStream_t stream) {
    const bool sink = f.sink && f.n_splits == 1, codes = f.c.k_scales != nullptr;
    if (codes) return sink ? launch_s<true, true>(f, rows, stream) : launch_s<true, false>(f, rows, stream);
    return sink ? launch_s<false, true>(f, rows, stream) : launch_s<false, false>(f, rows, stream);
}

}  // namespace fmha
