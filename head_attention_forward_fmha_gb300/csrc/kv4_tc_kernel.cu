// kv4_tc_kernel.cu -- attention over a KV cache held in 4 bits for 128-row query
// tiles, on the tcgen05 tensor cores.
//
// One thread block owns 128 query rows that share a KV head and one chunk of
// that sequence's keys.  The cache's codes cannot feed the tensor cores (its scales
// cover 16 columns, and Q and P have no 4-bit form that keeps their bits), so
// eight warps turn each tile of codes into fp16 operands in shared memory --
// exact, see kv4_kernel.cu -- while the tensor cores work on the tile before:
//   S_j = Q K_j^T   tcgen05.mma M = 128, N = BN, K = hd    (both from shared memory)
//   O  += P_j V_j   tcgen05.mma M = 128, N = hd, K = BN    (P from tensor memory)
// At hd 512 two blocks share a row tile: each computes all of S and one 256-column
// half of O (which fills tensor memory next to S), and K's single stage is
// refilled in two column chunks, each as soon as the MMAs have read it.
//
// Warp roles (13 warps): 0..3 Q's conversion to fp16 (scaled by a power of two
// per row), then softmax and epilogue, one query row per thread; 4 tensor memory
// and MMA issue; 5..12 the conversion.  A conversion thread holds its share of two
// tiles in registers, so that their loads are in flight while it converts another.
//
// Measured on GB300: 128 tokens of 64/8 heads of 128 over 4 x 4096 keys 83 us, 823
// TFLOP/s; over a window of 2048 with four ragged lengths 29 to 51 us (eight sets of
// lengths; a sequence's chunk is one block's chain of tiles); 128 heads of 512 on one KV head,
// 16 ragged sequences up to 4096 keys 31 to 35 us.  A clock trace of a block says what
// bounds it.  At hd 128 a tile of 128 keys takes ~1900 clocks, of which the softmax
// warps ~1750 (the exponentials alone 512), with MMAs and conversion beside them; a tile
// in which the reference moves takes up to twice that.  At hd 512 a tile of 64 keys
// takes ~3000, the softmax ~1170 of them, and it waits ~1850 for S: with N = 64 its 32
// MMAs read Q (4 KB of shared memory each) for half as many keys as at N = 128, for
// which there is no room.  What mattered on the way: at hd 512 no spilled register, descriptors
// by addition among them (with 227 KB of shared memory there is hardly an L1, and
// each reload is a trip to L2), and conversion in coalesced pieces (75 -> 49 us);
// MMAs issued by an elected lane of a converged warp (49 -> 41); partials in fp16
// (39 -> 33), of empty chunks none (33 -> 31).  Small loops in the softmax (unrolled over the tile, the 4 x 4096 keys
// took 156 us instead of 94).  Two threads per row (17 warps, 96 registers) were
// slower: 113 us instead of 95 there, at hd 512 64 instead of 41.
#include <climits>
#include <atomic>
#include "internal.h"
#include "kv4_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

template <int HD>
struct K4TCfg {
    static constexpr int BM = 128;
    static constexpr int BN = HD <= 128 ? 128 : 64;       // keys per tile
    static constexpr int HDV = HD == 512 ? 256 : HD;      // columns of O per block
    static constexpr int PARTS = HD / HDV;                // blocks per row tile
    static constexpr int STG = HD == 512 ? 1 : 2;         // K and V stages
    static constexpr int NSB = 2;                         // S buffers
    static constexpr int Q_BYTES = BM * HD * 2;
    static constexpr int K_TILE = BN * HD * 2;
    static constexpr int V_TILE = BN * HDV * 2;
    static constexpr int THREADS = 13 * 32;
    static constexpr int CT = 256;                        // conversion threads
    static constexpr int NKC = HD == 512 ? 2 : 1;         // column chunks of a K tile, each with barriers of its own
    static constexpr int KCH = HD / NKC;                  // columns of a chunk
    static constexpr int KP = BN * KCH / 32 / CT;         // 32-column pieces of a K chunk, of V, per conversion thread
    static constexpr int VP = BN * HDV / 32 / CT;
    static constexpr int O_COL = NSB * BN;
    static constexpr int P_COL = O_COL + HDV;             // P buffers, BN / 2 columns of fp16 pairs each
    static constexpr int TMEM_COLS = 512;
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + STG * K_TILE;
    static constexpr int OFF_BAR = OFF_V + STG * V_TILE;
    static constexpr int N_BARS = 1 + 2 * STG * NKC + 2 * STG + 3 * NSB + 1;
    static constexpr int OFF_QS = OFF_BAR + N_BARS * 8 + 16;   // per-row factor of Q (before it: tensor-memory address, sequence, length)
    static constexpr int NEED = 1024 + OFF_QS + BM * 4;
    static constexpr int SMEM = NEED < 120000 ? 120000 : NEED;  // one block per SM: each takes all of tensor memory
    static_assert(P_COL + NSB * BN / 2 <= TMEM_COLS, "S, O and P fit in tensor memory");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct K4TArgs {
    Kv4Fwd f;
    int group, R;
    ScoreScale sl2;
    long long rows_total;
};

// 16 consecutive 32-bit columns of this thread's TMEM lane from raw words.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Instruction descriptor, kind::f16 with fp16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One conversion thread's share of a tile: N pieces of 32 columns (16 bytes of
// codes, two scales).  The tile's pieces, PPR per key, go round the CT threads in
// order, so a warp's load covers 512 neighbouring bytes (or whole 128-byte parts of
// rows).  Piece i of its key starts at column 32 i of the tile; STRIDE pieces lie
// between two keys in memory.
template <int N, int PPR, int STRIDE, int CT>
struct Pieces {
    uint4 codes[N];
    uint32_t scales[N];  // packing them would wait for the loads

    // c, s: piece 0 of the tile's first key; `keys` of them are there, `left` pieces up to the cache's end.
    __device__ __forceinline__ void load(int tid, const uint4* c, const unsigned short* s, int keys, long long left,
                                         unsigned* status) {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int idx = p * CT + tid, key = idx / PPR;
            const int at = STRIDE == PPR ? idx : key * STRIDE + idx % PPR;
            const bool live = key < keys && FMHA_IN_BOUNDS(at >= 0 && at < left, kSiteKv4Copy, status);
            codes[p] = live ? __ldg(c + at) : make_uint4(0u, 0u, 0u, 0u);
            scales[p] = live ? __ldg(s + at) : 0u;
        }
    }

    // As fp16 into a tile of 64-column boxes of `rows` 128-byte rows (16-byte
    // chunk c of row r at chunk c ^ (r % 8)).  A piece is four chunks; lanes take
    // theirs in different orders, c ^ x, so that eight lanes always store to eight
    // different chunk positions (bank groups).
    __device__ __forceinline__ void store(int tid, uint8_t* tile, int rows, unsigned* status) const {
#pragma unroll
        for (int p = 0; p < N; ++p) {
            const int idx = p * CT + tid;
            const int key = idx / PPR, i = idx % PPR;
            const int x = PPR == 4 ? (i >> 1) * 2 : (i >> 1) & 3;
            const uint32_t pair = e4m3x2_to_f16(scales[p]);
            uint32_t s0 = __byte_perm(pair, pair, 0x1010), s1 = __byte_perm(pair, pair, 0x3232);
            uint32_t w[4] = {codes[p].x, codes[p].y, codes[p].z, codes[p].w};
            if constexpr (PPR > 4) {
                const bool swap = x & 1;
                const uint32_t t0 = swap ? w[1] : w[0], t1 = swap ? w[0] : w[1];
                const uint32_t t2 = swap ? w[3] : w[2], t3 = swap ? w[2] : w[3];
                w[0] = t0; w[1] = t1; w[2] = t2; w[3] = t3;
            }
            if constexpr (PPR >= 4) {
                const bool swap = x & 2;
                const uint32_t t0 = swap ? w[2] : w[0], t1 = swap ? w[3] : w[1];
                const uint32_t t2 = swap ? w[0] : w[2], t3 = swap ? w[1] : w[3];
                w[0] = t0; w[1] = t1; w[2] = t2; w[3] = t3;
                const uint32_t u = swap ? s1 : s0;
                s1 = swap ? s0 : s1;
                s0 = u;
            }
            const int off = (i >> 1) * rows * 128 + key * 128;
            if (!FMHA_IN_BOUNDS(key < rows && off >= 0 && off + 128 <= rows * ((PPR + 1) / 2) * 128, kSiteKv4Key, status)) continue;
            uint8_t* row = tile + off;
            const int pos = ((i & 1) * 4) ^ x ^ (key & 7);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t r[4];
                e2m1x8_to_f16(w[c], r);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = mul_f16x2(r[e], c < 2 ? s0 : s1);
                *reinterpret_cast<uint4*>(row + ((pos ^ c) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
    }
};

template <int HD, bool SINK>
__global__ void __launch_bounds__(K4TCfg<HD>::THREADS, 1) kv4_tc_kernel(const K4TArgs a) {
    using C = K4TCfg<HD>;
    constexpr int BM = C::BM, BN = C::BN, NSB = C::NSB, STG = C::STG;
    const Kv4Fwd& f = a.f;
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
    uint64_t* s_full = v_empty + STG;    // [NSB]
    uint64_t* p_ready = s_full + NSB;    // [NSB]
    uint64_t* o_done = p_ready + NSB;    // [NSB]
    uint64_t* mma_drain = o_done + NSB;  // every MMA the issuer launched has completed (exit drain)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
    float* row_fac = reinterpret_cast<float*>(smem + C::OFF_QS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x / C::PARTS, part = blockIdx.x % C::PARTS;
    const int split = blockIdx.y;
    int b = blockIdx.z / f.n_kv_h;
    const int kvh = blockIdx.z - b * f.n_kv_h;
    const int r_begin = rt * BM;
    const int r_end = min(a.R, r_begin + BM);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 12 * 32);
        for (int s = 0; s < STG * C::NKC; ++s) {
            mbar_init(&k_full[s], C::CT);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < STG; ++s) {
            mbar_init(&v_full[s], C::CT);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < NSB; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_ready[s], 128);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(mma_drain, 1);
        mbar_fence_init();
    }
    grid_dependency_wait();  // every global access below follows the preceding kernel

    // Keys: the virtual axis of kv4_kernel.cu, with tiles of BN keys and a
    // window part that starts at its first key.
    // One warp reads the lengths for all: such that another stream changes meanwhile give results of any value, but no
    // warps that disagree on what the block does.
    int len = f.s_k;
    if (f.seq_lens) {
        int* const seq = reinterpret_cast<int*>(tmem_slot + 1);
        if (warp == 4) {
            if (f.n_splits == 1 && f.batch <= 32) {
                // Blocks start in the order of their index: with the longest sequence first,
                // the shortest fill the last gaps (chunks of 128 tokens over four ragged
                // sequences 38.6 -> 33.6 us).  Slot b holds the sequence that b others exceed.
                // Chunks are even without it (16 sequences in 8 chunks at hd 512: 33.0, sorted 36.6 us).
                const int mine = lane < f.batch ? seq_len(f, lane) : -1;
                int ahead = 0;
                for (int i = 0; i < f.batch; ++i) {
                    const int other = __shfl_sync(0xffffffffu, mine, i);
                    ahead += other > mine || (other == mine && i < lane);
                }
                b = __ffs(__ballot_sync(0xffffffffu, lane < f.batch && ahead == b)) - 1;
                len = __shfl_sync(0xffffffffu, mine, b);
            } else {
                len = seq_len(f, b);
            }
            if (lane == 0) {
                seq[0] = b;
                seq[1] = len;
            }
        }
        __syncthreads();
        b = __shfl_sync(0xffffffffu, seq[0], 0);
        len = __shfl_sync(0xffffffffu, seq[1], 0);
    }
    const int slab = b * f.n_kv_h + kvh;
    const long long row0 = ((long long)b * f.n_h + (long long)kvh * a.group) * f.T;  // slab's first query row
    const int n_first = f.window > 0 ? min(f.n_first, len) : 0;
    const int head_span = (n_first + BN - 1) / BN * BN;
    int body = 0;
    if (f.window > 0) body = max(n_first, max(0, len - f.T - f.window + 1));
    const long long v_lo = (long long)split * f.kv_chunk, v_hi = v_lo + f.kv_chunk;
    const int h_lo = (int)min(v_lo, (long long)head_span), h_hi = (int)min(v_hi, (long long)head_span);
    const int n_head = (h_hi - h_lo) / BN;
    const int b_lo = (int)min((long long)len, body + max(0LL, v_lo - head_span));
    int b_hi = (int)min((long long)len, body + max(0LL, v_hi - head_span));
    int u_lo = b_lo;
    {
        // ... that some row of this block attends
        int t0 = 0, t1 = f.T - 1;
        if (r_end - r_begin < f.T && (r_end - 1) % f.T >= r_begin % f.T) {
            t0 = r_begin % f.T;
            t1 = (r_end - 1) % f.T;
        }
        if (f.causal) b_hi = min(b_hi, len - f.T + t1 + 1);
        if (f.window > 0) u_lo = max(u_lo, len - f.T + t0 - f.window + 1);
    }
    const int n_body = b_hi > u_lo ? (b_hi - u_lo + BN - 1) / BN : 0;
    const int n_tiles = n_head + n_body;
    if (n_tiles == 0) {  // nothing to attend in this chunk: no tensor memory, no Q
        write_empty_rows(f, a.rows_total, row0 + r_begin, r_end - r_begin, split, part * C::HDV, C::HDV, part == 0,
                         SINK ? kvh * a.group : -1, r_begin);
        return;
    }
    if (warp == 4) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto tile_key = [&](int j) { return j < n_head ? h_lo + j * BN : u_lo + (j - n_head) * BN; };
    auto tile_end = [&](int j) { return j < n_head ? n_first : b_hi; };

    // Q's rows w, w + 12, ... of the tile (pairs or quads of rows at hd 128 and
    // 64) as fp16, scaled by a power of two per row and by the sign of the
    // scale, into 64-column boxes of 128 swizzled rows; all but the MMA warp
    // take part, w = 0 .. 11.
    auto load_q = [&](int w) {
        constexpr int LPR = HD >= 256 ? 32 : HD / 8, RPI = 32 / LPR, VEC = HD >= 256 ? HD / 256 : 1;
        constexpr int SETS = BM / RPI, BATCH = HD == 512 ? 3 : 6;
        const int lr = lane / LPR, lc = lane % LPR;
#pragma unroll 1
        for (int base = w; base < SETS; base += 12 * BATCH) {
            uint4 u[BATCH][VEC];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = (base + 12 * i) * RPI + lr;
                const bool live = row < BM && r_begin + row < r_end &&
                                  FMHA_IN_BOUNDS(row0 + r_begin + row >= 0 && row0 + r_begin + row < a.rows_total, kSiteKv4Q, f.status);
                const uint4* src = reinterpret_cast<const uint4*>(f.q + (row0 + r_begin + (live ? row : 0)) * HD);
#pragma unroll
                for (int v = 0; v < VEC; ++v) u[i][v] = live ? __ldg(src + v * 32 + lc) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int row = (base + 12 * i) * RPI + lr;
                uint32_t mx = 0;
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u[i][v].x & 0x7FFF7FFFu, u[i][v].y & 0x7FFF7FFFu),
                                               __vmaxu2(u[i][v].z & 0x7FFF7FFFu, u[i][v].w & 0x7FFF7FFFu)));
                mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, m));
                const int e = (int)(mx >> 7);
                const int k = (e > 0 && e < 255) ? min(max(14 - (e - 127), -120), 120) : 0;
                const float up = __uint_as_float((uint32_t)(127 + k) << 23) * a.sl2.sign;
                if (row >= BM) continue;
                if (lc == 0) row_fac[row] = score_factor(a.sl2.mant, a.sl2.expo - k);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const int col = v * 256 + lc * 8;
                    const uint32_t x[4] = {u[i][v].x, u[i][v].y, u[i][v].z, u[i][v].w};
                    uint32_t h[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) h[y] = pack_f16x2(bf16_lo(x[y]) * up, bf16_hi(x[y]) * up);
                    const int at = (col >> 6) * BM * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
                    if (FMHA_IN_BOUNDS(at >= 0 && at + 16 <= C::Q_BYTES, kSiteKv4Q, f.status))
                        *reinterpret_cast<uint4*>(sq + at) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
    };

    if (warp >= 5) {
        // ------------------------------------------------------------ conversion
        // K_0, K_1, V_0, K_2, V_1, ...: the order the MMA warp takes them in.
        // NBUF tiles of K and V are held in registers, their loads in flight
        // while others are converted.
        const int tid = threadIdx.x - 5 * 32;
        constexpr int NBUF = 2;
        constexpr int KPPR = C::KCH / 32, VPPR = C::HDV / 32, RP = HD / 32;
        Pieces<C::KP, KPPR, RP, C::CT> kb[NBUF][C::NKC];
        Pieces<C::VP, VPPR, RP, C::CT> vb[NBUF];
        const long long base = (long long)slab * f.cap * RP, total = (long long)f.batch * f.n_kv_h * f.cap * RP;
        const uint4* const kc = reinterpret_cast<const uint4*>(f.k_codes) + base;
        const uint4* const vc = reinterpret_cast<const uint4*>(f.v_codes) + base + part * VPPR;
        const unsigned short* const ks = reinterpret_cast<const unsigned short*>(f.k_scales) + base;
        const unsigned short* const vs = reinterpret_cast<const unsigned short*>(f.v_scales) + base + part * VPPR;
        auto keys_of = [&](int j, long long& at) {
            const int k0 = tile_key(j), n = min(BN, tile_end(j) - k0);
            at = (long long)k0 * RP;
            return FMHA_IN_BOUNDS(k0 >= 0 && k0 + n <= f.cap, kSiteKv4Copy, f.status) ? n : 0;
        };
        auto fetch_k = [&](auto& p, int j) {
            long long at;
            const int n = keys_of(j, at);
#pragma unroll
            for (int c = 0; c < C::NKC; ++c)
                p[c].load(tid, kc + at + c * KPPR, ks + at + c * KPPR, n, total - base - at - c * KPPR, f.status);
        };
        auto fetch_v = [&](auto& p, int j) {
            long long at;
            const int n = keys_of(j, at);
            p.load(tid, vc + at, vs + at, n, total - base - at - part * VPPR, f.status);
        };
#pragma unroll
        for (int i = 0; i < NBUF; ++i)
            if (i < n_tiles) {
                fetch_k(kb[i], i);
                fetch_v(vb[i], i);
            }
        load_q(warp - 1);
        bool ok = true;
        // K_j and then V_{j-1}, for j up to n_tiles (where there is no K_j)
#pragma unroll 1
        for (int j0 = 0; ok && j0 <= n_tiles; j0 += NBUF) {
#pragma unroll
            for (int i = 0; i < NBUF; ++i) {
                const int j = j0 + i;
                if (!ok || j > n_tiles) continue;
                const int s = STG == 1 ? 0 : j & 1;
                if (j < n_tiles) {
#pragma unroll
                    for (int c = 0; c < C::NKC; ++c) {
                        const int q = s * C::NKC + c;
                        ok = ok && (j < STG || mbar_wait(&k_empty[q], ((j / STG) - 1) & 1, f.status));
                        if (ok && FMHA_IN_BOUNDS(s < STG, kSiteKv4Key, f.status)) {
                            kb[i][c].store(tid, sk + s * C::K_TILE + c * (C::K_TILE / C::NKC), BN, f.status);
                            fence_proxy_async_smem();
                            mbar_arrive(&k_full[q]);
                        }
                    }
                    if (j + NBUF < n_tiles) fetch_k(kb[i], j + NBUF);
                }
                if (j > 0) {
                    constexpr int LAST = NBUF - 1;
                    auto& v = vb[i == 0 ? LAST : i - 1];
                    const int jv = j - 1, sv_ = STG == 1 ? 0 : jv & 1;
                    ok = ok && (jv < STG || mbar_wait(&v_empty[sv_], ((jv / STG) - 1) & 1, f.status));
                    if (ok && FMHA_IN_BOUNDS(sv_ < STG, kSiteKv4Key, f.status)) {
                        v.store(tid, sv + sv_ * C::V_TILE, BN, f.status);
                        fence_proxy_async_smem();
                        mbar_arrive(&v_full[sv_]);
                        if (jv + NBUF < n_tiles) fetch_v(v, jv + NBUF);
                    }
                }
            }
        }
    } else if (warp == 4) {
        // ------------------------------------------------------------ MMA issuer
        // Order: QK_0 .. QK_{NSB-1}, then per tile j: PV_j, QK_{j+NSB}.
        // The whole warp walks the loop and one elected lane issues, so that the
        // descriptors stay in uniform registers: issued by `lane == 0` alone, each MMA
        // took ~95 clocks (hd 512: 3000 per tile of 32) however small it was.
        {
            constexpr uint32_t idesc_s = idesc_f16_f32(BM, BN, 0);
            constexpr uint32_t idesc_o = idesc_f16_f32(BM, C::HDV, 1);
            // A descriptor's low word holds the address in units of 16 bytes: the
            // operands of a step are a constant distance from the stage's first.
            const uint64_t q_desc = smem_desc_sw128(smem_u32(sq), 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(smem_u32(sk), 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(sv), BN * 128, 1024);
            bool ok = mbar_wait(q_full, 0, f.status);
            auto issue_qk = [&](int j) -> bool {
                const int s = STG == 1 ? 0 : j & 1;
                const uint32_t d = tmem + (j % NSB) * BN;
                if (!FMHA_IN_BOUNDS(s >= 0 && s < STG && C::OFF_K + (s + 1) * C::K_TILE <= C::OFF_V, kSiteKv4Desc, f.status) ||
                    !FMHA_IN_BOUNDS(d - tmem + BN <= C::O_COL, kSiteKv4Tmem, f.status))
                    return false;
                const uint64_t b0 = k_desc + s * (C::K_TILE / 16);
#pragma unroll 1
                for (int c = 0; c < C::NKC; ++c) {
                    if (!mbar_wait(&k_full[s * C::NKC + c], (j / STG) & 1, f.status)) return false;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int y = 0; y < C::KCH / 64; ++y) {  // 64-column boxes
                            const int x = c * (C::KCH / 64) + y;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)  // 16 columns = 32 bytes into the swizzled row
                                tc_mma_f16(d, q_desc + x * (BM * 128 / 16) + kk * 2, b0 + x * (BN * 128 / 16) + kk * 2, idesc_s,
                                           (c > 0 || y > 0 || kk > 0) ? 1u : 0u);
                        }
                        tc_commit(&k_empty[s * C::NKC + c]);
                        if (c == C::NKC - 1) tc_commit(&s_full[j % NSB]);
                    }
                    __syncwarp();
                }
                return true;
            };
            for (int j = 0; ok && j < NSB && j < n_tiles; ++j) ok = issue_qk(j);
            for (int j = 0; ok && j < n_tiles; ++j) {
                const int s = STG == 1 ? 0 : j & 1, pb = j % NSB;
                if (!mbar_wait(&v_full[s], (j / STG) & 1, f.status)) break;
                if (!mbar_wait(&p_ready[pb], (j / NSB) & 1, f.status)) break;
                tc_fence_after();
                const uint64_t b0 = v_desc + s * (C::V_TILE / 16);
                const uint32_t p_col = tmem + C::P_COL + pb * (BN / 2);
                if (!FMHA_IN_BOUNDS(s >= 0 && s < STG && C::OFF_V + (s + 1) * C::V_TILE <= C::OFF_BAR, kSiteKv4Desc, f.status) ||
                    !FMHA_IN_BOUNDS(p_col - tmem + BN / 2 <= C::TMEM_COLS, kSiteKv4Tmem, f.status))
                    break;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        tc_mma_f16_ts(tmem + C::O_COL, p_col + kk * 8, b0 + kk * (16 * 128 / 16), idesc_o,
                                      (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&o_done[pb]);
                    tc_commit(&v_empty[s]);
                }
                __syncwarp();
                if (j + NSB < n_tiles && !issue_qk(j + NSB)) break;
            }
            // Exit drain: whatever the loop issued has completed before tensor
            // memory and the operand buffers are released, even if a wait gave up.
            if (elect_one()) tc_commit(mma_drain);
            __syncwarp();
            mbar_wait(mma_drain, 0, f.status);
        }
    } else {
        load_q(warp);
        // ------------------------------------------------------------ softmax
        const int row = threadIdx.x;  // tile row and TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        auto o_addr = [&](int c) {  // columns 32 c .. 32 c + 31 of O
            return t_lane + C::O_COL + (FMHA_IN_BOUNDS(warp < 4 && c * 32 + 32 <= C::HDV, kSiteKv4Tmem, f.status) ? c * 32 : 0);
        };
        const int grow = r_begin + row;
        const bool valid = grow < r_end;
        int jlo = INT_MAX, jhi = -1, fhi = -1;
        if (valid) {
            const int p = len - f.T + grow % f.T;
            jlo = u_lo;
            jhi = b_hi - 1;
            fhi = n_first - 1;
            if (f.causal) {
                jhi = min(jhi, p);
                fhi = min(fhi, p);
            }
            if (f.window > 0) jlo = max(jlo, p - f.window + 1);
        }
        float m_ref = -INFINITY, l = 0.f;
        bool ok = mbar_wait(q_full, 0, f.status);
        const float qs = ok && FMHA_IN_BOUNDS(row >= 0 && row < BM, kSiteKv4Q, f.status) ? row_fac[row] : 1.f;
        for (int j = 0; ok && j < n_tiles; ++j) {
            const int pb = j % NSB;
            if (!mbar_wait(&s_full[pb], (j / NSB) & 1, f.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t s_addr = t_lane + pb * BN;
            const int key0 = tile_key(j);
            const int lo = j < n_head ? 0 : jlo, hi = j < n_head ? fhi : jhi;
            const bool full = key0 >= lo && key0 + BN - 1 <= hi;
            const uint32_t p_addr = t_lane + C::P_COL + pb * (BN / 2);
            float alpha = 1.f;
            // The row's scores from column `col` of the tile on, those outside [lo, hi] at
            // -inf.  64 at a time: each wait for tensor memory costs (by 32, 4 x 4096 keys at hd
            // 128 take 90 instead of 84 us); the maximum by 32 where there is one pass
            // of 64 anyway (by 64 it spills at hd 512, 46 instead of 41 us).
            auto load_scores = [&](int col, auto& x) {
                constexpr int N = sizeof(x) / sizeof(x[0]);
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    const bool in = FMHA_IN_BOUNDS(pb * BN + col + h * 32 + 32 <= C::O_COL, kSiteKv4Tmem, f.status);
                    tmem_ld32(s_addr + (in ? col + h * 32 : 0), x[h]);
                }
                tmem_wait_ld();
                if (!full) {
#pragma unroll
                    for (int h = 0; h < N; ++h) {
                        const int first = key0 + col + h * 32;
                        const int k0 = max(0, lo - first), k1 = min(31, hi - first);
                        const uint32_t in = k1 >= k0 ? (0xffffffffu >> (31 - k1)) & (0xffffffffu << k0) : 0u;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[h][i] = (in >> i) & 1u ? x[h][i] : -INFINITY;
                    }
                }
            };
            // P against the present reference; S stays as it is.  Usually the reference
            // stands; where a row of the warp has none yet, or a P came out above
            // 2^14 (a score above the reference by more than 8), it moves to the
            // tile's maximum first and the tile is done (again).  The loops are kept
            // small: unrolled over the tile, this one ran at 0.6 of its speed.  The P
            // buffer is free: S_j's QK was queued after PV_{j-NSB}, which read it.
            bool move = m_ref == -INFINITY;
#pragma unroll 1
            for (int again = 0; again < 2; ++again) {
                if (__any_sync(0xffffffffu, move)) {
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int col = 0; col < BN; col += BN / 2) {
                        float x[BN / 64][32];
                        load_scores(col, x);
#pragma unroll
                        for (int h = 0; h < BN / 64; ++h)
#pragma unroll
                            for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[h][i], x[h][i + 1]));
                    }
                    const float mt = mx * qs;
                    if (mt > m_ref + 8.f) {
                        alpha = ex2_approx(m_ref - mt);  // 0 when the reference was -inf
                        m_ref = mt;
                        l *= alpha;
                    }
                    again = 1;  // within 8 of the maximum now
                }
                const float mu = kPBias - (m_ref == -INFINITY ? 0.f : m_ref);
                uint64_t s2[2] = {0ull, 0ull};
                uint32_t top = 0u;
                const uint64_t q2 = f32x2(qs, qs), mu2 = f32x2(mu, mu);
#pragma unroll 1
                for (int col = 0; col < BN; col += 64) {
                    float x[2][32];
                    load_scores(col, x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            f32x2_split(fma_f32x2(f32x2(x[h][2 * i], x[h][2 * i + 1]), q2, mu2), y0, y1);
                            y0 = ex2_approx(y0);
                            y1 = ex2_approx(y1);
                            pk[i] = pack_f16x2(y0, y1);
                            top = __vmaxu2(top, pk[i]);  // not negative: fp16 bits compare as integers
                            s2[i & 1] = add_f32x2(s2[i & 1], f32x2(y0, y1));
                        }
                        const bool in = FMHA_IN_BOUNDS(col / 2 + h * 16 + 16 <= BN / 2 && pb < NSB, kSiteKv4Tmem, f.status);
                        tmem_st16u(p_addr + (in ? col / 2 + h * 16 : 0), pk);
                    }
                }
                move = max(top & 0xFFFFu, top >> 16) > 0x7400u;  // 2^14
                if (again == 0 && __any_sync(0xffffffffu, move)) {
                    tmem_wait_st();  // P is written to the same columns once more
                    continue;
                }
                float a0, a1, b0, b1;
                f32x2_split(s2[0], a0, a1);
                f32x2_split(s2[1], b0, b1);
                l += (a0 + a1) + (b0 + b1);
                break;
            }
            // a rescale of O needs PV_{j-1}
            const bool rescale = j > 0 && __any_sync(0xffffffffu, alpha != 1.f);
            if (rescale && !mbar_wait(&o_done[(j - 1) % NSB], ((j - 1) / NSB) & 1, f.status)) {
                ok = false;
                break;
            }
            if (rescale) {
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
            tc_fence_before();
            mbar_arrive(&p_ready[pb]);
        }
        // ------------------------------------------------------------ epilogue
        if (ok) ok = mbar_wait(&o_done[(n_tiles - 1) % NSB], ((n_tiles - 1) / NSB) & 1, f.status);
        ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld below is warp-collective
        tc_fence_after();
        float inv, lse;
        finish_row_nan(m_ref - kPBias, l,
                   (SINK && valid) ? sink_log2_of(f.sink, kvh * a.group + grow / f.T, f.n_h, f.status) : -INFINITY, inv, lse);
        inv *= f.v_global;
        const long long gr = row0 + grow;
        const bool store = valid && ok && FMHA_IN_BOUNDS(gr >= 0 && gr < a.rows_total && split < f.n_splits, kSiteKv4Out, f.status);
        const long long prow = (long long)split * a.rows_total + gr;
        if (ok) {
            float range = 1.f;
            if constexpr (HD == 512) {
                if (f.n_splits > 1) {
                    // fp16 partials, scaled per row half so that the largest |O| lies in
                    // [2^14, 2^15), and the factor that undoes it
                    float mx = 0.f;
#pragma unroll 1
                    for (int c = 0; c < C::HDV / 32; ++c) {
                        float ov[32];
                        tmem_ld32(o_addr(c), ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(ov[i]));
                    }
                    mx *= inv;
                    const int e = (int)((__float_as_uint(mx) >> 23) & 0xffu) - 127;
                    if (mx > 0.f && e < 128) {  // leave zero, inf and NaN rows as they are
                        const int k = min(max(e - 14, -100), 100);
                        inv *= __uint_as_float((uint32_t)(127 - k) << 23);
                        range = __uint_as_float((uint32_t)(127 + k) << 23);
                    }
                    if (store && FMHA_IN_BOUNDS(prow >= 0 && prow < f.n_splits * a.rows_total && part < 2, kSiteKv4Range, f.status))
                        f.range_part[prow * 2 + part] = range;
                }
            }
            // partials go through a 4 KB corner of Q's place per warp (its MMAs are
            // done), so that a store covers 128 (fp16: 64) bytes of a row
            uint8_t* stage = sq + warp * 4096;
            const unsigned rows_live = __ballot_sync(0xffffffffu, store);
#pragma unroll 1
            for (int c = 0; c < C::HDV / 32; ++c) {
                float ov[32];
                tmem_ld32(o_addr(c), ov);
                tmem_wait_ld();
                const int col = part * C::HDV + c * 32;
                if (f.n_splits == 1) {
                    if (!store || !FMHA_IN_BOUNDS(col + 32 <= HD, kSiteKv4Out, f.status)) continue;
                    uint4* dst = reinterpret_cast<uint4*>(f.o + gr * HD + col);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        dst[q] = make_uint4(pack_bf16x2(ov[8 * q] * inv, ov[8 * q + 1] * inv),
                                            pack_bf16x2(ov[8 * q + 2] * inv, ov[8 * q + 3] * inv),
                                            pack_bf16x2(ov[8 * q + 4] * inv, ov[8 * q + 5] * inv),
                                            pack_bf16x2(ov[8 * q + 6] * inv, ov[8 * q + 7] * inv));
                } else if (FMHA_IN_BOUNDS(col + 32 <= HD && warp * 4096 + 4096 <= C::Q_BYTES, kSiteKv4Comb, f.status)) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                            make_float4(ov[4 * q] * inv, ov[4 * q + 1] * inv, ov[4 * q + 2] * inv, ov[4 * q + 3] * inv);
                    __syncwarp();
                    const long long at = ((long long)split * a.rows_total + row0 + r_begin + warp * 32) * HD + col;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // 4 rows of 8 x 16 bytes
                        const int r = i * 4 + (lane >> 3), q = lane & 7;
                        if (!((rows_live >> r) & 1u)) continue;
                        const float4 v = *reinterpret_cast<const float4*>(stage + r * 128 + ((q ^ (r & 7)) << 4));
                        if constexpr (HD == 512)
                            *reinterpret_cast<uint2*>(static_cast<__half*>(f.o_part) + at + (long long)r * HD + q * 4) =
                                make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(static_cast<float*>(f.o_part) + at + (long long)r * HD + q * 4) = v;
                    }
                    __syncwarp();
                }
            }
        }
        if (store && part == 0) {
            if (f.n_splits == 1)
                f.lse[gr] = lse;
            else
                f.lse_part[prow] = lse;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int HD, bool SINK>
cudaError_t launch_t(const Kv4Fwd& f, cudaStream_t stream) {
    using C = K4TCfg<HD>;
    auto kern = kv4_tc_kernel<HD, SINK>;
    static std::atomic<bool> attr_set[128];  // set once per device; any host thread may set it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 128) attr_set[dev] = true;
    }
    K4TArgs a;
    a.f = f;
    a.group = f.n_h / f.n_kv_h;
    a.R = a.group * f.T;
    a.sl2 = score_scale(f);
    a.rows_total = (long long)f.batch * f.n_h * f.T;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.R + C::BM - 1) / C::BM * C::PARTS, f.n_splits, f.batch * f.n_kv_h);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool SINK>
cudaError_t launch_s(const Kv4Fwd& f, cudaStream_t stream) {
    switch (f.hd) {
        case 64: return launch_t<64, SINK>(f, stream);
        case 128: return launch_t<128, SINK>(f, stream);
        case 256: return launch_t<256, SINK>(f, stream);
        case 512: return launch_t<512, SINK>(f, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int kv4_tc_kv_tile(int hd) { return hd <= 128 ? K4TCfg<128>::BN : K4TCfg<256>::BN; }
int kv4_tc_blocks_per_row_tile(int hd) { return hd == 512 ? K4TCfg<512>::PARTS : 1; }

cudaError_t launch_kv4_tc(const Kv4Fwd& f, cudaStream_t stream) {
    return f.sink && f.n_splits == 1 ? launch_s<true>(f, stream) : launch_s<false>(f, stream);
}

}  // namespace fmha
