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
// half of O (which fills tensor memory next to S).
//
// Warp roles (13 warps): 0..3 Q's conversion to fp16 (scaled by a power of two
// per row), then softmax and epilogue, one query row per thread; 4 tensor memory
// and MMA issue; 5..8 K's conversion; 9..12 V's conversion.  A conversion thread
// holds part of one key's row: its loads for the next tile are in flight
// while it converts this one, and eight lanes store to eight different
// 16-byte columns of the swizzled tile.
//
// Bounded by the tensor cores and the softmax beside the conversion: per 128 keys
// at hd 128 the MMAs take ~1000 clocks, the exponentials 512 and the
// conversion's stores 512 of the SM's shared-memory writes.
#include <climits>
#include <atomic>
#include "internal.h"
#include "ptx.cuh"

namespace fmha {
namespace {

constexpr float kPBias = 6.f;  // log2 of the factor that P and its sum carry (kv4_kernel.cu)

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
    static constexpr int TPK = 128 / BN;                  // conversion threads per key
    static constexpr int KCOLS = HD / TPK, VCOLS = HDV / TPK;  // columns per conversion thread
    static constexpr int O_COL = NSB * BN;
    static constexpr int P_COL = O_COL + HDV;             // P buffers, BN / 2 columns of fp16 pairs each
    static constexpr int TMEM_COLS = 512;
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + STG * K_TILE;
    static constexpr int OFF_BAR = OFF_V + STG * V_TILE;
    static constexpr int N_BARS = 1 + 4 * STG + 3 * NSB + 1;
    static constexpr int OFF_QS = OFF_BAR + N_BARS * 8 + 16;   // per-row factor of Q
    static constexpr int NEED = 1024 + OFF_QS + BM * 4;
    static constexpr int SMEM = NEED < 120000 ? 120000 : NEED;  // one block per SM: each takes all of tensor memory
    static_assert(P_COL + NSB * BN / 2 <= TMEM_COLS, "S, O and P fit in tensor memory");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct K4TArgs {
    Kv4Fwd f;
    int group, R;
    float sl2, sl2_sign;  // as in kv4_kernel.cu
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

// Codes and scales of COLS consecutive columns of one key.
template <int COLS>
struct RowPart {
    uint4 codes[COLS / 32];
    uint32_t scales[COLS / 64];

    __device__ __forceinline__ void load(const uint8_t* c, const uint8_t* s, bool live) {
#pragma unroll
        for (int i = 0; i < COLS / 32; ++i)
            codes[i] = live ? __ldg(reinterpret_cast<const uint4*>(c) + i) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (COLS == 64) {
            scales[0] = live ? __ldg(reinterpret_cast<const unsigned int*>(s)) : 0u;
        } else if constexpr (COLS == 128) {
            const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(s)) : make_uint2(0u, 0u);
            scales[0] = v.x; scales[1] = v.y;
        } else {
            const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(s)) : make_uint4(0u, 0u, 0u, 0u);
            scales[0] = v.x; scales[1] = v.y; scales[2] = v.z; scales[3] = v.w;
        }
    }

    // As fp16 into row `key` of a tile of 64-column boxes of `rows` 128-byte
    // rows (16-byte chunk c of row r at chunk c ^ (r % 8)), from column col0 on.
    __device__ __forceinline__ void store(uint8_t* tile, int rows, int key, int col0) const {
#pragma unroll
        for (int b = 0; b < COLS / 16; ++b) {  // 16-column blocks
            const uint32_t pair = e4m3x2_to_f16(scales[b / 4] >> (16 * ((b / 2) & 1)));
            const uint32_t s2 = __byte_perm(pair, pair, b & 1 ? 0x3232 : 0x1010);
            const uint4 c4 = codes[b / 2];
            const uint32_t w[2] = {b & 1 ? c4.z : c4.x, b & 1 ? c4.w : c4.y};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[4];
                e2m1x8_to_f16(w[h], r);
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = mul_f16x2(r[e], s2);
                const int col = col0 + b * 16 + h * 8;
                uint8_t* dst = tile + (col >> 6) * rows * 128 + key * 128 + ((((col & 63) >> 3) ^ (key & 7)) << 4);
                *reinterpret_cast<uint4*>(dst) = make_uint4(r[0], r[1], r[2], r[3]);
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
    uint64_t* k_empty = k_full + STG;
    uint64_t* v_full = k_empty + STG;
    uint64_t* v_empty = v_full + STG;
    uint64_t* s_full = v_empty + STG;    // [NSB]
    uint64_t* p_ready = s_full + NSB;    // [NSB]
    uint64_t* o_done = p_ready + NSB;    // [NSB]
    uint64_t* mma_drain = o_done + NSB;  // every MMA the issuer launched has completed (exit drain)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BARS);
    float* row_fac = reinterpret_cast<float*>(smem + C::OFF_QS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x / C::PARTS, part = blockIdx.x % C::PARTS;
    const int split = blockIdx.y, slab = blockIdx.z;
    const int b = slab / f.n_kv_h, kvh = slab - b * f.n_kv_h;
    const long long row0 = ((long long)b * f.n_h + (long long)kvh * a.group) * f.T;  // slab's first query row
    const int r_begin = rt * BM;
    const int r_end = min(a.R, r_begin + BM);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        for (int s = 0; s < STG; ++s) {
            mbar_init(&k_full[s], 128);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 128);
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
    if (warp == 4) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();  // every global access below follows the preceding kernel

    // Keys: the virtual axis of kv4_kernel.cu, with tiles of BN keys and a
    // window part that starts at its first key.
    const int len = f.seq_lens ? min(max(__ldg(f.seq_lens + b), 0), f.s_k) : f.s_k;
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
    auto tile_key = [&](int j) { return j < n_head ? h_lo + j * BN : u_lo + (j - n_head) * BN; };
    auto tile_end = [&](int j) { return j < n_head ? n_first : b_hi; };

    if (warp >= 5) {
        // ------------------------------------------------------------ conversion
        const bool is_v = warp >= 9;
        const int tid = threadIdx.x - (is_v ? 9 : 5) * 32;
        const int key = tid % BN, sub = tid / BN;
        auto convert = [&](auto part_type, uint8_t* tiles, int tile_bytes, const uint8_t* codes, const uint8_t* scales,
                           uint64_t* full, uint64_t* empty, int col0, int smem_col0) {
            using Part = decltype(part_type);
            Part cur, next;
            auto fetch = [&](Part& p, int j) {
                const int k = tile_key(j) + key;
                const bool live = k < tile_end(j) && FMHA_IN_BOUNDS(k >= 0 && k < f.cap, kSiteKv4Copy, f.status);
                const long long r = (long long)slab * f.cap + (live ? k : 0);
                p.load(codes + r * (HD / 2) + col0 / 2, scales + r * (HD / 16) + col0 / 16, live);
            };
            if (n_tiles > 0) fetch(cur, 0);
            for (int j = 0; j < n_tiles; ++j) {
                const int s = j % STG;
                if (j + 1 < n_tiles) fetch(next, j + 1);
                if (j >= STG && !mbar_wait(&empty[s], ((j / STG) - 1) & 1, f.status)) break;
                cur.store(tiles + s * tile_bytes, BN, key, smem_col0);
                fence_proxy_async_smem();
                mbar_arrive(&full[s]);
                cur = next;
            }
        };
        if (is_v)
            convert(RowPart<C::VCOLS>{}, sv, C::V_TILE, f.v_codes, f.v_scales, v_full, v_empty,
                    part * C::HDV + sub * C::VCOLS, sub * C::VCOLS);
        else
            convert(RowPart<C::KCOLS>{}, sk, C::K_TILE, f.k_codes, f.k_scales, k_full, k_empty, sub * C::KCOLS,
                    sub * C::KCOLS);
    } else if (warp == 4) {
        // ------------------------------------------------------------ MMA issuer
        // Order: QK_0 .. QK_{NSB-1}, then per tile j: PV_j, QK_{j+NSB}.
        if (lane == 0 && n_tiles > 0) {
            constexpr uint32_t idesc_s = idesc_f16_f32(BM, BN, 0);
            constexpr uint32_t idesc_o = idesc_f16_f32(BM, C::HDV, 1);
            const uint32_t q_addr = smem_u32(sq), k_addr = smem_u32(sk), v_addr = smem_u32(sv);
            bool ok = mbar_wait(q_full, 0, f.status);
            auto issue_qk = [&](int j) -> bool {
                const int s = j % STG;
                if (!mbar_wait(&k_full[s], (j / STG) & 1, f.status)) return false;
                tc_fence_after();
                const uint32_t d = tmem + (j % NSB) * BN;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off = (kk & 3) * 32;  // 16 columns = 32 bytes into the swizzled row
                    const uint64_t ad = smem_desc_sw128(q_addr + (kk >> 2) * BM * 128 + off, 16, 1024);
                    const uint64_t bd = smem_desc_sw128(k_addr + s * C::K_TILE + (kk >> 2) * BN * 128 + off, 16, 1024);
                    tc_mma_f16(d, ad, bd, idesc_s, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[j % NSB]);
                tc_commit(&k_empty[s]);
                return true;
            };
            for (int j = 0; ok && j < NSB && j < n_tiles; ++j) ok = issue_qk(j);
            for (int j = 0; ok && j < n_tiles; ++j) {
                const int s = j % STG, pb = j % NSB;
                if (!mbar_wait(&v_full[s], (j / STG) & 1, f.status)) break;
                if (!mbar_wait(&p_ready[pb], (j / NSB) & 1, f.status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    const uint64_t bd = smem_desc_sw128(v_addr + s * C::V_TILE + kk * 16 * 128, BN * 128, 1024);
                    tc_mma_f16_ts(tmem + C::O_COL, tmem + C::P_COL + pb * (BN / 2) + kk * 8, bd, idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(&o_done[pb]);
                tc_commit(&v_empty[s]);
                if (j + NSB < n_tiles && !issue_qk(j + NSB)) break;
            }
            // Exit drain: whatever the loop issued has completed before tensor
            // memory and the operand buffers are released, even if a wait gave up.
            tc_commit(mma_drain);
            mbar_wait(mma_drain, 0, f.status);
        }
    } else {
        // ------------------------------------------------------------ Q
        // A warp takes its 32 rows; lanes hold 8 columns each (16 lanes or 8 per
        // row at hd 128 and 64).  The sign of the scale goes into Q.
        constexpr int LPR = HD >= 256 ? 32 : HD / 8, RPI = 32 / LPR, VEC = HD >= 256 ? HD / 256 : 1;
        if (n_tiles > 0) {
            const int lr = lane / LPR, lc = lane % LPR;
#pragma unroll 4
            for (int i = 0; i < 32 / RPI; ++i) {
                const int row = warp * 32 + i * RPI + lr;
                const bool live = r_begin + row < r_end;
                const uint4* src = reinterpret_cast<const uint4*>(f.q + (row0 + r_begin + (live ? row : 0)) * HD);
                uint4 u[VEC];
                uint32_t mx = 0;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    u[v] = live ? __ldg(src + v * 32 + lc) : make_uint4(0u, 0u, 0u, 0u);
                    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(u[v].x & 0x7FFF7FFFu, u[v].y & 0x7FFF7FFFu),
                                               __vmaxu2(u[v].z & 0x7FFF7FFFu, u[v].w & 0x7FFF7FFFu)));
                }
                mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, m));
                const int e = (int)(mx >> 7);
                const int k = (e > 0 && e < 255) ? min(max(14 - (e - 127), -120), 120) : 0;
                const float up = __uint_as_float((uint32_t)(127 + k) << 23) * a.sl2_sign;
                if (lc == 0) row_fac[row] = __uint_as_float((uint32_t)(127 - k) << 23) * a.sl2;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const int col = v * 256 + lc * 8;
                    const uint32_t w[4] = {u[v].x, u[v].y, u[v].z, u[v].w};
                    uint32_t h[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) h[x] = pack_f16x2(bf16_lo(w[x]) * up, bf16_hi(w[x]) * up);
                    *reinterpret_cast<uint4*>(sq + (col >> 6) * BM * 128 + row * 128 +
                                              ((((col & 63) >> 3) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
            __syncwarp();  // row_fac of this warp's rows
        }
        // ------------------------------------------------------------ softmax
        const int row = threadIdx.x;  // tile row and TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
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
        const float qs = n_tiles > 0 ? row_fac[row] : 1.f;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
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
            float sum = 0.f, mx = -INFINITY;
            // P of the whole tile against the present reference, its sum, and the
            // tile's largest score; S stays as it is.  The P buffer is free: S_j's QK
            // was queued after PV_{j-NSB}, which read it.
            auto pass = [&](bool exps) {
                const float mu = kPBias - (m_ref == -INFINITY ? 0.f : m_ref);
                sum = 0.f;
                mx = -INFINITY;
                uint64_t s2[2] = {0ull, 0ull};
                const uint64_t q2 = f32x2(qs, qs), mu2 = f32x2(mu, mu);
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    float x[32];
                    tmem_ld32(s_addr + c * 32, x);
                    tmem_wait_ld();
                    if (!full) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int key = key0 + c * 32 + i;
                            x[i] = (key >= lo && key <= hi) ? x[i] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[i], x[i + 1]));
                    if (exps) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y0, y1;
                            f32x2_split(fma_f32x2(f32x2(x[2 * i], x[2 * i + 1]), q2, mu2), y0, y1);
                            y0 = ex2_approx(y0);
                            y1 = ex2_approx(y1);
                            pk[i] = pack_f16x2(y0, y1);
                            s2[i & 1] = add_f32x2(s2[i & 1], f32x2(y0, y1));
                        }
                        tmem_st16u(p_addr + c * 16, pk);
                    }
                }
                float a0, a1, b0, b1;
                f32x2_split(s2[0], a0, a1);
                f32x2_split(s2[1], b0, b1);
                sum = (a0 + a1) + (b0 + b1);
            };
            // Usually the reference stands; where a row of the warp has none yet or
            // exceeds it by more than 8, it moves to the tile's maximum first.
            bool redo = __any_sync(0xffffffffu, m_ref == -INFINITY);
            pass(!redo);
            float alpha = 1.f;
            const float mt = mx * qs;
            const bool grow_ref = mt > m_ref + 8.f;
            redo = __any_sync(0xffffffffu, grow_ref) || redo;
            if (redo) {
                if (grow_ref) {
                    alpha = ex2_approx(m_ref - mt);  // 0 when the reference was -inf
                    m_ref = mt;
                    l *= alpha;
                }
                pass(true);
            }
            l += sum;
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
                    tmem_ld32(t_lane + C::O_COL + c * 32, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] *= alpha;
                    tmem_st32(t_lane + C::O_COL + c * 32, ov);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_ready[pb]);
        }
        // ------------------------------------------------------------ epilogue
        if (ok && n_tiles > 0) ok = mbar_wait(&o_done[(n_tiles - 1) % NSB], ((n_tiles - 1) / NSB) & 1, f.status);
        ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld below is warp-collective
        tc_fence_after();
        float inv, lse;
        finish_row(m_ref - kPBias, l,
                   (SINK && valid) ? sink_log2_of(f.sink, kvh * a.group + grow / f.T, f.n_h, f.status) : -INFINITY, inv, lse);
        inv *= f.v_global;
        const long long gr = row0 + grow;
        const bool store = valid && ok && FMHA_IN_BOUNDS(gr >= 0 && gr < a.rows_total && split < f.n_splits, kSiteKv4Out, f.status);
        const long long prow = (long long)split * a.rows_total + gr;
        if (ok) {
#pragma unroll 1
            for (int c = 0; c < C::HDV / 32; ++c) {
                float ov[32];
                if (n_tiles > 0) {
                    tmem_ld32(t_lane + C::O_COL + c * 32, ov);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] = 0.f;
                }
                if (!store) continue;
                const int col = part * C::HDV + c * 32;
                if (f.n_splits == 1) {
                    uint4* dst = reinterpret_cast<uint4*>(f.o + gr * HD + col);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        dst[q] = make_uint4(pack_bf16x2(ov[8 * q] * inv, ov[8 * q + 1] * inv),
                                            pack_bf16x2(ov[8 * q + 2] * inv, ov[8 * q + 3] * inv),
                                            pack_bf16x2(ov[8 * q + 4] * inv, ov[8 * q + 5] * inv),
                                            pack_bf16x2(ov[8 * q + 6] * inv, ov[8 * q + 7] * inv));
                } else {
                    float4* dst = reinterpret_cast<float4*>(f.o_part + prow * HD + col);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q] = make_float4(ov[4 * q] * inv, ov[4 * q + 1] * inv, ov[4 * q + 2] * inv, ov[4 * q + 3] * inv);
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
    const double sl2 = (double)f.scale * f.k_global * 1.4426950408889634;
    a.sl2_sign = sl2 > 0 ? 1.f : sl2 < 0 ? -1.f : 0.f;
    a.sl2 = sl2 != 0 ? (float)(sl2 < 0 ? -sl2 : sl2) : 1.f;
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
