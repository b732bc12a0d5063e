// kv4_kernel.cu -- attention over a KV cache held in 4 bits, for few query rows
// per KV head.
//
// A cached row is hd E2M1 codes with one E4M3 scale s per 16 columns (see
// nvfp4.cuh); its value is g * s * e.  The products s * e have at most six
// significant bits between 2^-10 and 2688, so they are exact in fp16: the
// kernel multiplies codes by scales in fp16, feeds fp16 tensor-core products
// with fp32 accumulation, and applies K's g to the scores and V's g to O.  Q is
// scaled by a power of two per row so that its largest element lies in
// [2^14, 2^15) and rounded to fp16: every element within 2^-29 of the
// largest keeps all of bf16's bits.  P is rounded to fp16 (11 bits, against a
// bf16 output's 8).
//
// One thread block takes RT = 8 NB query rows that share a KV head and one chunk
// of that sequence's keys; each of its W warps takes every W-th tile of KT
// keys through a ring of its own (four bulk copies per tile: K and V codes and
// scales, each contiguous over keys), so no warp waits for another before the
// end.  Per 16 keys a warp computes S^T = K Q^T and O^T += V^T P^T with
// mma.sync m16n8k16, keys respectively head-dim columns as the M dimension, so
// that 8 query rows fill N.
//
// Both contractions may be summed in any order, and the order is chosen so that
// the codes never have to be shuffled between lanes.  S^T: lane (g, t) = (lane
// / 4, lane % 4) of a row-g fragment takes columns 32 t .. 32 t + 31 of each 128
// columns (16 bytes of codes, two scales), and Q's fragments are laid out to
// match.  O^T: lane (g, t) takes the four keys of its P fragment and the
// 16-column block g, whose codes of two keys are interleaved into (key, key')
// pairs by two shifts and two selects per 8 codes.
//
// What bounds it: HBM, as long as the conversion keeps up.  Per 32 codes a
// lane spends 16 conversions and 16 multiplications (64 lanes per clock and SM
// each) where HBM delivers 24 bytes per clock and SM, 42 codes.  Measured on GB300
// (hd 128, 8 rows per KV head): 19 sequences of 32768 keys 120 us, 5.97 TB/s, 88 % of
// the measured copy rate (152 blocks of 16 warps); 32 of them 216 us, 5.6 TB/s;
// ragged lengths up to that 115 to 127 us (eight sets of lengths); one sequence of 8191 keys 9.3 us with its
// merge, of which set-up, first copies and the merge are the larger part.  A tile
// without masked keys has code of its own (159 -> 140 us for the ragged batch), the four
// copies of a tile come from four lanes, and each warp parks its O in fragment
// order for the block's sum (both 138 -> 131 us).  Merging the chunks in clusters
// through distributed shared memory instead of by the merge kernel, with the same
// blocks, was no faster: 11.5 against 11.6 us for one sequence, 289 against 238 us for 32.
//
// The softmax runs in the log2 domain with a running reference per row that
// only moves when a score exceeds it by more than 8; then O is rescaled.  P
// carries a factor of 2^6, so that it lies below 2^14 and keeps fp16's 11 bits
// down to 2^-20 of the reference.
#include <climits>
#include <atomic>
#include <type_traits>
#include "internal.h"
#include "kv4_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

template <int HD, int NB, int W>
struct K4Cfg {
    static constexpr int WARPS = W;
    static constexpr int RT = 8 * NB;                  // query rows per block
    static constexpr int KT = HD >= 256 ? 16 : 32;     // keys per tile
    static constexpr int GR = KT / 16;                 // 16-key groups per tile
    static constexpr int CB = HD / 2;                  // code bytes per key
    static constexpr int SB = HD / 16;                 // scale bytes per key
    static constexpr int OFF_KS = KT * CB;             // stage: K codes, K scales, V codes, V scales
    static constexpr int OFF_VC = OFF_KS + KT * SB;
    static constexpr int OFF_VS = OFF_VC + KT * CB;
    static constexpr int STAGE = OFF_VS + KT * SB;
    static constexpr int STAGES = W > 4 || HD == 512 ? 2 : HD == 256 ? 4 : 3;
    static constexpr int RING = STAGES * STAGE;        // per warp
    static constexpr int NCH = HD >= 128 ? HD / 128 : 1;  // 128-column chunks
    static constexpr int TW = HD >= 128 ? 32 : 16;     // columns of a chunk per lane in S^T
    static constexpr int QSTEPS = HD / 16;             // MMA steps of S^T
    static constexpr int ODB = HD / 16;                // MMAs of O^T
    static constexpr bool QREG = HD * NB <= 256;       // Q fragments in registers, else in shared memory
    static constexpr int Q_BYTES = QREG ? 0 : QSTEPS * NB * 256;
    static constexpr int COMB = W * RT * HD * 4;  // epilogue: fp32 O of each warp
    static constexpr int BODY = W * RING > COMB ? W * RING : COMB;
    static constexpr int OFF_Q = BODY;
    static constexpr int OFF_BAR = OFF_Q + Q_BYTES;
    static constexpr int OFF_ML = OFF_BAR + W * STAGES * 8;   // [W][RT] (reference, sum)
    static constexpr int OFF_FLAG = OFF_ML + W * RT * 8;
    static constexpr int SMEM = OFF_FLAG + 16;
    static_assert(STAGE % 16 == 0 && OFF_KS % 16 == 0 && OFF_VC % 16 == 0, "bulk copies are 16-byte aligned");
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct K4Args {
    Kv4Fwd f;
    int group, R;
    ScoreScale sl2;
    long long rows_total;
};

// Key that row m of a 16-key MMA group stands for.  Rows 2t and 2t + 1 (the
// two keys of lane t's P fragment) fall into different 128-byte halves.
__device__ __forceinline__ int key_of_row(int m) { return m ^ ((m >> 1) & 1); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}

// S^T operand: `W` words of codes of one row (8 codes each, a scale per two
// words) as scaled fp16 pairs.
template <int W>
__device__ __forceinline__ void scaled_row(const uint32_t (&w)[W], uint32_t scales, uint32_t (&r)[W][4]) {
    const uint32_t s = e4m3x2_to_f16(scales);
    const uint32_t s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        e2m1x8_to_f16(w[i], r[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = mul_f16x2(r[i][j], i < 2 ? s0 : s1);
    }
}

// O^T operand: 8 codes each of keys x and y -> for column pairs j = 0 .. 3 the
// fp16 pairs (x, y) of columns 2j (lo) and 2j + 1 (hi), times the keys' scales.
__device__ __forceinline__ void key_pairs(uint32_t x, uint32_t y, uint32_t s, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
    e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), lo);
    e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = mul_f16x2(lo[j], s);
        hi[j] = mul_f16x2(hi[j], s);
    }
}

template <int HD, int NB, int W>
__global__ void __launch_bounds__(W * 32, (HD * NB <= 128 && W == 4) ? 4 : 1) kv4_fwd_kernel(const K4Args a) {
    using C = K4Cfg<HD, NB, W>;
    constexpr int kWarps = W;
    constexpr int KT = C::KT, GR = C::GR;
    const Kv4Fwd& f = a.f;
    launch_dependents();  // the merge grid may be scheduled now; it waits for this grid's results
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_FLAG);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int split = blockIdx.y, slab = blockIdx.z;
    const int b = slab / f.n_kv_h, kvh = slab - b * f.n_kv_h;
    const int r_begin = blockIdx.x * C::RT;
    const int r_end = min(a.R, r_begin + C::RT);
    const long long row0 = ((long long)b * f.n_h + (long long)kvh * a.group) * f.T;  // slab's first query row
    auto row_t = [&](int r) { return f.T == 1 ? 0 : r % f.T; };
    if (threadIdx.x < 32) {
        for (int i = threadIdx.x; i < kWarps * C::STAGES; i += 32) mbar_init(&bars[i], 1);
        if (threadIdx.x == 0) *abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();         // barriers initialised
    grid_dependency_wait();  // every global access below follows the preceding kernel

    // Q's loads are issued before the sequence's length is known (NB = 1: all of them).
    auto q_row = [&](int nb) {
        const int r = r_begin + nb * 8 + g;
        const long long row = row0 + (r < r_end ? r : r_begin);
        return reinterpret_cast<const uint2*>(
            f.q + (FMHA_IN_BOUNDS(row >= 0 && row < a.rows_total, kSiteKv4Q, f.status) ? row * HD : 0));
    };
    uint2 early[C::QSTEPS];
    {
        const uint2* src = q_row(0);
#pragma unroll
        for (int i = 0; i < C::QSTEPS; ++i)
            early[i] = __ldg(src + (128 * (i / (C::TW / 4)) + C::TW * t4 + 4 * (i % (C::TW / 4))) / 4);
    }
    auto load_q = [&](int nb, uint2 (&raw)[C::QSTEPS]) {
        const bool live = r_begin + nb * 8 + g < r_end;
        const uint2* src = q_row(nb);
#pragma unroll
        for (int i = 0; i < C::QSTEPS; ++i) {
            raw[i] = nb == 0 ? early[i]
                             : __ldg(src + (128 * (i / (C::TW / 4)) + C::TW * t4 + 4 * (i % (C::TW / 4))) / 4);
            if (!live) raw[i] = make_uint2(0u, 0u);
        }
    };

    // Keys.  Row t sits at position len - T + t.  The chunks divide a virtual
    // key axis: the first keys (rounded up to whole tiles), then the keys from
    // the first one that row 0's window holds (rounded down to 16, the copies' unit).
    const int len = f.seq_lens ? seq_len(f, b) : f.s_k;
    const int n_first = f.window > 0 ? min(f.n_first, len) : 0;
    const int head_span = (n_first + KT - 1) / KT * KT;
    int body = 0;
    if (f.window > 0) body = max(n_first, max(0, len - f.T - f.window + 1));
    const int body16 = body & ~15;
    const long long v_lo = (long long)split * f.kv_chunk, v_hi = v_lo + f.kv_chunk;
    const int h_lo = (int)min(v_lo, (long long)head_span), h_hi = (int)min(v_hi, (long long)head_span);
    const int n_head = (h_hi - h_lo + KT - 1) / KT;
    // this chunk's body keys
    const int b_lo = (int)min((long long)len, body16 + max(0LL, v_lo - head_span));
    int b_hi = (int)min((long long)len, body16 + max(0LL, v_hi - head_span));
    int u_lo = b_lo;
    {
        // ... that some row of this block attends
        int t0 = 0, t1 = f.T - 1;
        if (r_end - r_begin < f.T && (r_end - 1) % f.T >= r_begin % f.T) {
            t0 = r_begin % f.T;
            t1 = (r_end - 1) % f.T;
        }
        if (f.causal) b_hi = min(b_hi, len - f.T + t1 + 1);
        u_lo = max(b_lo, body);
        if (f.window > 0) u_lo = max(u_lo, len - f.T + t0 - f.window + 1);
    }
    const int k16 = u_lo & ~15;  // >= body16: chunks are multiples of 16 keys
    const int n_body = b_hi > u_lo ? (b_hi - k16 + KT - 1) / KT : 0;
    const int n_tiles = n_head + n_body;
    if (n_tiles == 0) {  // nothing to attend in this chunk
        write_empty_rows(f, a.rows_total, row0 + r_begin, r_end - r_begin, split, 0, HD, true,
                         f.sink && f.n_splits == 1 ? kvh * a.group : -1, r_begin);
        return;
    }
    const int body_end16 = (b_hi + 15) & ~15, head_end16 = (n_first + 15) & ~15;

    const uint32_t ring = smem_u32(smem) + warp * C::RING;
    uint64_t* full = bars + warp * C::STAGES;
    const uint64_t pol = l2_policy_evict_first();
    const int my_tiles = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;

    // Tile i of this warp: first key, keys [key, end) that may be attended.
    auto tile_of = [&](int i, int& key, int& end) {
        const int j = warp + i * kWarps;
        if (j < n_head) {
            key = h_lo + j * KT;
            end = n_first;
        } else {
            key = k16 + (j - n_head) * KT;
            end = b_hi;
        }
    };
    // Lanes 0 .. 3 copy a tile's K codes, K scales, V codes and V scales, one each.
    const bool copier = lane < 4;
    const uint8_t* my_src = lane == 0 ? f.k_codes : lane == 1 ? f.k_scales : lane == 2 ? f.v_codes : f.v_scales;
    const int my_row = (lane & 1) ? C::SB : C::CB;
    my_src += (long long)slab * f.cap * my_row;
    const uint32_t my_dst = ring + (lane == 0 ? 0 : lane == 1 ? C::OFF_KS : lane == 2 ? C::OFF_VC : C::OFF_VS);
    auto issue = [&](int i, int s) {  // the copying lanes; tile i into stage s = i % STAGES, which is free
        int key, end;
        tile_of(i, key, end);
        const int n = min(KT, ((warp + i * kWarps) < n_head ? head_end16 : body_end16) - key);
        if (!FMHA_IN_BOUNDS(key >= 0 && key % 16 == 0 && n > 0 && n % 16 == 0 && key + n <= f.cap, kSiteKv4Copy, f.status))
            return false;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], n * 2 * (C::CB + C::SB));
        bulk_load_hint(my_dst + s * C::STAGE, my_src + (unsigned long long)(unsigned)key * my_row, n * my_row, &full[s], pol);
        return true;
    };
    int issued = 0;  // copying lanes: tiles issued
    if (copier) {
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i)
            if (issued == i && i < my_tiles && issue(i, i)) ++issued;
    }

    // Q fragments: for step s of chunk c, row n = g: columns 128 c + TW t + 4 s ..+3.
    uint2 qf[C::QREG ? C::QSTEPS : 1][NB];
    float qs[NB][2];  // per row: score factor (log2 units)
    {
        float fac_g[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            uint2 raw[C::QSTEPS];
            load_q(nb, raw);
            uint32_t mx = 0;  // largest magnitude, as bf16 bits
#pragma unroll
            for (int i = 0; i < C::QSTEPS; ++i)
                mx = __vmaxu2(mx, __vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu));
            mx = max(mx & 0xFFFFu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // 2^k takes the largest magnitude into [2^14, 2^15); rows of zeros,
            // subnormals, infinities or NaN stay as they are
            const int e = (int)(mx >> 7);
            const int k = (e > 0 && e < 255) ? min(max(14 - (e - 127), -120), 120) : 0;
            // the sign of the scale goes into Q, so that a larger product is a larger score
            const float up = __uint_as_float((uint32_t)(127 + k) << 23) * a.sl2.sign;
            fac_g[nb] = score_factor(a.sl2.mant, a.sl2.expo - k);
#pragma unroll
            for (int i = 0; i < C::QSTEPS; ++i) {
                const uint2 v = make_uint2(pack_f16x2(bf16_lo(raw[i].x) * up, bf16_hi(raw[i].x) * up),
                                           pack_f16x2(bf16_lo(raw[i].y) * up, bf16_hi(raw[i].y) * up));
                if constexpr (C::QREG) {
                    qf[i][nb] = v;
                } else {
                    if (warp == 0 && FMHA_IN_BOUNDS((i * NB + nb) * 256 + lane * 8 + 8 <= C::Q_BYTES, kSiteKv4Q, f.status))
                        *reinterpret_cast<uint2*>(smem + C::OFF_Q + (i * NB + nb) * 256 + lane * 8) = v;
                }
            }
        }
        // the factor of row 2 t + i, from a lane whose g is that row
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) qs[nb][i] = __shfl_sync(0xffffffffu, fac_g[nb], (2 * t4 + i) * 4);
        if constexpr (!C::QREG) __syncthreads();
    }

    // Attended keys of the accumulator rows (query rows nb * 8 + 2 t + i):
    // [jlo, jhi] in the body, [0, fhi] among the first keys.
    int jlo[NB][2], jhi[NB][2];
    int full_lo = 0, full_hi = INT_MAX;  // keys that every row attends
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r_begin + nb * 8 + 2 * t4 + i;
            int lo = INT_MAX, hi = -1;
            if (r < r_end) {
                const int p = len - f.T + row_t(r);
                lo = u_lo;
                hi = b_hi - 1;
                if (f.causal) hi = min(hi, p);
                if (f.window > 0) lo = max(lo, p - f.window + 1);
                full_lo = max(full_lo, lo);
                full_hi = min(full_hi, hi);
            }
            jlo[nb][i] = lo;
            jhi[nb][i] = hi;
        }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, m));
        full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, m));
    }

    float m_ref[NB][2], l[NB][2], o[C::ODB][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        m_ref[nb][0] = m_ref[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
        for (int d = 0; d < C::ODB; ++d) o[d][nb][0] = o[d][nb][1] = o[d][nb][2] = o[d][nb][3] = 0.f;
    }

    const int row_a = key_of_row(g), row_b = row_a + 8;            // S^T rows of this lane
    const int key_x = key_of_row(2 * t4), key_y = key_of_row(2 * t4 + 1);  // P's keys (and + 8)
    // A shared-memory address inside [lo, hi), of `bytes` bytes (checked build: lo if it is not).
    auto inside = [&](uint32_t addr, uint32_t bytes, uint32_t lo, uint32_t hi) {
        return FMHA_IN_BOUNDS(addr >= lo && addr + bytes <= hi, kSiteKv4Key, f.status) ? addr : lo;
    };
    // One tile.  EDGE: some key of it is masked for some row, or holds no data.
    auto tile_step = [&](auto edge, uint32_t st, int key0, int end, bool head) {
        constexpr bool EDGE = decltype(edge)::value;
        st = inside(st, C::STAGE, ring, ring + C::RING);
        float sc[GR][NB][4];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) sc[gr][nb][0] = sc[gr][nb][1] = sc[gr][nb][2] = sc[gr][nb][3] = 0.f;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c) {
                constexpr int WD = C::TW / 8;
                uint32_t wa[WD], wb[WD], ra[WD][4], rb[WD][4];
                const uint32_t pa = inside(st + (gr * 16 + row_a) * C::CB + c * 64 + t4 * (C::TW / 2), 8 * C::CB + C::TW / 2,
                                           st, st + C::OFF_KS);
                const uint32_t pb = pa + 8 * C::CB;
                const uint32_t qa = inside(st + C::OFF_KS + (gr * 16 + row_a) * C::SB + c * 8 + t4 * (C::TW / 16),
                                           8 * C::SB + C::TW / 16, st + C::OFF_KS, st + C::OFF_VC);
                uint32_t sa, sb;
                if constexpr (C::TW == 32) {
                    const uint4 u = lds128(pa), v = lds128(pb);
                    wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
                    wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
                    sa = lds16(qa);
                    sb = lds16(qa + 8 * C::SB);
                } else {
                    const uint2 u = lds64(pa), v = lds64(pb);
                    wa[0] = u.x; wa[1] = u.y;
                    wb[0] = v.x; wb[1] = v.y;
                    sa = lds8(qa);
                    sb = lds8(qa + 8 * C::SB);
                }
                scaled_row<WD>(wa, sa, ra);
                scaled_row<WD>(wb, sb, rb);
#pragma unroll
                for (int w = 0; w < WD; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int step = c * (C::TW / 4) + 2 * w + h;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            uint2 q;
                            if constexpr (C::QREG) q = qf[step][nb];
                            else q = lds64(inside(smem_u32(smem) + C::OFF_Q + (step * NB + nb) * 256 + lane * 8, 8,
                                                  smem_u32(smem) + C::OFF_Q, smem_u32(smem) + C::OFF_Q + C::Q_BYTES));
                            mma_f16_16816(sc[gr][nb], ra[w][2 * h], rb[w][2 * h], ra[w][2 * h + 1], rb[w][2 * h + 1], q.x,
                                          q.y);
                        }
                    }
            }
        }

        // mask, running reference
        if constexpr (EDGE) {
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + gr * 16 + (e < 2 ? row_a : row_b);
                        bool in = key >= jlo[nb][e & 1] && key <= jhi[nb][e & 1];
                        if (head) {
                            const int r = r_begin + nb * 8 + 2 * t4 + (e & 1);
                            in = r < r_end && key < n_first && (!f.causal || key <= len - f.T + row_t(r));
                        }
                        sc[gr][nb][e] = in ? sc[gr][nb][e] : -INFINITY;
                    }
        }
        float mx[NB][2];
        bool grow = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float m = -INFINITY;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) m = fmaxf(m, fmaxf(sc[gr][nb][q], sc[gr][nb][2 + q]));
                mx[nb][q] = m * qs[nb][q];
                grow |= mx[nb][q] > m_ref[nb][q] + 8.f;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float m = mx[nb][q];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    if (m > m_ref[nb][q] + 8.f) {
                        const float alpha = ex2_approx(m_ref[nb][q] - m);  // 0 when the reference was -inf
                        m_ref[nb][q] = m;
                        l[nb][q] *= alpha;
#pragma unroll
                        for (int d = 0; d < C::ODB; ++d) {
                            o[d][nb][q] *= alpha;
                            o[d][nb][2 + q] *= alpha;
                        }
                    }
                }
        }
        uint32_t pb[GR][NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float mu0 = kPBias - (m_ref[nb][0] == -INFINITY ? 0.f : m_ref[nb][0]);
            const float mu1 = kPBias - (m_ref[nb][1] == -INFINITY ? 0.f : m_ref[nb][1]);
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const float p0 = ex2_approx(fmaf(sc[gr][nb][0], qs[nb][0], mu0));
                const float p1 = ex2_approx(fmaf(sc[gr][nb][1], qs[nb][1], mu1));
                const float p2 = ex2_approx(fmaf(sc[gr][nb][2], qs[nb][0], mu0));
                const float p3 = ex2_approx(fmaf(sc[gr][nb][3], qs[nb][1], mu1));
                l[nb][0] += p0 + p2;
                l[nb][1] += p1 + p3;
                pb[gr][nb][0] = movmatrix_t(pack_f16x2(p0, p1));
                pb[gr][nb][1] = movmatrix_t(pack_f16x2(p2, p3));
            }
        }

        // O^T += V^T P^T
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
            // Keys outside [from, end) hold stale or no data: their scales count as
            // zero, so that P = 0 meets 0 and never a NaN.
            bool in_x = true, in_y = true, in_x8 = true, in_y8 = true;
            if constexpr (EDGE) {
                const int kx = key0 + gr * 16 + key_x, ky = key0 + gr * 16 + key_y;
                const int from = head ? 0 : u_lo;
                in_x = kx >= from && kx < end;
                in_y = ky >= from && ky < end;
                in_x8 = kx + 8 >= from && kx + 8 < end;
                in_y8 = ky + 8 >= from && ky + 8 < end;
            }
#pragma unroll
            for (int c = 0; c < C::NCH; ++c) {
                const int last = max(key_x, key_y) + 8;
                const uint32_t sv = inside(st + C::OFF_VS + gr * 16 * C::SB + c * 8 + (HD >= 128 ? g : g >> 1), last * C::SB + 1,
                                           st + C::OFF_VS, st + C::STAGE);
                uint32_t s0 = lds8(sv + key_x * C::SB), s1 = lds8(sv + key_y * C::SB);
                uint32_t s2 = lds8(sv + (key_x + 8) * C::SB), s3 = lds8(sv + (key_y + 8) * C::SB);
                if constexpr (EDGE) {
                    s0 = in_x ? s0 : 0u;
                    s1 = in_y ? s1 : 0u;
                    s2 = in_x8 ? s2 : 0u;
                    s3 = in_y8 ? s3 : 0u;
                }
                const uint32_t sp = e4m3x2_to_f16(s0 | (s1 << 8)), sq = e4m3x2_to_f16(s2 | (s3 << 8));
                constexpr int WV = HD >= 128 ? 2 : 1;
                const uint32_t cv = inside(st + C::OFF_VC + gr * 16 * C::CB + c * 64 + g * (4 * WV), last * C::CB + 4 * WV,
                                           st + C::OFF_VC, st + C::OFF_VS);
                uint32_t x[WV], y[WV], x8[WV], y8[WV];
                if constexpr (WV == 2) {
                    const uint2 u0 = lds64(cv + key_x * C::CB), u1 = lds64(cv + key_y * C::CB);
                    const uint2 u2 = lds64(cv + (key_x + 8) * C::CB), u3 = lds64(cv + (key_y + 8) * C::CB);
                    x[0] = u0.x; x[1] = u0.y;
                    y[0] = u1.x; y[1] = u1.y;
                    x8[0] = u2.x; x8[1] = u2.y;
                    y8[0] = u3.x; y8[1] = u3.y;
                } else {
                    x[0] = lds32(cv + key_x * C::CB);
                    y[0] = lds32(cv + key_y * C::CB);
                    x8[0] = lds32(cv + (key_x + 8) * C::CB);
                    y8[0] = lds32(cv + (key_y + 8) * C::CB);
                }
#pragma unroll
                for (int w = 0; w < WV; ++w) {
                    uint32_t lo[4], hi[4], lo8[4], hi8[4];
                    key_pairs(x[w], y[w], sp, lo, hi);
                    key_pairs(x8[w], y8[w], sq, lo8, hi8);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_f16_16816(o[(c * WV + w) * 4 + j][nb], lo[j], hi[j], lo8[j], hi8[j], pb[gr][nb][0],
                                          pb[gr][nb][1]);
                }
            }
        }
    };
    bool ok = true;
    int s = 0;
    unsigned phase = 0;
    for (int i = 0; i < my_tiles; ++i) {
        if (!mbar_wait(&full[s], phase, f.status)) {
            ok = false;
            break;
        }
        int key0, end;
        tile_of(i, key0, end);
        const bool head = warp + i * kWarps < n_head;
        if (!head && key0 >= full_lo && key0 + KT - 1 <= full_hi)
            tile_step(std::false_type{}, ring + s * C::STAGE, key0, end, false);
        else
            tile_step(std::true_type{}, ring + s * C::STAGE, key0, end, head);
        __syncwarp();  // every lane is done with the stage
        if (copier && issued == i + C::STAGES && issued < my_tiles && issue(issued, s)) ++issued;
        if (++s == C::STAGES) {
            s = 0;
            phase ^= 1;
        }
    }

    // ------------------------------------------------------------ epilogue
    // Every copy that was waited for has landed; after a wait that gave up the
    // others are waited for here.
    if (!ok) {
        if (lane == 0) {
            drain_ring(full, C::STAGES, issued, f.status);
            atomicOr(abort_flag, 1);
        }
        __syncwarp();
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 4);
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 8);
            l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], 16);
        }
    if (g == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = warp * C::RT + nb * 8 + 2 * t4 + i;
                if (FMHA_IN_BOUNDS(at < W * C::RT, kSiteKv4Comb, f.status)) ml[at] = make_float2(m_ref[nb][i], l[nb][i]);
            }
    }
    __syncthreads();  // every warp is done with its ring
    if (*abort_flag) return;

    // Each warp parks its O as it lies in the fragments: [warp][MMA d][nb][i][lane],
    // the column pair of row nb * 8 + 2 t + i, so that neither the stores nor the
    // loads below meet a bank twice.
    constexpr int WV = HD >= 128 ? 2 : 1;
    float2* comb = reinterpret_cast<float2*>(smem);
    constexpr int SLICE = C::ODB * NB * 2 * 32;  // one warp's share
#pragma unroll
    for (int d = 0; d < C::ODB; ++d)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = warp * SLICE + ((d * NB + nb) * 2 + i) * 32 + lane;
                if (FMHA_IN_BOUNDS(at < W * SLICE, kSiteKv4Comb, f.status)) comb[at] = make_float2(o[d][nb][i], o[d][nb][2 + i]);
            }
    __syncthreads();
    // A job is 8 neighbouring columns (four MMAs) of the 32 lanes' rows: sum the warps,
    // weighted by their references, divide, write out.
    constexpr int JOBS = C::NCH * WV * NB * 2;
    for (int job = warp; job < JOBS; job += kWarps) {
        const int i = job & 1, nb = (job >> 1) % NB, cw = job / (2 * NB);  // cw: 8-column half of a block (with its chunk)
        const int r = nb * 8 + 2 * t4 + i;
        if (r_begin + r >= r_end) continue;
        if (!FMHA_IN_BOUNDS(r < C::RT && (((cw * 4 + 3) * NB + nb) * 2 + i) * 32 + lane < SLICE, kSiteKv4Comb, f.status)) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * C::RT + r].x);
        const float Mu = (M == -INFINITY) ? 0.f : M;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 v = ml[w * C::RT + r];
            const float fac = exp2f(v.x - Mu);  // 0 for a warp without keys
            L += v.y * fac;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = comb[w * SLICE + (((cw * 4 + j) * NB + nb) * 2 + i) * 32 + lane];
                acc[2 * j] += u.x * fac;
                acc[2 * j + 1] += u.y * fac;
            }
        }
        float inv, lse;
        finish_row_nan(M - kPBias, L,
                   f.sink && f.n_splits == 1 ? sink_log2_of(f.sink, kvh * a.group + (r_begin + r) / f.T, f.n_h, f.status)
                                             : -INFINITY,
                   inv, lse);
        inv *= f.v_global;
        const int col = 128 * (cw / WV) + g * (8 * WV) + 8 * (cw % WV);
        const long long grow = row0 + r_begin + r;
        if (!FMHA_IN_BOUNDS(grow >= 0 && grow < a.rows_total && split < f.n_splits && col + 8 <= HD, kSiteKv4Out, f.status)) continue;
        if (f.n_splits == 1) {
            uint4 pk;
            pk.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
            pk.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
            pk.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
            pk.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
            *reinterpret_cast<uint4*>(f.o + grow * HD + col) = pk;
            if (col == 0) f.lse[grow] = lse;
        } else {
            const long long prow = (long long)split * a.rows_total + grow;
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(f.o_part) + prow * HD + col);
            dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
            if (col == 0) f.lse_part[prow] = lse;
        }
    }
}

template <int HD, int NB, int W>
cudaError_t launch_t(const Kv4Fwd& f, cudaStream_t stream) {
    using C = K4Cfg<HD, NB, W>;
    auto kern = kv4_fwd_kernel<HD, NB, W>;
    static std::atomic<bool> attr_set[128];  // set once per device; any host thread may set it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 128) attr_set[dev] = true;
    }
    K4Args a;
    a.f = f;
    a.group = f.n_h / f.n_kv_h;
    a.R = a.group * f.T;
    a.sl2 = score_scale(f);
    a.rows_total = (long long)f.batch * f.n_h * f.T;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.R + C::RT - 1) / C::RT, f.n_splits, f.batch * f.n_kv_h);
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

constexpr int big_warps(int hd, int rows) { return hd * rows <= 1024 ? 16 : 8; }

template <int HD, int NB>
cudaError_t launch_w(const Kv4Fwd& f, cudaStream_t stream) {
    return f.warps > 4 ? launch_t<HD, NB, big_warps(HD, 8 * NB)>(f, stream) : launch_t<HD, NB, 4>(f, stream);
}

template <int HD>
cudaError_t launch_hd(const Kv4Fwd& f, cudaStream_t stream) {
    const int rows = kv4_rows_per_cta(HD, (long long)f.n_h / f.n_kv_h * f.T);
    if constexpr (HD == 64)
        if (rows == 32) return launch_w<HD, 4>(f, stream);
    if constexpr (HD <= 256)
        if (rows == 16) return launch_w<HD, 2>(f, stream);
    return launch_w<HD, 1>(f, stream);
}

}  // namespace

int kv4_kv_tile(int hd) { return hd >= 256 ? 16 : 32; }

int kv4_rows_per_cta(int hd, long long rows) {
    if (rows > 16 && hd == 64) return 32;  // at hd 128 its accumulators do not fit the registers
    return rows > 8 && hd <= 256 ? 16 : 8;
}

int kv4_big_warps(int hd, int rows_per_cta) { return big_warps(hd, rows_per_cta); }

int kv4_ctas_per_sm(int hd, int rows_per_cta, int warps) {
    if (warps > 4) return 1;
    return hd * rows_per_cta <= 128 * 8 ? 4 : 2;  // by registers and shared memory
}

cudaError_t launch_kv4_fwd(const Kv4Fwd& f, cudaStream_t stream) {
    switch (f.hd) {
        case 64: return launch_hd<64>(f, stream);
        case 128: return launch_hd<128>(f, stream);
        case 256: return launch_hd<256>(f, stream);
        case 512: return launch_hd<512>(f, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fmha
