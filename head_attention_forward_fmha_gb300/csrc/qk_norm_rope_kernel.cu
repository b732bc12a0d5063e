// qk_norm_rope_kernel.cu -- from the rows of a QKV projection to what the
// attention forward takes, in one pass: per-head RMS norm of Q and K, rotation
// by the token's position, V copied, token-major rows to head-major tensors.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                      (Q and K heads with a weight)
//   (y_lo, y_hi) -> (y_lo cos - y_hi sin, y_hi cos + y_lo sin)
// over the first `rot` columns of the head, the pair of rotation i being
// columns (i, rot / 2 + i), or (2i, 2i + 1) when interleaved; the columns from
// `rot` on pass unrotated.  All of it in fp32, rounded to bf16 once at the
// end; V rows are copied bit for bit.
//
// The pass reads and writes every element once (4 bytes of traffic each) and
// does ~10 flops on it: it is bound by HBM when there are many tokens and by
// launch latency when there are few.  A head row is spread over hd / 8 lanes,
// each holding two 4-element vectors that contain whole rotation pairs (the
// lower and the upper half's columns, or 8 neighbouring ones when
// interleaved), so the rotation needs no exchange between lanes and the sum of
// squares is one shuffle tree.  A warp takes up to UNROLL row sets of one kind
// (query, key or value heads) of one token, with all their loads issued before
// any arithmetic.  Norm weight and rotation are one linear map of a pair of
// columns, out = x A + x' B with A, B made of the weights, cosines and sines;
// a warp forms A and B once and applies them to all its heads, two columns per
// instruction (packed fp32 pairs).
//
// Measured on GB300: four prompts of 4095 tokens, 64 + 2 x 8 heads of 128 (679 MB)
// 109 us, 6.2 TB/s, 92 % of the measured copy rate, 60 % of the issue slots; one
// token of the same 1.7 us.  With weight, norm and rotation applied one after
// the other to single elements the prompts took 138 us, with 64-bit task
// arithmetic and plain stores 121.
//
// Four row sets per warp or one: four form A and B once for more heads and keep more loads
// in flight, one spreads few rows over more warps.  They cross between 8192 and 32768 head
// rows (one / four, us, 64 query and 8 KV heads): hd 64 16320 rows
// 2.7 / 3.0, 32720 rows 3.9 / 3.5, 262080 rows 21.8 / 14.3; hd 128 8160 rows 2.7 / 2.7,
// 16320 rows 4.0 / 3.8, 262080 rows 41.4 / 23.5; hd 256 4080 rows 2.7 / 2.8, 16320 rows
// 6.6 / 5.0; hd 512 4080 rows 3.1 / 3.9, 16320 rows 9.9 / 9.0, 262080 rows 128 / 89.  So four
// from 16384 rows on, at every head dim.
#include "internal.h"
#include "ptx.cuh"

namespace fmha {
namespace {

constexpr int kNrWarps = 4;

template <int HD>
struct NrCfg {
    static constexpr int LANES = HD >= 256 ? 32 : HD / 8;  // lanes per head row
    static constexpr int RPW = 32 / LANES;                 // rows per warp and row set
    static constexpr int UNITS = HD / 8 / LANES;           // pairs of 4-element vectors per lane
};

template <int HD, int UNROLL>
__global__ void __launch_bounds__(kNrWarps * 32) qk_norm_rope_kernel(const QkNormRope a, int q_sets, int kv_sets) {
    using C = NrCfg<HD>;
    launch_dependents();
    const int lane = threadIdx.x & 31;
    constexpr int kSet = C::RPW * UNROLL;  // heads per warp
    const int sets = q_sets + 2 * kv_sets;
    const unsigned task = blockIdx.x * kNrWarps + (threadIdx.x >> 5);  // < 2^31 + 4
    const int token = (int)(task / (unsigned)sets);
    if (token >= a.batch * a.T) return;
    int set = (int)(task - (unsigned)token * sets);
    const int type = set < q_sets ? 0 : set < q_sets + kv_sets ? 1 : 2;  // q, k, v: the same for the warp
    if (type == 1) set -= q_sets;
    if (type == 2) set -= q_sets + kv_sets;
    const int heads = type == 0 ? a.n_h : a.n_kv_h;
    const int b = token / a.T, t = token - b * a.T;
    const int sub = lane / C::LANES, u0 = lane - sub * C::LANES;
    const int h0 = set * kSet + sub;  // this lane's heads of the kind: h0, h0 + RPW, ...
    const bool inter = a.interleaved != 0;
    const int half = a.rot >> 1;
    int col[C::UNITS][2];
    bool turned[C::UNITS];
#pragma unroll
    for (int k = 0; k < C::UNITS; ++k) {
        const int u = u0 + k * C::LANES;
        turned[k] = 8 * u < a.rot;
        col[k][0] = turned[k] && !inter ? 4 * u : 8 * u;
        col[k][1] = turned[k] && !inter ? half + 4 * u : 8 * u + 4;
    }
    grid_dependency_wait();  // every global access below follows the preceding kernel
    if (!FMHA_IN_BOUNDS(b >= 0 && b < a.batch && t >= 0 && t < a.T && set >= 0, kSiteNrRow, a.status)) return;

    // Every load is issued before any arithmetic.
    const __nv_bfloat16* src = a.qkv + b * a.batch_stride + t * a.token_stride +
                               (long long)(h0 + (type == 0 ? 0 : a.n_h + (type == 2 ? a.n_kv_h : 0))) * HD;
    uint2 raw[UNROLL][C::UNITS][2];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                raw[i][k][f] = make_uint2(0u, 0u);
                if (h0 + i * C::RPW < heads && FMHA_IN_BOUNDS(col[k][f] >= 0 && col[k][f] + 4 <= HD, kSiteNrCol, a.status))
                    raw[i][k][f] = __ldcs(reinterpret_cast<const uint2*>(src + i * C::RPW * HD + col[k][f]));
            }
    const int pos = a.rot > 0 ? __ldg(a.positions + token) : 0;
    if (a.rot > 0 && (pos < 0 || pos >= a.max_pos)) return;  // a padding token: nothing of it is written
    __nv_bfloat16* dst;
    long long step;  // elements from one head to the next
    if (type == 0) {
        step = (long long)a.T * HD;
        dst = a.q + ((long long)b * a.n_h * a.T + t) * HD;
    } else {
        const long long kv_row = (a.kv_start ? __ldg(a.kv_start + b) : 0) + (long long)t;
        if (kv_row < 0 || kv_row >= a.kv_rows) return;
        step = (long long)a.kv_rows * HD;
        dst = (type == 1 ? a.k : a.v) + ((long long)b * a.n_kv_h * a.kv_rows + kv_row) * HD;
    }
    dst += h0 * step;
    if (!FMHA_IN_BOUNDS(col[0][0] >= 0 && col[C::UNITS - 1][1] + 4 <= HD && col[C::UNITS - 1][0] + 4 <= HD, kSiteNrCol, a.status))
        return;

    if (type != 2) {
        // A and B of this lane's columns, as pairs of neighbouring columns
        const float* w = type == 0 ? a.q_weight : a.k_weight;
        uint64_t ca[C::UNITS][2][2], cb[C::UNITS][2][2];
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k) {
            float w4[2][4], c4[4] = {1.f, 1.f, 1.f, 1.f}, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const float4 v = w ? __ldg(reinterpret_cast<const float4*>(w + col[k][f])) : make_float4(1.f, 1.f, 1.f, 1.f);
                w4[f][0] = v.x; w4[f][1] = v.y; w4[f][2] = v.z; w4[f][3] = v.w;
            }
            if (turned[k] && FMHA_IN_BOUNDS(pos >= 0 && pos < a.max_pos && 4 * (u0 + k * C::LANES) + 4 <= half, kSiteNrTable, a.status)) {
                const float* tab = a.cos_sin + (long long)pos * a.rot + 4 * (u0 + k * C::LANES);
                const float4 c = __ldg(reinterpret_cast<const float4*>(tab));
                const float4 s = __ldg(reinterpret_cast<const float4*>(tab + half));
                c4[0] = c.x; c4[1] = c.y; c4[2] = c.z; c4[3] = c.w;
                s4[0] = s.x; s4[1] = s.y; s4[2] = s.z; s4[3] = s.w;
            }
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * e, j = 2 * e + 1;
                    if (inter) {  // columns i and j of one vector are a pair, number 2 f + e
                        const float c = c4[2 * f + e], s = s4[2 * f + e];
                        ca[k][f][e] = f32x2(w4[f][i] * c, w4[f][j] * c);
                        cb[k][f][e] = f32x2(-w4[f][j] * s, w4[f][i] * s);
                    } else {  // column i of the lower vector pairs with column i of the upper one
                        ca[k][f][e] = f32x2(w4[f][i] * c4[i], w4[f][j] * c4[j]);
                        const float sign = f == 0 ? -1.f : 1.f;
                        cb[k][f][e] = f32x2(sign * w4[1 - f][i] * s4[i], sign * w4[1 - f][j] * s4[j]);
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            uint64_t x[C::UNITS][2][2], ss2 = 0ull;
#pragma unroll
            for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    x[k][f][0] = bf16x2_to_f32x2(raw[i][k][f].x);
                    x[k][f][1] = bf16x2_to_f32x2(raw[i][k][f].y);
                    ss2 = fma_f32x2(x[k][f][0], x[k][f][0], ss2);
                    ss2 = fma_f32x2(x[k][f][1], x[k][f][1], ss2);
                }
            float inv = 1.f;
            if (w) {
                float s0, s1;
                f32x2_split(ss2, s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int m = C::LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                inv = rsqrtf(ss * (1.f / HD) + a.eps);
            }
            const uint64_t inv2 = f32x2(inv, inv);
#pragma unroll
            for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    uint32_t out[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t y = mul_f32x2(x[k][f][e], inv2);
                        uint64_t r = mul_f32x2(y, ca[k][f][e]);
                        if (turned[k]) {
                            uint64_t z;
                            if (inter) {
                                float y0, y1;
                                f32x2_split(y, y0, y1);
                                z = f32x2(y1, y0);
                            } else {
                                z = mul_f32x2(x[k][1 - f][e], inv2);
                            }
                            r = fma_f32x2(z, cb[k][f][e], r);
                        }
                        float r0, r1;
                        f32x2_split(r, r0, r1);
                        out[e] = pack_bf16x2(r0, r1);
                    }
                    raw[i][k][f] = make_uint2(out[0], out[1]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        if (h0 + i * C::RPW >= heads) break;
        const long long at = dst + i * C::RPW * step - (type == 0 ? a.q : type == 1 ? a.k : a.v);
        if (!FMHA_IN_BOUNDS(at >= 0 && at + HD <= (long long)a.batch * HD * (type == 0 ? (long long)a.n_h * a.T : (long long)a.n_kv_h * a.kv_rows),
                            kSiteNrRow, a.status))
            break;
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f) __stcs(reinterpret_cast<uint2*>(dst + i * C::RPW * step + col[k][f]), raw[i][k][f]);
    }
}

template <int HD, int UNROLL>
cudaError_t launch_u(const QkNormRope& a, cudaStream_t stream) {
    constexpr int kSet = NrCfg<HD>::RPW * UNROLL;
    const int q_sets = (a.n_h + kSet - 1) / kSet, kv_sets = (a.n_kv_h + kSet - 1) / kSet;
    const long long tasks = (long long)a.batch * a.T * (q_sets + 2 * kv_sets);
    const long long blocks = (tasks + kNrWarps - 1) / kNrWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kNrWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<HD, UNROLL>, a, q_sets, kv_sets);
}

template <int HD>
cudaError_t launch_hd(const QkNormRope& a, cudaStream_t stream) {
    const long long rows = (long long)a.batch * a.T * (a.n_h + 2 * a.n_kv_h);
    return rows >= 16384 ? launch_u<HD, 4>(a, stream) : launch_u<HD, 1>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope& a, int hd, cudaStream_t stream) {
    switch (hd) {
        case 64: return launch_hd<64>(a, stream);
        case 128: return launch_hd<128>(a, stream);
        case 256: return launch_hd<256>(a, stream);
        case 512: return launch_hd<512>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fmha
