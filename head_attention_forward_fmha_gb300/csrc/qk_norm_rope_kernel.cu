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
// squares is one shuffle tree.  A warp takes UNROLL row sets of one token at
// a time, with all their loads issued before any arithmetic; the cosines and
// sines of the token stay in registers for all of its heads.
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

// Columns of vector `half` (0 lower, 1 upper) of unit u of a head row.
template <int HD>
__device__ __forceinline__ int nr_column(int u, int half, int rot, bool interleaved) {
    const int c = 8 * u;
    if (interleaved || c >= rot) return c + 4 * half;
    return 4 * u + half * (rot >> 1);
}

__device__ __forceinline__ void nr_unpack(uint2 v, float (&x)[4]) {
    x[0] = bf16_lo(v.x);
    x[1] = bf16_hi(v.x);
    x[2] = bf16_lo(v.y);
    x[3] = bf16_hi(v.y);
}

template <int HD, int UNROLL>
__global__ void __launch_bounds__(kNrWarps * 32) qk_norm_rope_kernel(const QkNormRope a) {
    using C = NrCfg<HD>;
    launch_dependents();
    grid_dependency_wait();  // every global access below follows the preceding kernel
    const int lane = threadIdx.x & 31;
    const int heads = a.n_h + 2 * a.n_kv_h;
    constexpr int kSet = C::RPW * UNROLL;  // heads per warp
    const int sets = (heads + kSet - 1) / kSet;
    const long long task = (long long)blockIdx.x * kNrWarps + (threadIdx.x >> 5);
    const long long token = task / sets;
    if (token >= (long long)a.batch * a.T) return;
    const int set = (int)(task - token * sets);
    const int b = (int)(token / a.T), t = (int)(token - (long long)b * a.T);
    const int sub = lane / C::LANES, u0 = lane - sub * C::LANES;

    // Every load is issued before any arithmetic.
    const __nv_bfloat16* row = a.qkv + b * a.batch_stride + t * a.token_stride;
    uint2 raw[UNROLL][C::UNITS][2];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int h = set * kSet + i * C::RPW + sub;
        if (h >= heads) continue;
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f)
                raw[i][k][f] = __ldcs(reinterpret_cast<const uint2*>(
                    row + (long long)h * HD + nr_column<HD>(u0 + k * C::LANES, f, a.rot, a.interleaved)));
    }
    const int pos = a.rot > 0 ? __ldg(a.positions + token) : 0;
    if (a.rot > 0 && (pos < 0 || pos >= a.max_pos)) return;  // a padding token: nothing of it is written
    float4 cs[C::UNITS], sn[C::UNITS];
#pragma unroll
    for (int k = 0; k < C::UNITS; ++k) {
        const int u = u0 + k * C::LANES;
        cs[k] = make_float4(1.f, 1.f, 1.f, 1.f);
        sn[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (8 * u < a.rot) {
            const float* tab = a.cos_sin + (long long)pos * a.rot + 4 * u;
            cs[k] = __ldg(reinterpret_cast<const float4*>(tab));
            sn[k] = __ldg(reinterpret_cast<const float4*>(tab + (a.rot >> 1)));
        }
    }
    const long long kv_row = (a.kv_start ? __ldg(a.kv_start + b) : 0) + (long long)t;
    const bool kv_ok = kv_row >= 0 && kv_row < a.kv_rows;

#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int h = set * kSet + i * C::RPW + sub;
        const bool live = h < heads;
        const int type = h < a.n_h ? 0 : h < a.n_h + a.n_kv_h ? 1 : 2;  // q, k, v
        float x[C::UNITS][2][4];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                nr_unpack(live ? raw[i][k][f] : make_uint2(0u, 0u), x[k][f]);
#pragma unroll
                for (int e = 0; e < 4; ++e) ss += x[k][f][e] * x[k][f][e];
            }
#pragma unroll
        for (int m = C::LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (!live) continue;
        __nv_bfloat16* dst;
        if (type == 0) {
            dst = a.q + (((long long)b * a.n_h + h) * a.T + t) * HD;
        } else {
            if (!kv_ok) continue;
            const int kvh = h - a.n_h - (type == 2 ? a.n_kv_h : 0);
            dst = (type == 1 ? a.k : a.v) + (((long long)b * a.n_kv_h + kvh) * a.kv_rows + kv_row) * HD;
        }
        const float* w = type == 0 ? a.q_weight : a.k_weight;
        const float inv = rsqrtf(ss * (1.f / HD) + a.eps);
#pragma unroll
        for (int k = 0; k < C::UNITS; ++k) {
            const int u = u0 + k * C::LANES;
            const int col0 = nr_column<HD>(u, 0, a.rot, a.interleaved), col1 = nr_column<HD>(u, 1, a.rot, a.interleaved);
            uint2 out0 = raw[i][k][0], out1 = raw[i][k][1];
            if (type != 2) {
                float(&lo)[4] = x[k][0];
                float(&hi)[4] = x[k][1];
                if (w) {
                    const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + col0));
                    const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + col1));
                    lo[0] *= inv * w0.x; lo[1] *= inv * w0.y; lo[2] *= inv * w0.z; lo[3] *= inv * w0.w;
                    hi[0] *= inv * w1.x; hi[1] *= inv * w1.y; hi[2] *= inv * w1.z; hi[3] *= inv * w1.w;
                }
                const float c4[4] = {cs[k].x, cs[k].y, cs[k].z, cs[k].w};
                const float s4[4] = {sn[k].x, sn[k].y, sn[k].z, sn[k].w};
                if (8 * u >= a.rot) {
                    // past the rotated columns
                } else if (a.interleaved) {  // pairs (0,1) (2,3) of the lower vector, then of the upper one
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float l0 = lo[2 * e], l1 = lo[2 * e + 1], h0 = hi[2 * e], h1 = hi[2 * e + 1];
                        lo[2 * e] = l0 * c4[e] - l1 * s4[e];
                        lo[2 * e + 1] = l1 * c4[e] + l0 * s4[e];
                        hi[2 * e] = h0 * c4[2 + e] - h1 * s4[2 + e];
                        hi[2 * e + 1] = h1 * c4[2 + e] + h0 * s4[2 + e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float l0 = lo[e], h0 = hi[e];
                        lo[e] = l0 * c4[e] - h0 * s4[e];
                        hi[e] = h0 * c4[e] + l0 * s4[e];
                    }
                }
                out0 = make_uint2(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]));
                out1 = make_uint2(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
            }
            if (!FMHA_IN_BOUNDS(col0 >= 0 && col0 + 4 <= HD && col1 >= 0 && col1 + 4 <= HD, kSiteNrCol, a.status)) continue;
            *reinterpret_cast<uint2*>(dst + col0) = out0;
            *reinterpret_cast<uint2*>(dst + col1) = out1;
        }
    }
}

template <int HD, int UNROLL>
cudaError_t launch_u(const QkNormRope& a, cudaStream_t stream) {
    const int heads = a.n_h + 2 * a.n_kv_h;
    const int sets = (heads + NrCfg<HD>::RPW * UNROLL - 1) / (NrCfg<HD>::RPW * UNROLL);
    const long long tasks = (long long)a.batch * a.T * sets;
    const long long blocks = (tasks + kNrWarps - 1) / kNrWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kNrWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<HD, UNROLL>, a);
}

template <int HD>
cudaError_t launch_hd(const QkNormRope& a, cudaStream_t stream) {
    const long long rows = (long long)a.batch * a.T * (a.n_h + 2 * a.n_kv_h);
    return rows >= 65536 ? launch_u<HD, 4>(a, stream) : launch_u<HD, 1>(a, stream);
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
