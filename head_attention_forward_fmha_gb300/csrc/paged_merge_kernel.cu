// paged_merge_kernel.cu -- LSE merge of the chunks of the attention over a cache in pages:
//   LSE = ln(sum_i exp(lse_i) + exp(sink)),   O = sum_i exp(lse_i - LSE) O_i.
// One warp per (row of o, slice of up to 128 columns), as in merge_kernel.cu; what differs:
// rows behind the last sequence of a ragged batch are left as they are, of a chunk with
// LSE = -inf (nothing attended, as most chunks of short sequences) O is neither written nor read,
// and a chunk with LSE = NaN makes O and LSE of its row NaN.  Bound by the latency of two rounds of loads: about 3 us
// behind a decode step; partials of many rows (4 x 512 tokens of 64 heads: 67 MB a chunk) by L2, which is why the
// plan splits long chunks of tokens only where there are too few blocks.
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.693147180559945309f;

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) paged_merge_kernel(const PagedFwd f) {
    constexpr int V = HD >= 128 ? 4 : 2, SLICE = 32 * V, NSLICE = HD / SLICE;
    grid_dependency_wait();  // the chunks' partials are complete and visible
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (task >= f.rows * NSLICE) return;
    const long long row = task / NSLICE;
    const int col = (int)(task - row * NSLICE) * SLICE + lane * V;
    if (f.t.cu) {  // rows that are no tokens
        const long long token = row / f.n_h;
        if (token < __ldg(f.t.cu) || token >= __ldg(f.t.cu + f.t.batch)) return;
    }
    const int head = f.t.cu ? (int)(row % f.n_h) : (int)(row / f.t.T % f.n_h);
    const float sink = f.sink && FMHA_IN_BOUNDS(head >= 0 && head < f.n_h, kSitePagedOut, f.status) ? __ldg(f.sink + head) : -INFINITY;
    float mx = sink;
    bool nan = false;
    for (int i = lane; i < f.n_splits; i += 32) {
        const float lse = __ldg(f.lse_part + i * f.rows + row);
        mx = fmaxf(mx, lse);
        nan |= lse != lse;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    float den = 0.f;
    if (mx != -INFINITY) {
        for (int base = 0; base < f.n_splits; base += 32) {
            const int mine = base + lane;
            const float lse = mine < f.n_splits ? __ldg(f.lse_part + mine * f.rows + row) : -INFINITY;
            const float w = exp2f((lse - mx) * kLog2e);
            unsigned live = __ballot_sync(0xffffffffu, lse != -INFINITY);
            float sum = w;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            den += sum;
            while (live) {  // four chunks in flight; the last one again, with weight 0, where there are fewer
                float v[4][V], wi[4];
                int last = 0;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const bool some = live != 0u;
                    if (some) last = __ffs(live) - 1;
                    live &= live - 1u;
                    const float* src = f.o_part + ((long long)(base + last) * f.rows + row) * HD + col;
                    if constexpr (V == 4) {
                        const float4 u = __ldg(reinterpret_cast<const float4*>(src));
                        v[y][0] = u.x; v[y][1] = u.y; v[y][2] = u.z; v[y][3] = u.w;
                    } else {
                        const float2 u = __ldg(reinterpret_cast<const float2*>(src));
                        v[y][0] = u.x; v[y][1] = u.y;
                    }
                    const float at = __shfl_sync(0xffffffffu, w, last);
                    wi[y] = some ? at : 0.f;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] += wi[y] * v[y][e];
            }
        }
        if (sink != -INFINITY) den += exp2f((sink - mx) * kLog2e);
    }
    if (__any_sync(0xffffffffu, nan)) den = NAN;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    if (!FMHA_IN_BOUNDS(row >= 0 && row < f.rows && col + V <= HD, kSitePagedOut, f.status)) return;
    __nv_bfloat16* dst = f.o + row * HD + col;
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && col == 0) f.lse[row] = den == 0.f ? -INFINITY : mx + log2f(den) * kLn2;
}

template <int HD>
cudaError_t launch_t(const PagedFwd& f, cudaStream_t stream) {
    const long long blocks = (f.rows * (HD / (HD >= 128 ? 128 : 64)) + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<HD>, f);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedFwd& f, cudaStream_t stream) {
    switch (f.c.hd) {
        case 64: return launch_t<64>(f, stream);
        case 128: return launch_t<128>(f, stream);
        case 256: return launch_t<256>(f, stream);
        case 512: return launch_t<512>(f, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fmha
