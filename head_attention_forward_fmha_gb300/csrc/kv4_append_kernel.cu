// kv4_append_kernel.cu -- new K and V rows into a cache held in 4 bits.
//
// Row t of sequence b goes to cache row start[b] + t: each 16-element block
// becomes 16 E2M1 codes (8 bytes) and one E4M3 scale byte, by the block
// quantiser of nvfp4.cuh on the bf16 values widened to fp32.  Optionally the
// values that the cache now stands for, g * s * e, come back as bf16 rows (s
// e has at most 6 significant bits, so only the product with g can round).
//
// One thread per block, K and V in one launch: 32 bytes in, 9 out (41 with the
// values).  Bound by HBM for long prompts, by launch latency for decode steps.
#include "internal.h"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

__global__ void __launch_bounds__(128) kv4_append_kernel(const Kv4Append a, int blocks_per_row) {
    launch_dependents();
    grid_dependency_wait();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long rows = (long long)a.batch * a.n_kv_h * a.T;
    const long long row = i / blocks_per_row;
    const int blk = (int)(i - row * blocks_per_row);
    if (row >= rows) return;
    const bool is_v = blockIdx.y != 0;
    const long long slab = row / a.T;
    const long long at = __ldg(a.start + slab / a.n_kv_h) + (row - slab * a.T);
    if (at < 0 || at >= a.cap) return;  // outside the cache: left out
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? a.v : a.k) + i * 16);
    const uint4 u0 = __ldcs(src), u1 = __ldcs(src + 1);
    const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[2 * e] = bf16_lo(w[e]);
        x[2 * e + 1] = bf16_hi(w[e]);
    }
    uint32_t pk[2];
    const float g = is_v ? a.v_global : a.k_global;
    const uint32_t sc = nvfp4_block(x, g, pk);
    const long long dst = (slab * a.cap + at) * blocks_per_row + blk;
    if (!FMHA_IN_BOUNDS(dst >= 0 && dst < (long long)a.batch * a.n_kv_h * a.cap * blocks_per_row, kSiteKv4Append, a.status))
        return;
    *reinterpret_cast<uint2*>((is_v ? a.v_codes : a.k_codes) + dst * 8) = make_uint2(pk[0], pk[1]);
    (is_v ? a.v_scales : a.k_scales)[dst] = (uint8_t)sc;
    __nv_bfloat16* out = is_v ? a.v_out : a.k_out;
    if (out) {
        const float s = e4m3_value(sc);
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const uint32_t c = (pk[e >> 2] >> (8 * (e & 3) + 4 * f)) & 15u;
                v[f] = __fmul_rn(__fmul_rn(e2m1_value(c), s), g);
            }
            o[e] = pack_bf16x2(v[0], v[1]);
        }
        uint4* to = reinterpret_cast<uint4*>(out + i * 16);
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Append& a, int hd, cudaStream_t stream) {
    const int per_row = hd / 16;
    const long long blocks = (long long)a.batch * a.n_kv_h * a.T * per_row;
    if ((blocks + 127) / 128 > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((blocks + 127) / 128), 2);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_append_kernel, a, per_row);
}

}  // namespace fmha
