// kv4_append_kernel.cu -- new K and V rows into a cache held in 4 bits.
//
// Row t of sequence b goes to cache row start[b] + t: each 16-element block
// becomes 16 E2M1 codes (8 bytes) and one E4M3 scale byte, by the block
// quantiser of nvfp4.cuh on the bf16 values widened to fp32.  Optionally the
// values that the cache now stands for, g * s * e, come back as bf16 rows (s
// e has at most 6 significant bits, so only the product with g can round).
//
// Two threads per 16-element block (16 bytes in each, coalesced), each for K and V.
// 2 bytes in and 0.5625 out per element (2.5625 with the values): bound by HBM
// for long prompts if the quantiser's arithmetic is cheap, by launch latency
// for decode steps.  So the codes' divisions x / (g s) are done as
//   q = x r,  q' = q + (x - q g s) r,  r = 1 / (g s) correctly rounded,
// which is the correctly rounded quotient (Markstein 1990) as long as nothing
// overflows or underflows, and the roundings to E4M3 and E2M1 are the
// hardware's conversions, which go to nearest, ties to even, and saturate, as
// the format asks.  A block whose scale code is the largest (0x7E, where it may have
// saturated, and x r overflow: the correction makes that a NaN, whose conversion has no
// sign; infinities are there too) or a NaN, or whose scale g s lies outside [2^-90,
// 2^90], takes the quantiser of nvfp4.cuh, and all of them give its codes.
//
// Measured on GB300: four prompts of 4095 tokens, 8 heads of 128, with the values
// (153 MB) 30.4 us, 5.0 TB/s; with IEEE divisions and comparisons 68 us, with
// 64-bit index arithmetic repeated for K and for V 40 us.  At 72 % of the issue
// slots (363 instructions per 16 elements) the arithmetic still stands beside the
// memory.  32 single tokens 2.2 us.
#include "internal.h"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

// Eight fp32 values (as pairs) -> eight E2M1 codes, element i in bits 4 i.  The
// conversion keeps the sign of values that round to zero; the format has none there.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&y)[4]) {
    uint32_t w;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(y[i], v[2 * i], v[2 * i + 1]);
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    const uint32_t some = (w | (w >> 1) | (w >> 2)) & 0x11111111u;  // magnitude not zero
    return w & (0x77777777u | (some << 3));
}

// E4M3 code of a >= 0, finite.
__device__ __forceinline__ uint32_t e4m3_code_cvt(float a) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(a));
    return c;
}

// Codes, scale and values of this thread's 8 columns, of which its neighbour has the block's other 8.
__device__ __forceinline__ void quantise8(const uint4& u, const __nv_bfloat16* block, float g, int half, uint32_t& codes,
                                          uint32_t& sc) {
    uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t top = max(m & 0xFFFFu, m >> 16);  // largest magnitude of the block, as bf16 bits
    sc = e4m3_code_cvt(__fdiv_rn(__uint_as_float(top << 16), __fmul_rn(6.f, g)));
    const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16(sc) & 0xFFFFu)));
    const float gs = __fmul_rn(g, s);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    codes = 0u;
    if (sc < 0x7Eu && (s == 0.f || (gs >= 0x1p-90f && gs <= 0x1p90f))) {
        if (s > 0.f) {
            const float r = __frcp_rn(gs);
            const uint64_t r2 = f32x2(r, r), n2 = f32x2(-gs, -gs);
            uint64_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t x = bf16x2_to_f32x2(w[e]);
                const uint64_t q = mul_f32x2(x, r2);
                y[e] = fma_f32x2(fma_f32x2(q, n2, x), r2, q);
            }
            codes = e2m1x8(y);
        }
    } else {
        float x[16];
        const uint4* src = reinterpret_cast<const uint4*>(block);
        const uint4 u0 = __ldg(src), u1 = __ldg(src + 1);
        const uint32_t z[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[2 * e] = bf16_lo(z[e]);
            x[2 * e + 1] = bf16_hi(z[e]);
        }
        uint32_t pk[2];
        sc = nvfp4_block(x, g, pk);
        codes = half ? pk[1] : pk[0];
    }
}

// The bf16 values of 8 codes under scale code sc.
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t sc, float g) {
    const uint32_t s2 = __byte_perm(e4m3x2_to_f16(sc), 0u, 0x1010);
    uint32_t f[4], o[4];
    e2m1x8_to_f16(codes, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[e] = mul_f16x2(f[e], s2);  // exact
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[e]));
        o[e] = pack_bf16x2(__fmul_rn(v.x, g), __fmul_rn(v.y, g));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// One thread: 8 columns of one row of K and of V.  log_tpr: log2 of hd / 8.
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Append a, int log_tpr) {
    launch_dependents();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const unsigned rows = (unsigned)(a.batch * a.n_kv_h) * (unsigned)a.T;  // < 2^31
    const unsigned row = (unsigned)(i >> log_tpr);
    const int part = (int)i & ((1 << log_tpr) - 1);
    const unsigned slab = row / (unsigned)a.T, t = row - slab * (unsigned)a.T;
    grid_dependency_wait();
    // The two threads of a block are neighbours in a warp and live or die together.
    long long at = -1;
    uint4 uk = make_uint4(0u, 0u, 0u, 0u), uv = uk;
    if (row < rows && FMHA_IN_BOUNDS(i >= 0 && i < (long long)rows << log_tpr && slab / (unsigned)a.n_kv_h < (unsigned)a.batch,
                                     kSiteKv4Append, a.status)) {
        uk = __ldcs(reinterpret_cast<const uint4*>(a.k + i * 8));
        uv = __ldcs(reinterpret_cast<const uint4*>(a.v + i * 8));
        at = __ldg(a.start + slab / (unsigned)a.n_kv_h) + (long long)t;
    }
    uint32_t ck, cv, sk, sv;
    quantise8(uk, a.k + (i & ~1LL) * 8, a.k_global, part & 1, ck, sk);
    quantise8(uv, a.v + (i & ~1LL) * 8, a.v_global, part & 1, cv, sv);
    if (at < 0 || at >= a.cap) return;  // outside the cache, or past the rows: left out
    const long long dst = (((long long)slab * a.cap + at) << log_tpr) + part;
    if (!FMHA_IN_BOUNDS(dst >= 0 && dst < ((long long)a.batch * a.n_kv_h * a.cap) << log_tpr, kSiteKv4Append, a.status)) return;
    *reinterpret_cast<uint32_t*>(a.k_codes + dst * 4) = ck;
    *reinterpret_cast<uint32_t*>(a.v_codes + dst * 4) = cv;
    if ((part & 1) == 0) {
        a.k_scales[dst >> 1] = (uint8_t)sk;
        a.v_scales[dst >> 1] = (uint8_t)sv;
    }
    if (a.k_out) {
        __stcs(reinterpret_cast<uint4*>(a.k_out + i * 8), values8(ck, sk, a.k_global));
        __stcs(reinterpret_cast<uint4*>(a.v_out + i * 8), values8(cv, sv, a.v_global));
    }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Append& a, int hd, cudaStream_t stream) {
    const int log_tpr = hd == 64 ? 3 : hd == 128 ? 4 : hd == 256 ? 5 : 6;
    const long long blocks = (((long long)a.batch * a.n_kv_h * a.T << log_tpr) + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_append_kernel, a, log_tpr);
}

}  // namespace fmha
