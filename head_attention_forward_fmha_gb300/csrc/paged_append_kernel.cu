// paged_append_kernel.cu -- new K and V rows into a cache in pages, and rows of it back.
//
// Append: token t of sequence b goes to position start[b] + t, through the sequence's row of the
// block table, as bf16 or in 8 bits: the row's scale is the smallest power of two, 2^-127 at
// least, that brings its largest magnitude to 448 (E4M3's largest value) or less, and the codes are
// E4M3(x / scale), to nearest, ties to even.  A power of two wastes nothing of a floating-point
// code (its smallest values lose at most one of 17 binades), the division by it is exact, so
// that each value is rounded once, and code * scale is a bf16 value again: gather
// and the attention read exactly what was stored.  A row that holds a NaN or an infinity gets the scale
// byte 255, under which all of it reads as NaN.
//
// Gather: positions start[b] .. start[b] + rows - 1 below the sequence's length come back as
// contiguous bf16 rows; the others, and those whose page is not there, are left as they are.
//
// Both only move memory: a row of K and of V by a few lanes, each of which loads all that it needs before it
// stores, rows in the order of the contiguous tensors.  Measured (GB300, 16 x 4096 rows of 8 heads of 128, K and V;
// a plain copy runs at 6.71 TB/s):
//   append bf16 79.1 us, 6.79 TB/s; codes 60.9 us, 6.63 TB/s (ragged 64.4).  With 8 columns of K and V a lane in place
//   of 16 the codes took 85.9: what is done once a lane (page, reduction over the row) and not the quantiser filled the ALUs.
//   gather bf16 79.9 us, 6.72 TB/s; codes 60.9 us, 6.63 TB/s (69 with 16 codes in a row a lane, whose stores leave gaps).
// One token of 64 sequences takes 1.7 to 2.1 us (ragged 2.3 to 3.1, with the search for a token's sequence): the latency of a launch.
#include "internal.h"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace fmha {
namespace {

// Two fp32 values -> two E4M3 codes (lo in the low byte), saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

__device__ __forceinline__ uint32_t abs_max(const uint4& u) {
    return __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
}

// One thread: VEC times 8 columns of one row of K and of V, 8 * 2^log_tpr columns apart (2 for codes and where a row of 512
// has to lie in a warp).
template <bool CODES, int VEC>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAppend a, int log_tpr) {
    launch_dependents();
    const PagedCache& c = a.c;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int lane = threadIdx.x & 31, part = (int)i & ((1 << log_tpr) - 1);
    const unsigned row = (unsigned)(i >> log_tpr);
    const unsigned rows = (unsigned)(a.t.cu ? a.t.total : a.t.batch * a.t.T) * (unsigned)c.n_kv_h;  // < 2^31
    grid_dependency_wait();
    // The rows of uniform sequences run along a head's tokens, those of ragged ones along a token's heads.
    int b, h, t;
    long long token;  // by which the input's token stride goes
    if (!a.t.cu) {
        const unsigned slab = row / (unsigned)a.t.T;
        t = (int)(row - slab * (unsigned)a.t.T);
        b = (int)(slab / (unsigned)c.n_kv_h);
        h = (int)(slab - (unsigned)b * (unsigned)c.n_kv_h);
        token = t;
    } else {
        const int tok = (int)(row / (unsigned)c.n_kv_h);
        h = (int)(row - (unsigned)tok * (unsigned)c.n_kv_h);
        token = tok;
        // the first sequence whose end lies behind the token: ends at or before it are counted, or searched in large batches
        b = 0;
        if (a.t.batch <= kPagedScan) {
            for (int b0 = 0; b0 < a.t.batch; b0 += 32) {
                int end = INT_MAX;
                if (b0 + lane < a.t.batch) end = __ldg(a.t.cu + b0 + lane + 1);
                for (int g = 0; g < 32; g += 1 << log_tpr) {
                    const unsigned before = __ballot_sync(0xffffffffu, end <= __shfl_sync(0xffffffffu, tok, g));
                    if ((lane >> log_tpr) == (g >> log_tpr)) b += __popc(before);
                }
            }
        } else {
            for (int n = a.t.batch; n > 0;) {  // ends b .. b + n - 1 may lie behind it
                const int half = n >> 1;
                if (__ldg(a.t.cu + b + half + 1) <= tok) {
                    b += half + 1;
                    n -= half + 1;
                } else {
                    n = half;
                }
            }
        }
        t = -1;
        if (b < a.t.batch && tok < a.t.total && FMHA_IN_BOUNDS(b >= 0, kSitePagedSeq, a.status)) t = tok - __ldg(a.t.cu + b);
    }
    const bool live = row < rows && t >= 0 && FMHA_IN_BOUNDS(b >= 0 && b < a.t.batch && h < c.n_kv_h, kSitePagedIo, a.status);
    uint4 u[2][VEC];
    long long dst = -1;
    if (live) {
        const long long pos = (long long)__ldg(a.start + b) + t;
        const long long ka = (a.t.cu ? 0 : b * a.k_strides[0]) + token * a.k_strides[1] + h * a.k_strides[2] + part * 8;
        const long long va = (a.t.cu ? 0 : b * a.v_strides[0]) + token * a.v_strides[1] + h * a.v_strides[2] + part * 8;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            u[0][v] = __ldcs(reinterpret_cast<const uint4*>(a.k + ka + (v * 8 << log_tpr)));
            u[1][v] = __ldcs(reinterpret_cast<const uint4*>(a.v + va + (v * 8 << log_tpr)));
        }
        if (pos >= 0 && pos < (long long)c.width << c.log_page)
            dst = paged_row(c, paged_page(c, paged_entry(c, a.t.batch, b, (int)(pos >> c.log_page), a.status)), h, (int)(pos & (c.page - 1)));
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) u[0][v] = u[1][v] = make_uint4(0u, 0u, 0u, 0u);
    }
    const bool store = dst >= 0 && FMHA_IN_BOUNDS(paged_row_ok(c, dst), kSitePagedRow, a.status);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if constexpr (!CODES) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(x ? c.v_pages : c.k_pages) + dst * c.hd + part * 8;
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (store) *reinterpret_cast<uint4*>(out + (v * 8 << log_tpr)) = u[x][v];
        } else {
            uint32_t m = abs_max(u[x][0]);
            if constexpr (VEC == 2) m = __vmaxu2(m, abs_max(u[x][1]));
            for (int s = 1; s < 1 << log_tpr; s <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, s));
            const uint32_t top = max(m & 0xFFFFu, m >> 16);  // largest magnitude of the row, as bf16 bits
            // 448 = 1.75 * 2^8: a mantissa above 1.75 takes the next power
            const int e = (int)(top >> 7) - 8 + ((top & 0x7Fu) > 96u ? 1 : 0);
            const bool finite = top < 0x7F80u;
            const uint32_t byte = finite ? (uint32_t)max(e, 0) : 255u;
            const float up = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte); bytes of finite rows end at 247
            if (!store) continue;
            uint8_t* out = static_cast<uint8_t*>(x ? c.v_pages : c.k_pages) + dst * c.hd + part * 8;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const uint32_t w[4] = {u[x][v].x, u[x][v].y, u[x][v].z, u[x][v].w};
                uint32_t q[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) q[y] = finite ? e4m3x2(bf16_lo(w[y]) * up, bf16_hi(w[y]) * up) : 0u;
                *reinterpret_cast<uint2*>(out + (v * 8 << log_tpr)) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
            }
            if (part == 0) (x ? c.v_scales : c.k_scales)[dst] = (uint8_t)byte;
        }
    }
}

// One thread: 16 bytes of a stored row of K and of V, for codes in two pieces.
template <bool CODES>
__global__ void __launch_bounds__(256) paged_gather_kernel(const PagedGather a, int log_tpr) {
    launch_dependents();
    const PagedCache& c = a.c;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int part = (int)i & ((1 << log_tpr) - 1);
    const unsigned row = (unsigned)(i >> log_tpr), slab = row / (unsigned)a.rows;
    const int r = (int)(row - slab * (unsigned)a.rows);
    const int b = (int)(slab / (unsigned)c.n_kv_h), h = (int)(slab - (unsigned)b * (unsigned)c.n_kv_h);
    grid_dependency_wait();
    if (row >= (unsigned)(a.batch * c.n_kv_h) * (unsigned)a.rows) return;
    if (!FMHA_IN_BOUNDS(b >= 0 && b < a.batch, kSitePagedSeq, a.status)) return;
    const long long pos = (a.start ? (long long)__ldg(a.start + b) : 0) + r;
    if (pos < 0 || pos >= __ldg(a.seq_lens + b) || pos >= (long long)c.width << c.log_page) return;
    const int src = paged_row(c, paged_page(c, paged_entry(c, a.batch, b, (int)(pos >> c.log_page), a.status)), h, (int)(pos & (c.page - 1)));
    if (src < 0 || !FMHA_IN_BOUNDS(paged_row_ok(c, src), kSitePagedRow, a.status)) return;
    if constexpr (!CODES) {
        const long long at = ((long long)src << log_tpr) + part;  // in 16-byte units
        const uint4 uk = __ldcs(static_cast<const uint4*>(c.k_pages) + at), uv = __ldcs(static_cast<const uint4*>(c.v_pages) + at);
        __stcs(reinterpret_cast<uint4*>(a.k) + i, uk);
        __stcs(reinterpret_cast<uint4*>(a.v) + i, uv);
    } else {
        // two pieces of 8 codes, half a row apart: each becomes 16 bytes, so that a warp's loads and stores are dense
        const long long from = ((long long)src << (log_tpr + 1)) + part, to = ((long long)row << (log_tpr + 1)) + part;
        uint2 u[2][2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            u[0][v] = __ldcs(static_cast<const uint2*>(c.k_pages) + from + (v << log_tpr));
            u[1][v] = __ldcs(static_cast<const uint2*>(c.v_pages) + from + (v << log_tpr));
        }
        const PagedFactor fk = paged_factor(__ldg(c.k_scales + src)), fv = paged_factor(__ldg(c.v_scales + src));
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                uint32_t e0, o0, e1, o1;
                paged_values4(u[x][v].x, x ? fv : fk, e0, o0);
                paged_values4(u[x][v].y, x ? fv : fk, e1, o1);
                __stcs(reinterpret_cast<uint4*>(x ? a.v : a.k) + to + (v << log_tpr),
                       make_uint4(__byte_perm(e0, o0, 0x5410), __byte_perm(e0, o0, 0x7632), __byte_perm(e1, o1, 0x5410), __byte_perm(e1, o1, 0x7632)));
            }
    }
}

template <class Kernel, class Args>
cudaError_t launch_rows(Kernel kern, const Args& a, long long threads, int log_tpr, cudaStream_t stream) {
    const long long blocks = (threads + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {programmatic_launch_attr()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, log_tpr);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppend& a, cudaStream_t stream) {
    const bool codes = a.c.k_scales != nullptr;
    const int hd = a.c.hd, log_tpr = (hd == 64 ? 3 : hd == 128 ? 4 : hd == 256 ? 5 : 6) - (codes || hd == 512 ? 1 : 0);  // a row lies in one warp
    const long long tokens = a.t.cu ? a.t.total : (long long)a.t.batch * a.t.T;
    const long long threads = tokens * a.c.n_kv_h << log_tpr;
    if (codes) return launch_rows(paged_append_kernel<true, 2>, a, threads, log_tpr, stream);
    return hd == 512 ? launch_rows(paged_append_kernel<false, 2>, a, threads, log_tpr, stream)
                     : launch_rows(paged_append_kernel<false, 1>, a, threads, log_tpr, stream);
}

cudaError_t launch_paged_gather(const PagedGather& a, cudaStream_t stream) {
    const bool codes = a.c.k_scales != nullptr;
    const int hd = a.c.hd, log_tpr = (hd == 64 ? 3 : hd == 128 ? 4 : hd == 256 ? 5 : 6) - (codes ? 1 : 0);
    const long long threads = (long long)a.batch * a.c.n_kv_h * a.rows << log_tpr;
    return codes ? launch_rows(paged_gather_kernel<true>, a, threads, log_tpr, stream)
                 : launch_rows(paged_gather_kernel<false>, a, threads, log_tpr, stream);
}

}  // namespace fmha
