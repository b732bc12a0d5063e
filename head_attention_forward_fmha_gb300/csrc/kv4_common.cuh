// kv4_common.cuh -- pieces shared by the two kernels of the attention over a
// 4-bit cache (kv4_kernel.cu, kv4_tc_kernel.cu).
#pragma once
#include <cmath>
#include "internal.h"
#include "ptx.cuh"

namespace fmha {

constexpr float kPBias = 6.f;  // log2 of the factor that P and its sum carry

// |scale| * k_global * log2(e) as mant * 2^expo, mant in [1, 2), and the scale's sign
// (0 for a product of zero: mant 1, expo 0).  Apart because a row's factor, this times
// the power of two that undoes Q's scaling, may pass fp32's range on either side.
struct ScoreScale {
    float mant, sign;
    int expo;
};

inline ScoreScale score_scale(const Kv4Fwd& f) {
    const double s = (double)f.scale * f.k_global * 1.4426950408889634;
    ScoreScale r{1.f, 0.f, 0};
    if (s == 0) return r;
    r.sign = s > 0 ? 1.f : -1.f;
    r.mant = 2.f * (float)std::frexp(std::fabs(s), &r.expo);  // 2 if it was rounded up to 1
    r.expo -= 1;
    if (r.mant >= 2.f) {
        r.mant = 1.f;
        r.expo += 1;
    }
    return r;
}

// The row's factor mant * 2^e, e kept within fp32's normal numbers: neither 0, which would turn
// the masked scores' -inf into NaN, nor infinite, which would turn scores of 0 into NaN.
// Below 2^-126 it makes all weights equal as it should (products are below 2^36).
__device__ __forceinline__ float score_factor(float mant, int e) {
    return __uint_as_float(__float_as_uint(mant) + ((uint32_t)min(max(e, -126), 127) << 23));
}

// Sequence b's length.
__device__ __forceinline__ int seq_len(const Kv4Fwd& f, int b) {
    if (!FMHA_IN_BOUNDS(b >= 0 && b < f.batch, kSiteKv4Copy, f.status)) return 0;
    return min(max(__ldg(f.seq_lens + b), 0), f.s_k);
}

// End of a row: finish_row, but where a NaN score has made the sum NaN, so are O and
// LSE.  (finish_row gives such a row LSE = -inf, which marks an empty chunk: the merge
// would leave it out, and whether the NaN shows would depend on the number of chunks.)
__device__ __forceinline__ void finish_row_nan(float m, float l, float sink_l2, float& inv, float& lse) {
    finish_row(m, l, sink_l2, inv, lse);
    if (l != l) inv = lse = l;
}

// Output of a block whose rows attend no key of their chunk, by all of its
// threads: rows first .. first + n - 1, columns col0 .. col0 + ncol - 1: O = 0 and
// LSE = -inf, or the row's sink in a final output (sink_head0 >= 0: the query
// head of row_in_slab 0; the first row is row r0 of its slab).  Of a partial's O
// the merge reads nothing then, unless there are few chunks.
__device__ __forceinline__ void write_empty_rows(const Kv4Fwd& f, long long rows_total, long long first, int n, int split,
                                                 int col0, int ncol, bool with_lse, int sink_head0, int r0) {
    const int threads = blockDim.x, per_row = ncol / 8;
    for (int i = threadIdx.x; f.n_splits <= kMergeReadsAll && i < n * per_row; i += threads) {
        const int r = i / per_row, c = col0 + (i - r * per_row) * 8;
        if (!FMHA_IN_BOUNDS(first + r >= 0 && first + r < rows_total && c + 8 <= f.hd && split < f.n_splits, kSiteKv4Out,
                            f.status))
            continue;
        if (f.n_splits == 1) {
            *reinterpret_cast<uint4*>(f.o + (first + r) * f.hd + c) = make_uint4(0u, 0u, 0u, 0u);
        } else if (f.range_part) {
            *reinterpret_cast<uint4*>(static_cast<__half*>(f.o_part) + (split * rows_total + first + r) * f.hd + c) =
                make_uint4(0u, 0u, 0u, 0u);
        } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(f.o_part) + (split * rows_total + first + r) * f.hd + c);
            dst[0] = dst[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (f.n_splits > 1 && f.range_part)
        for (int r = threadIdx.x; r < n; r += threads)
            if (FMHA_IN_BOUNDS(first + r >= 0 && first + r < rows_total && split < f.n_splits && col0 / 256 < 2, kSiteKv4Range, f.status))
                f.range_part[(split * rows_total + first + r) * 2 + col0 / 256] = 1.f;
    if (!with_lse) return;
    for (int r = threadIdx.x; r < n; r += threads) {
        if (!FMHA_IN_BOUNDS(first + r >= 0 && first + r < rows_total && split < f.n_splits &&
                                (sink_head0 < 0 || sink_head0 + (r0 + r) / f.T < f.n_h),
                            kSiteKv4Out, f.status))
            continue;
        if (f.n_splits == 1)
            f.lse[first + r] = sink_head0 >= 0 ? __ldg(f.sink + sink_head0 + (r0 + r) / f.T) : -INFINITY;
        else
            f.lse_part[split * rows_total + first + r] = -INFINITY;
    }
}

}  // namespace fmha
