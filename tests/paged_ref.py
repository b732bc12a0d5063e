"""64-bit plain implementations of the cache in pages for its tests, with the error that its number formats allow.

Rounding to bf16 is off by at most 2^-8 of the value, to E4M3 by 2^-4 (2^-10 below its smallest normal number 2^-6), to fp32
by 2^-24.  The attention's bounds are those of serving_ref.py: a relative error d of every weight moves a weighted mean of V rows by at
most 2 d times A = sum p |v| / sum p."""
import math

import torch

import serving_ref

# every value of an E4M3 code (the two NaNs as 480, which no row holds)
E4M3 = [(-1.0 if c >= 128 else 1.0) * ((c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)]


def quantise(x):
    """(codes, scale bytes) of bf16 rows [..., hd] by the definition, on the host, in 64 bits: the smallest power of two from 2^-127 on
    that brings the largest magnitude to 448 or less, the nearest code (ties to the even one); byte 255 for rows that are not finite."""
    x = x.double().cpu()
    fine = torch.isfinite(x).all(-1)
    y = torch.where(fine[..., None], x, torch.zeros_like(x))
    most = y.abs().amax(-1)
    e = torch.full_like(most, -127.0)
    for k in range(-127, 128):
        e = torch.where(448.0 * 2.0 ** (k - 1) < most, torch.full_like(e, float(k)), e)
    z = y / torch.exp2(e)[..., None]
    table = torch.tensor(E4M3[:127], dtype=torch.float64)  # magnitudes, rising with the code
    at = torch.searchsorted(table, z.abs().contiguous()).clamp(max=126)
    below = (at - 1).clamp(min=0)
    up, down = table[at] - z.abs(), z.abs() - table[below]
    code = torch.where((down < up) | ((down == up) & (below % 2 == 0)), below, at)
    code = torch.where((z < 0) | ((z == 0) & (torch.copysign(torch.ones_like(y), y) < 0)), code + 128, code)
    byte = torch.where(fine, e + 127, torch.full_like(e, 255.0))
    return torch.where(fine[..., None], code, torch.zeros_like(code)).to(torch.uint8), byte.to(torch.uint8)


def values(rows, scales):
    """fp64 values of stored rows (bf16, or codes and scale bytes)."""
    if scales is None:
        return rows.double()
    table = torch.tensor(E4M3, dtype=torch.float64, device=rows.device)
    s = torch.where(scales == 255, torch.full(scales.shape, math.nan, dtype=torch.float64, device=rows.device), torch.exp2(scales.double() - 127))
    return table[rows.long()] * s[..., None]


def sequence(pages, scales, table_row, n, page):
    """(fp64 rows [n_kv, n, hd], which of them are there [n]) of one sequence."""
    n_pages, heads, _, hd = pages.shape
    out = torch.zeros((heads, n, hd), dtype=torch.float64, device=pages.device)
    there = torch.zeros(n, dtype=torch.bool, device=pages.device)
    for i, p in enumerate(table_row.tolist()):
        lo, hi = i * page, min(n, (i + 1) * page)
        if hi <= lo or not 0 <= p < n_pages:
            continue
        out[:, lo:hi] = values(pages[p, :, : hi - lo], None if scales is None else scales[p, :, : hi - lo])
        there[lo:hi] = True
    return out, there


def attend_sequence(q, k, v, there, scale, window, n_first, causal, sink):
    """o, lse and their bounds for q [n_h, T, hd] over k, v [n_kv, n, hd], all fp64."""
    nh, T, hd = q.shape
    nk, n = k.shape[:2]
    G, dev = nh // nk, q.device
    j = torch.arange(n, device=dev)[None]
    p = (n - T + torch.arange(T, device=dev))[:, None]
    seen = there[None].expand(T, n).clone()
    if causal:
        seen &= j <= p
    if window > 0:
        seen &= (j > p - window) | (j < n_first)
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    x = q @ kk.transpose(1, 2) * scale
    # fp32 accumulation of hd products, the scale, the log2 domain and the exponential
    size = (q.abs() @ kk.abs().transpose(1, 2)) * abs(scale) * seen
    err = (size.amax(-1) if n else torch.zeros((nh, T), dtype=torch.float64, device=dev)) * (hd + 16) * 2.0 ** -24 + 2.0 ** -21
    x = x.masked_fill(~seen, -math.inf)
    terms = x if sink is None else torch.cat([x, sink.double().view(nh, 1, 1).expand(nh, T, 1)], 2)
    lse = torch.logsumexp(terms, -1) if terms.shape[2] else torch.full((nh, T), -math.inf, dtype=torch.float64, device=dev)
    w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None]).masked_fill(~seen, 0.0)
    o = w @ vv
    top_v = vv.abs().amax() if vv.numel() else 0.0
    # P in bf16 (2^-8), fp32 sums over n terms and over chunks, and terms below fp32's range
    o_tol = o.abs() * 2.0 ** -8 + (w @ vv.abs()) * (2 * 2.0 ** -8 + 2 * err[..., None] + n * 2.0 ** -24) + n * 2.0 ** -30 * top_v + 1e-30
    l_tol = err + (n + 16) * 2.0 ** -24 + torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs()) * 2.0 ** -22
    return o, lse, o_tol, l_tol


def attend(q, cache, table, lens, page, cu=None, scale=None, window=0, n_first=0, causal=False, sink=None):
    """As binding.fmha_fwd_paged, lens and cu on the host: o, lse and their bounds, of q's layout (rows that are no tokens: zeros)."""
    k_pages, v_pages, k_scales, v_scales = cache
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    outs = [torch.zeros(q.shape if i % 2 == 0 else q.shape[:-1], dtype=torch.float64, device=q.device) for i in range(4)]
    for i, n in enumerate(lens):
        k, there = sequence(k_pages, k_scales, table[i], n, page)
        v, _ = sequence(v_pages, v_scales, table[i], n, page)
        rows = q[i] if cu is None else q[cu[i] : cu[i + 1]].transpose(0, 1)
        got = attend_sequence(rows.double(), k, v, there, scale, window, n_first, causal, sink)
        for out, x in zip(outs, got):
            if cu is None:
                out[i] = x
            else:
                out[cu[i] : cu[i + 1]] = x.transpose(0, 1)
    return tuple(outs)


assert_attention = serving_ref.assert_attention
