"""64-bit plain implementations of the serving operators (norm and rotation, 4-bit
cache, attention with first keys) for their tests, with the error that their
number formats allow.

Rounding to bf16 is off by at most 2^-8 of the value, to fp16 by 2^-11, to fp32 by
2^-24.  An attention output is a weighted mean of V rows: a relative error d of
every weight moves it by at most 2 d times A = sum p |v| / sum p, so the bounds
below are multiples of A, of the value itself and of the scores' error.
"""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dequantise(codes, scales, g):
    """fp64 rows of uint8 codes [..., hd / 2] and E4M3 bytes [..., hd / 16]."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=codes.device)
    x = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(torch.float64)
    return x * s.repeat_interleave(16, -1) * g


def norm_rope(x, weight, eps, cos, sin, interleaved):
    """x [..., hd] fp64; cos, sin [..., rot / 2] or None.  Returns (result, bound on its fp32 error)."""
    y = x
    if weight is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    out = y.clone()
    mag = y.abs()
    if cos is not None:
        h = cos.shape[-1]
        lo, hi = (y[..., 0 : 2 * h : 2], y[..., 1 : 2 * h : 2]) if interleaved else (y[..., :h], y[..., h : 2 * h])
        a, b = lo * cos - hi * sin, hi * cos + lo * sin
        m = lo.abs() + hi.abs()
        if interleaved:
            out[..., 0 : 2 * h : 2], out[..., 1 : 2 * h : 2] = a, b
            mag[..., 0 : 2 * h : 2], mag[..., 1 : 2 * h : 2] = m, m
        else:
            out[..., :h], out[..., h : 2 * h] = a, b
            mag[..., :h], mag[..., h : 2 * h] = m, m
    # sum of squares over hd terms, rsqrt (2 ulp), three products and a sum, all in fp32
    hd = x.shape[-1]
    return out, out.abs() * 2.0 ** -8 + mag * (hd / 2 + 16) * 2.0 ** -24 + 1e-38


def attend(q, k, v, lens, scale, window=0, n_first=0, causal=False, sink=None, p_bits=11):
    """fp64 attention over k, v [b, n_kv, n, hd] of which sequence i has lens[i] keys.
    Returns o, lse and the bounds on the errors of bf16 o and fp32 lse, P rounded to p_bits significant bits."""
    b, nh, T, hd = q.shape
    nk, n = k.shape[1], k.shape[2]
    dev = q.device
    q, k, v = q.double(), k.double(), v.double()
    o = torch.zeros((b, nh, T, hd), dtype=torch.float64, device=dev)
    lse = torch.full((b, nh, T), -math.inf, dtype=torch.float64, device=dev)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    G = nh // nk
    for i in range(b):
        m = int(lens[i])
        j = torch.arange(m, device=dev)[None, :]
        p = (m - T + torch.arange(T, device=dev))[:, None]
        seen = torch.ones((T, m), dtype=torch.bool, device=dev)
        if causal:
            seen &= j <= p
        if window > 0:
            seen &= (j > p - window) | (j < n_first)
        for h in range(nh):
            kk, vv = k[i, h // G, :m], v[i, h // G, :m]
            x = (q[i, h] @ kk.T) * scale
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            # fp32 accumulation of hd products, the scale, the log2 domain and the exponential
            size = (q[i, h].abs() @ kk.abs().T) * abs(scale) * seen
            err = (size.amax(-1) if m else torch.zeros(T, dtype=torch.float64, device=dev)) * (hd + 16) * 2.0 ** -24 + 2.0 ** -21
            terms = x if sink is None else torch.cat([x, sink[h].double().reshape(1, 1).expand(T, 1)], 1)
            if terms.shape[1] == 0:
                continue
            top = torch.logsumexp(terms, -1)
            w = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top)[:, None])
            w = torch.where(seen, w, torch.zeros_like(w))
            o[i, h], lse[i, h] = w @ vv, top
            A = w @ vv.abs()
            top_v = vv.abs().amax() if m else 0.0
            o_tol[i, h] = o[i, h].abs() * 2.0 ** -8 + A * (2 * 2.0 ** -p_bits + 2 * err[:, None] + m * 2.0 ** -24) + m * 2.0 ** -30 * top_v + 1e-30
            lse_tol[i, h] = err + (m + 16) * 2.0 ** -24 + torch.where(torch.isinf(top), torch.zeros_like(top), top.abs()) * 2.0 ** -22
    return o, lse, o_tol, lse_tol


def assert_attention(got, ref, label=""):
    (o, lse), (ro, rl, o_tol, l_tol) = got, ref
    o, lse = o.double(), lse.double()
    assert torch.isfinite(o).all(), label + ": O is not finite"
    assert torch.equal(torch.isinf(lse), torch.isinf(rl)), label + ": pattern of -inf in LSE differs"
    off = (o - ro).abs() - o_tol
    assert (off <= 0).all(), "%s: O off by %.3e beyond its bound" % (label, off.max().item())
    fin = torch.isfinite(rl)
    off = ((lse - rl).abs() - l_tol)[fin]
    assert off.numel() == 0 or (off <= 0).all(), "%s: LSE off by %.3e beyond its bound" % (label, off.max().item())
