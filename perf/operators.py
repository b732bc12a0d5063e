"""The serving operators around the attention forward, as cases that can be timed and compared.

Four operators, in the order in which a decode step or a prompt chunk runs them:

  norm_rope    one pass from the rows of a QKV projection (token-major) to what attention takes (head-major): RMS norm of
               every query and key head with a learned weight, rotation by the token's position, V copied over.
  kv4_append   new K and V rows quantised to 4 bits (16-element blocks of E2M1 codes under an E4M3 scale) and written into a
               cache at each sequence's own position; the values that the cache then stands for come back in bf16.
  kv4_attend   attention over such a cache, each sequence with a length of its own.
  first_attend attention over bf16 K and V with a sliding window and a few first keys that stay visible.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: this repository's entry points.
"""
import math

import torch

own = False

DEV = "cuda"

# ---------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of one sequence on its way into attention: the smallest call of a decode step
        dict(name="norm_rope one token", op="norm_rope", batch=1, T=1, n_h=64, n_kv_h=8, hd=128, rot=128, interleaved=False, pad=0, max_pos=32768),
        # a decode step of a full batch, rotating half of a wide head, on rows that lie inside a wider buffer
        dict(name="norm_rope decode batch", op="norm_rope", batch=256, T=1, n_h=32, n_kv_h=32, hd=256, rot=128, interleaved=True, pad=64, max_pos=32768),
        # prompts: four sequences, an odd number of tokens each
        dict(name="norm_rope prompts", op="norm_rope", batch=4, T=4095, n_h=64, n_kv_h=8, hd=128, rot=128, interleaved=False, pad=0, max_pos=32768),
        # the new token of each sequence of a decode batch goes into the cache
        dict(name="kv4_append decode batch", op="kv4_append", batch=32, n_kv_h=8, T=1, cap=8192, hd=128, g=1.0),
        # prompts go into the cache, sequences at odd positions
        dict(name="kv4_append prompts", op="kv4_append", batch=4, n_kv_h=8, T=4095, cap=8192, hd=128, g=0.25),
        # one user's decode step over some thousand tokens: latency counts
        dict(name="kv4_attend one user", op="kv4_attend", batch=1, n_h=64, n_kv_h=8, T=1, cap=8192, hd=128, window=0, n_first=0, causal=False, sink=False, ragged=False, g=1.0),
        # a decode batch of sequences of very different lengths, up to 32768 tokens
        dict(name="kv4_attend ragged batch", op="kv4_attend", batch=32, n_h=64, n_kv_h=8, T=1, cap=32768, hd=128, window=0, n_first=0, causal=False, sink=False, ragged=True, g=1.0),
        # one K/V head of 512 columns shared by 128 query heads
        dict(name="kv4_attend shared head", op="kv4_attend", batch=16, n_h=128, n_kv_h=1, T=1, cap=4096, hd=512, window=0, n_first=0, causal=False, sink=False, ragged=True, g=0.5),
        # a prompt chunk of 128 tokens over what the cache holds, windowed, the first four tokens kept visible
        dict(name="kv4_attend prompt chunk", op="kv4_attend", batch=4, n_h=64, n_kv_h=8, T=128, cap=4096, hd=128, window=2048, n_first=4, causal=True, sink=False, ragged=True, g=1.0),
        # one sequence's decode step with a short window
        dict(name="first_attend one user", op="first_attend", batch=1, n_h=16, n_kv_h=16, T=1, s_k=4096, hd=64, window=1024, n_first=4, causal=False, sink=False),
        # the sliding-window decode batch, with four first tokens
        dict(name="first_attend decode batch", op="first_attend", batch=32, n_h=64, n_kv_h=8, T=1, s_k=8192, hd=128, window=4096, n_first=4, causal=False, sink=False),
        # a prompt chunk of 128 tokens, windowed
        dict(name="first_attend prompt chunk", op="first_attend", batch=4, n_h=64, n_kv_h=8, T=128, s_k=4096, hd=128, window=2048, n_first=16, causal=True, sink=False),
    ]


# (n_h, n_kv_h): every head its own K/V, groups (odd ones too), one shared K/V head
HEADS = [(1, 1), (16, 16), (32, 32), (64, 8), (32, 8), (40, 8), (12, 4), (6, 2), (128, 1), (5, 1), (24, 3)]
HD = [64, 128, 128, 256, 512]


def _log(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def _scores(c):
    """Query rows times keys: what the plain form holds in 32 bits."""
    return c["batch"] * c["n_h"] * c["T"] * (c["cap"] if c["op"] == "kv4_attend" else c["s_k"])


def draw(rng):
    op = rng.choice(["norm_rope", "kv4_append", "kv4_attend", "kv4_attend", "first_attend", "first_attend"])
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    while True:
        n_h, n_kv_h = rng.choice(HEADS)
        hd = rng.choice(HD)
        batch = _log(rng, 1, 64)
        c = dict(op=op, batch=batch, n_h=n_h, n_kv_h=n_kv_h, hd=hd)
        if op == "norm_rope":
            c.update(T=_log(rng, 1, 4096) if rng.random() < 0.6 else 1, rot=rng.choice([hd, hd, hd // 2, hd // 4, hd // 8 * 3]),
                     interleaved=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 64]), max_pos=_log(rng, 8192, 131072))
        elif op == "kv4_append":
            del c["n_h"]
            c.update(T=_log(rng, 1, 4096) if rng.random() < 0.6 else 1, cap=16 * _log(rng, 256, 2048), g=rng.choice([1.0, 0.25, 0.5, 2.0]))
        elif op == "kv4_attend":
            T = 1 if rng.random() < 0.5 else _log(rng, 2, 128)
            c.update(T=T, cap=16 * _log(rng, 16, 2048), window=0 if rng.random() < 0.5 else _log(rng, 16, 4096),
                     n_first=rng.choice([0, 1, 4, 7, 64]), causal=T > 1 and rng.random() < 0.8, sink=rng.random() < 0.25,
                     ragged=rng.random() < 0.7, g=rng.choice([1.0, 0.25, 0.5, 2.0]))
        else:
            T = 1 if rng.random() < 0.5 else _log(rng, 2, 128)
            c.update(T=T, s_k=_log(rng, 256, 32768), window=_log(rng, 16, 4096), n_first=rng.choice([1, 4, 7, 64, 200]),
                     causal=T > 1 and rng.random() < 0.8, sink=rng.random() < 0.25)
        w = work(c)
        if w["bytes"] > top[op][0] or w["flops"] > top[op][1]:
            continue
        if op == "norm_rope" and c["max_pos"] * c["rot"] > 1 << 24:
            continue
        if op == "kv4_append" and c["T"] * 2 > c["cap"]:
            continue
        if op == "kv4_append" and c["batch"] * n_kv_h * c["cap"] * hd > 1 << 29:
            continue
        if op.endswith("attend"):
            keys = c["cap"] if op == "kv4_attend" else c["s_k"]
            if _scores(c) > 1 << 27 or c["batch"] * n_kv_h * keys * hd > 1 << 29 or c["T"] > keys:
                continue
        return c


# ----------------------------------------------------------------------------------------------------------- lengths, work


def _lens(c, seed):
    """The sequences' lengths, on the host.  Ragged: spread over the cache, one sequence with a single token."""
    if not c["ragged"]:
        return [c["cap"] - 1] * c["batch"]
    g = torch.Generator().manual_seed(seed + 77)
    lo = min(c["T"], c["cap"])
    lens = torch.randint(lo, c["cap"] + 1, (c["batch"],), generator=g).tolist()
    if c["batch"] > 2:
        lens[1] = lo
    return lens


def _visible(lens, T, window, n_first, causal):
    """(keys that some row of a sequence attends, pairs of rows and keys), summed over sequences."""
    keys = pairs = 0
    for n in lens:
        lo = n
        for t in sorted({0, T - 1}):
            p = n - T + t
            hi = min(n, p + 1) if causal else n
            first = max(0, p - window + 1) if window > 0 else 0
            lo = min(lo, first)
            got = max(0, hi - first) + min(n_first, first, max(0, hi))
            pairs += got * T / (2.0 if T > 1 else 1.0)
        lo = max(0, lo)
        keys += max(0, n - lo) + min(n_first, lo)
    return keys, pairs


def work(c):
    if c["op"] == "norm_rope":
        heads = c["n_h"] + 2 * c["n_kv_h"]
        tokens = c["batch"] * c["T"]
        n = tokens * heads * c["hd"]
        table = min(tokens, c["max_pos"]) * c["rot"] * 4
        return {"bytes": 4.0 * n + table + 8.0 * tokens + 8.0 * c["hd"], "flops": 10.0 * tokens * (c["n_h"] + c["n_kv_h"]) * c["hd"]}
    if c["op"] == "kv4_append":
        n = 2 * c["batch"] * c["n_kv_h"] * c["T"] * c["hd"]  # K and V: bf16 in, codes and scales out, bf16 values out
        return {"bytes": n * (2 + 0.5 + 1 / 16 + 2) + 4.0 * c["batch"], "flops": 8.0 * n}
    rows = c["batch"] * c["n_h"] * c["T"]
    if c["op"] == "kv4_attend":
        # ragged lengths are uniform over the cache whatever the seed: their expected sum is what counts
        lens = [(c["T"] + c["cap"]) / 2.0 if c["ragged"] else c["cap"] - 1] * c["batch"]
        per_key = 2 * c["hd"] * (0.5 + 1 / 16)
    else:
        lens = [c["s_k"]] * c["batch"]
        per_key = 2 * c["hd"] * 2
    keys, pairs = _visible(lens, c["T"], c["window"], c["n_first"], c["causal"])
    return {"bytes": keys * c["n_kv_h"] * per_key + rows * (4.0 * c["hd"] + 4), "flops": 4.0 * pairs * c["n_h"] * c["hd"]}


# ---------------------------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _keys(gen, *shape):
    """K rows: normal, with a few channels several times as large as the others, as trained models have them."""
    gain = 1.0 + 3.0 * (torch.rand((shape[1], 1, shape[3]), generator=gen, device=DEV) > 0.96)
    return (_normal(gen, *shape) * gain).to(torch.bfloat16)


def _filled_cache(gen, c):
    """Codes and scales of a cache that earlier tokens have filled to its end (rows behind a sequence are stale)."""
    b, h, cap, hd = c["batch"], c["n_kv_h"], c["cap"], c["hd"]
    out = {}
    for name in ("k", "v"):
        codes = torch.empty((b, h, cap, hd // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((b, h, cap, hd // 16), dtype=torch.uint8, device=DEV)
        for i in range(b):
            x = _keys(gen, 1, h, cap, hd) if name == "k" else _normal(gen, 1, h, cap, hd).to(torch.bfloat16)
            codes[i : i + 1], scales[i : i + 1], _ = _quantise(x, c["g"])
        out[name + "_codes"], out[name + "_scales"] = codes, scales
    return out


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    b, hd, T = c["batch"], c["hd"], c["T"]
    s = {"c": c}
    if c["op"] == "norm_rope":
        heads = c["n_h"] + 2 * c["n_kv_h"]
        wide = _normal(gen, b, T, heads * hd + c["pad"]).to(torch.bfloat16)
        s["qkv"] = wide[..., : heads * hd]
        s["q_weight"] = 1.0 + 0.2 * _normal(gen, hd)
        s["k_weight"] = 1.0 + 0.2 * _normal(gen, hd)
        # the table that a serving program keeps: cosines, then sines, of every position's angles (64 bits until rounded)
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        angle = torch.arange(c["max_pos"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        at = torch.randint(0, max(1, c["max_pos"] - T), (b, 1), generator=gen, device=DEV)
        s["positions"] = (at + torch.arange(T, device=DEV)).to(torch.int32)
        s["q"] = torch.zeros((b, c["n_h"], T, hd), dtype=torch.bfloat16, device=DEV)
        s["k"] = torch.zeros((b, c["n_kv_h"], T, hd), dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.zeros_like(s["k"])
        return s
    if c["op"] == "kv4_append":
        h, cap = c["n_kv_h"], c["cap"]
        s["k"] = _keys(gen, b, h, T, hd)
        s["v"] = _normal(gen, b, h, T, hd).to(torch.bfloat16)
        s["start"] = torch.randint(0, cap - T + 1, (b,), generator=gen, device=DEV).to(torch.int32)
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros((b, h, cap, hd // 2), dtype=torch.uint8, device=DEV)
            s[name + "_scales"] = torch.zeros((b, h, cap, hd // 16), dtype=torch.uint8, device=DEV)
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        return s
    s["q"] = _normal(gen, b, c["n_h"], T, hd).to(torch.bfloat16)
    s["o"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((b, c["n_h"], T), dtype=torch.float32, device=DEV)
    s["sink"] = _normal(gen, c["n_h"]) if c["sink"] else None
    if c["op"] == "kv4_attend":
        s.update(_filled_cache(gen, c))
        s["lens"] = torch.tensor(_lens(c, seed), dtype=torch.int32, device=DEV)
    else:
        s["k"] = _keys(gen, b, c["n_kv_h"], c["s_k"], hd)
        s["v"] = _normal(gen, b, c["n_kv_h"], c["s_k"], hd).to(torch.bfloat16)
        s["lens"] = torch.full((b,), c["s_k"], dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------------------ plain forms


def _norm_rope(s):
    c = s["c"]
    b, T, hd, rot = c["batch"], c["T"], c["hd"], c["rot"]
    x = s["qkv"].float().reshape(b, T, c["n_h"] + 2 * c["n_kv_h"], hd).transpose(1, 2)
    nh, nk = c["n_h"], c["n_kv_h"]
    row = s["cos_sin"][s["positions"].long()][:, None]  # [b, 1, T, rot]
    cos, sin = row[..., : rot // 2], row[..., rot // 2 :]

    def turned(y, weight):
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
        z = y[..., :rot]
        lo, hi = (z[..., 0::2], z[..., 1::2]) if c["interleaved"] else (z[..., : rot // 2], z[..., rot // 2 :])
        lo, hi = lo * cos - hi * sin, hi * cos + lo * sin
        z = torch.stack([lo, hi], -1).flatten(-2) if c["interleaved"] else torch.cat([lo, hi], -1)
        return torch.cat([z, y[..., rot:]], -1).to(torch.bfloat16)

    s["q"].copy_(turned(x[:, :nh], s["q_weight"]))
    s["k"].copy_(turned(x[:, nh : nh + nk], s["k_weight"]))
    s["v"].copy_(x[:, nh + nk :])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _quantise(x, g):
    """(codes two to a byte, scale bytes, the values they stand for) of bf16 rows, 16 elements to a block."""
    y = x.float().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1, keepdim=True) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scale.float()
    y = torch.where(sf > 0, y / (g * sf), torch.zeros_like(y))
    a = y.abs()
    e = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
         + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    sign = (y < 0) & (e > 0)
    v = table[e.int()] * sf * g
    v = torch.where(sign, -v, v).flatten(-2).to(torch.bfloat16)
    e = torch.where(sign, e + 8, e).flatten(-2)
    return e[..., 0::2] | (e[..., 1::2] << 4), scale.view(torch.uint8).squeeze(-1), v


def _kv4_append(s):
    c = s["c"]
    b = torch.arange(c["batch"], device=DEV)[:, None, None]
    h = torch.arange(c["n_kv_h"], device=DEV)[None, :, None]
    at = (s["start"].long()[:, None] + torch.arange(c["T"], device=DEV))[:, None]
    for name in ("k", "v"):
        codes, scales, values = _quantise(s[name], c["g"])
        s[name + "_codes"][b, h, at] = codes
        s[name + "_scales"][b, h, at] = scales
        s[name + "_out"].copy_(values)
    return _appended(s)


def _appended(s):
    return {n: s[n] for n in ("k_out", "v_out", "k_codes", "k_scales", "v_codes", "v_scales")}


def _values(codes, scales, g):
    """fp32 rows from codes and scale bytes."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    x = x.unflatten(-1, (-1, 16)) * (scales.view(torch.float8_e4m3fn).float() * g)[..., None]
    return x.flatten(-2)


def _attend(s, k, v):
    c, q = s["c"], s["q"]
    b, nh, T, hd = q.shape
    nk, n = k.shape[1], k.shape[2]
    j = torch.arange(n, device=DEV)[None, None]
    p = (s["lens"].long()[:, None] - T + torch.arange(T, device=DEV))[..., None]
    seen = (j < s["lens"].long()[:, None, None]).expand(b, T, n)
    if c["causal"]:
        seen = seen & (j <= p)
    if c["window"] > 0:
        seen = seen & ((j > p - c["window"]) | (j < c["n_first"]))
    x = q.float().reshape(b, nk, nh // nk * T, hd) @ k.transpose(-1, -2) * hd ** -0.5
    x = x.view(b, nk, nh // nk, T, n).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        extra = s["sink"].view(1, nk, nh // nk, 1, 1)
        top = torch.maximum(top, extra)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(extra - top)
    o = (w.flatten(2, 3) @ v).view(b, nk, nh // nk, T, hd)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["o"].copy_(o.reshape(b, nh, T, hd))
    s["lse"].copy_((top + torch.log(total)).reshape(b, nh, T))
    return {"o": s["o"], "lse": s["lse"]}


def run(s):
    c = s["c"]
    if own:
        from head_attention_forward_fmha_gb300 import binding

        if c["op"] == "norm_rope":
            q, k, v = binding.fmha_qk_norm_rope(s["qkv"], s["cos_sin"], s["positions"], c["n_h"], c["n_kv_h"], q_weight=s["q_weight"],
                                                k_weight=s["k_weight"], eps=1e-6, interleaved=c["interleaved"], q=s["q"], k=s["k"], v=s["v"])
            return {"q": q, "k": k, "v": v}
        if c["op"] == "kv4_append":
            binding.fmha_kv4_append(s["k"], s["v"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["start"],
                                    k_global=c["g"], v_global=c["g"], k_out=s["k_out"], v_out=s["v_out"])
            return _appended(s)
        if c["op"] == "kv4_attend":
            o, lse = binding.fmha_fwd_kv4(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["lens"], o=s["o"], lse=s["lse"],
                                          k_global=c["g"], v_global=c["g"], window=c["window"], n_first=c["n_first"], causal=c["causal"], sink=s["sink"])
        else:
            o, lse = binding.fmha_fwd_first(s["q"], s["k"], s["v"], c["n_first"], o=s["o"], lse=s["lse"], window=c["window"], causal=c["causal"],
                                            sink=s["sink"])
        return {"o": o, "lse": lse}
    if c["op"] == "norm_rope":
        return _norm_rope(s)
    if c["op"] == "kv4_append":
        return _kv4_append(s)
    if c["op"] == "kv4_attend":
        return _attend(s, _values(s["k_codes"], s["k_scales"], c["g"]), _values(s["v_codes"], s["v_scales"], c["g"]))
    return _attend(s, s["k"].float(), s["v"].float())


# ------------------------------------------------------------------------------------------------------- 64-bit definition


def _exact_rows(codes, scales, g):
    """64-bit values of a sequence's cache, straight from the bits."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    neg = n >= 8
    n = torch.where(neg, n - 8, n)
    expo, man = torch.div(n, 2, rounding_mode="floor"), n % 2
    mag = torch.where(expo == 0, man * 0.5, (1 + man * 0.5) * torch.exp2(expo - 1))
    s = scales.double()
    expo, man = torch.div(s, 8, rounding_mode="floor"), s % 8
    s = torch.where(expo == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(expo - 7))
    return torch.where(neg, -mag, mag) * s.repeat_interleave(16, -1) * g


def _exact_quantised(x, g):
    """64-bit values of quantised rows: nearest E4M3 scale, then nearest E2M1 magnitude, ties to the even code."""
    x = x.double()
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    want = blocks.abs().amax(-1) / (6 * g)
    expo = torch.floor(torch.log2(want.clamp(min=2.0 ** -40))).clamp(min=-6, max=8)
    s = (torch.round(want / torch.exp2(expo - 3)) * torch.exp2(expo - 3)).clamp(max=448.0)
    a = blocks.abs() / torch.where(s > 0, s * g, torch.full_like(s, math.inf))[..., None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    e = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(blocks) * e * s[..., None] * g).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    b, T, hd = c["batch"], c["T"], c["hd"]
    if c["op"] == "norm_rope":
        heads = s["qkv"].double().reshape(b, T, -1, hd).permute(0, 2, 1, 3)
        half = c["rot"] // 2
        angle = s["cos_sin"].double()[s["positions"].long()].unsqueeze(1)
        turn = torch.complex(angle[..., :half], angle[..., half:])
        out = {}
        for name, lo, hi in (("q", 0, c["n_h"]), ("k", c["n_h"], c["n_h"] + c["n_kv_h"])):
            y = heads[:, lo:hi]
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / hd + 1e-6) * s[name + "_weight"].double()
            if c["interleaved"]:
                z = torch.view_as_complex(y[..., : 2 * half].reshape(*y.shape[:-1], half, 2).contiguous()) * turn
                y[..., : 2 * half] = torch.view_as_real(z).reshape(*y.shape[:-1], 2 * half)
            else:
                z = torch.complex(y[..., :half], y[..., half : 2 * half]) * turn
                y[..., :half], y[..., half : 2 * half] = z.real, z.imag
            out[name] = y
        out["v"] = heads[:, c["n_h"] + c["n_kv_h"] :]
        return out
    if c["op"] == "kv4_append":
        return {"k_out": _exact_quantised(s["k"], c["g"]), "v_out": _exact_quantised(s["v"], c["g"]),
                "k_codes": None, "k_scales": None, "v_codes": None, "v_scales": None}
    nh, nk = c["n_h"], c["n_kv_h"]
    o = torch.zeros((b, nh, T, hd), dtype=torch.float64, device=DEV)
    lse = torch.full((b, nh, T), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["lens"].tolist()):
        if c["op"] == "kv4_attend":
            k = _exact_rows(s["k_codes"][i, :, :n], s["k_scales"][i, :, :n], c["g"])
            v = _exact_rows(s["v_codes"][i, :, :n], s["v_scales"][i, :, :n], c["g"])
        else:
            k, v = s["k"][i].double(), s["v"][i].double()
        at = torch.arange(n - T, n, device=DEV)[:, None] - torch.arange(n, device=DEV)  # how far behind the row a key is
        hide = torch.zeros_like(at, dtype=torch.bool)
        if c["window"]:
            hide = at >= c["window"]
            hide[:, : c["n_first"]] = False
        if c["causal"]:
            hide |= at < 0
        for head in range(nk):
            rows = slice(head * (nh // nk), (head + 1) * (nh // nk))
            x = torch.einsum("gtd,nd->gtn", s["q"][i, rows].double(), k[head]) / math.sqrt(hd)
            x = torch.where(hide, torch.full_like(x, -math.inf), x)
            total = torch.logsumexp(x, -1)
            if s["sink"] is not None:
                total = torch.logaddexp(total, s["sink"][rows].double()[:, None].expand_as(total))
            lse[i, rows] = total
            o[i, rows] = torch.einsum("gtn,nd->gtd", torch.nan_to_num(torch.exp(x - total[..., None]), nan=0.0), v[head])
    return {"o": o, "lse": lse}
