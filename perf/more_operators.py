"""A KV cache in pages, as cases that can be timed and compared.

Three operators, in the order in which a serving loop runs them on a batch of sequences that share a pool of pages:

  append   new K and V rows go to each sequence's next positions, through its row of the block table: as bf16, or in 8 bits
           (E4M3 codes under a power of two per row and head).
  gather   rows of a sequence come back as contiguous bf16 K and V, from either kind of page.
  attend   attention of each sequence's new tokens (one, a chunk of a prompt, or of every length in one batch) over its pages.

A page holds `page` rows of every K/V head: K and V pages are [n_pages, n_kv_h, page, hd], scale bytes [n_pages, n_kv_h, page]
(a byte e stands for 2^(e - 127)).  Row p of a sequence lies in page block_table[b, p // page], row p % page; an entry
outside the pool is a page that is not there.  New tokens come as [b, heads, T, hd], T for every sequence, or as
[total, heads, hd] with the sequences' bounds cu_q.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: this repository's entry points.
"""
import math

import torch

own = False

DEV = "cuda"

# ---------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # the new token of each sequence of a decode batch goes into the cache: the smallest call of a step
        dict(name="append decode batch, 8 bits", op="append", batch=32, T=1, ragged_q=False, n_kv_h=8, hd=128, page=16, cap=8192, bits=8),
        # prompts of different lengths go into the cache, straight from the rows of a QKV projection
        dict(name="append ragged prompts, 8 bits", op="append", batch=4, T=4095, ragged_q=True, n_kv_h=8, hd=128, page=64, cap=8192, bits=8),
        # prompts of one length, as they are
        dict(name="append prompts, bf16", op="append", batch=4, T=4095, ragged_q=False, n_kv_h=8, hd=128, page=16, cap=8192, bits=16),
        # a short prefix of one sequence comes back for a call that wants contiguous rows
        dict(name="gather one prefix, bf16", op="gather", batch=1, rows=513, n_kv_h=8, hd=64, page=16, cap=4096, bits=16),
        # whole sequences come back from 8 bits
        dict(name="gather sequences, 8 bits", op="gather", batch=8, rows=8192, n_kv_h=8, hd=128, page=32, cap=8192, bits=8),
        # one user's decode step over some thousand tokens: latency counts
        dict(name="attend one user", op="attend", batch=1, n_h=64, n_kv_h=8, T=1, ragged_q=False, cap=8192, hd=128, page=16, bits=16, window=0, n_first=0, causal=True, sink=False, ragged=False),
        # a decode batch of sequences of very different lengths, up to 32768 tokens
        dict(name="attend decode batch, 8 bits", op="attend", batch=32, n_h=64, n_kv_h=8, T=1, ragged_q=False, cap=32768, hd=128, page=64, bits=8, window=0, n_first=0, causal=True, sink=False, ragged=True),
        # the sliding-window decode batch: pages behind the window are given back, the first four tokens stay
        dict(name="attend windowed decode batch", op="attend", batch=32, n_h=64, n_kv_h=8, T=1, ragged_q=False, cap=8192, hd=128, page=16, bits=16, window=4096, n_first=4, causal=True, sink=True, ragged=False),
        # one K/V head of 512 columns shared by 128 query heads
        dict(name="attend shared head, 8 bits", op="attend", batch=16, n_h=128, n_kv_h=1, T=1, ragged_q=False, cap=4096, hd=512, page=64, bits=8, window=0, n_first=0, causal=True, sink=False, ragged=True),
        # a chunk of 512 new tokens of each prompt, over what the cache holds already
        dict(name="attend prompt chunks", op="attend", batch=4, n_h=64, n_kv_h=8, T=512, ragged_q=False, cap=8192, hd=128, page=16, bits=16, window=0, n_first=0, causal=True, sink=False, ragged=True),
        # one batch of decode steps and chunks of every length, from pages of 8 bits
        dict(name="attend mixed batch, 8 bits", op="attend", batch=16, n_h=32, n_kv_h=8, T=512, ragged_q=True, pad=3, cap=8192, hd=128, page=32, bits=8, window=0, n_first=0, causal=True, sink=False, ragged=True),
        # a long chunk of one sequence with wide heads
        dict(name="attend long chunk, wide heads", op="attend", batch=1, n_h=32, n_kv_h=4, T=2047, ragged_q=False, cap=8192, hd=256, page=128, bits=16, window=0, n_first=0, causal=True, sink=False, ragged=False),
    ]


# (n_h, n_kv_h): every head its own K/V, groups (odd ones too), one shared K/V head
HEADS = [(1, 1), (16, 16), (32, 32), (64, 8), (32, 8), (40, 8), (12, 4), (6, 2), (128, 1), (5, 1), (24, 3)]
HD = [64, 128, 128, 256, 512]
PAGES = [16, 16, 32, 64, 128, 256]


def _log(rng, lo, hi):
    """An integer spread over [lo, hi] by its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["append", "gather", "attend", "attend", "attend"])
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    while True:
        n_h, n_kv_h = rng.choice(HEADS)
        page = rng.choice(PAGES)
        c = dict(op=op, batch=_log(rng, 1, 64), n_h=n_h, n_kv_h=n_kv_h, hd=rng.choice(HD), page=page, bits=rng.choice([8, 16]))
        c["cap"] = page * max(1, _log(rng, 64, 32768) // page)
        if op == "append":
            del c["n_h"]
            T = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
            c.update(T=T, ragged_q=T > 1 and rng.random() < 0.5)
        elif op == "gather":
            del c["n_h"]
            c.update(rows=_log(rng, 1, c["cap"]))
        else:
            T = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
            windowed = rng.random() < 0.4
            c.update(T=T, ragged_q=T > 1 and rng.random() < 0.5, pad=rng.choice([0, 0, 1, 9]), window=_log(rng, 16, 8192) if windowed else 0,
                     n_first=rng.choice([0, 1, 4, 7, 64]) if windowed else 0, causal=T == 1 or rng.random() < 0.9,
                     sink=rng.random() < 0.25, ragged=rng.random() < 0.7)
        w = work(c)
        if w["bytes"] > top[op][0] or w["flops"] > top[op][1]:
            continue
        if c.get("T", c.get("rows", 1)) > c["cap"] or c["batch"] * n_kv_h * c["cap"] * c["hd"] > 1 << 30:
            continue
        if op == "attend" and c["batch"] * n_h * c["T"] * c["cap"] > 1 << 31:  # what the plain form holds in 32 bits
            continue
        return c


# ----------------------------------------------------------------------------------------------------------- lengths, work


def _new_tokens(c):
    """The sequences' numbers of new tokens, in rising order.  Ragged: spread over [1, T] by their logarithm, the last one T and
    (of three or more) the first one 1."""
    b, T = c["batch"], c["T"]
    if not c["ragged_q"]:
        return [T] * b
    new = [max(1, min(T, int((T + 1.0) ** ((i + 0.5) / b)))) for i in range(b)]
    new[-1] = T
    if b > 2:
        new[0] = 1
    return new


def _lens(c, seed, new):
    """The sequences' lengths, new tokens included, on the host.  Ragged: spread over the cache, one of them all new."""
    if not c["ragged"]:
        return [c["cap"] - (1 if c["cap"] > c["T"] else 0)] * c["batch"]
    g = torch.Generator().manual_seed(seed + 77)
    u = torch.rand(c["batch"], generator=g).tolist()
    lens = [n + int(x * (c["cap"] - n + 0.999)) for x, n in zip(u, new)]
    if c["batch"] > 2:
        lens[1] = new[1]
    return lens


def _visible(n, T, c):
    """(keys that some row of a sequence of n keys and T new tokens attends, pairs of rows and keys)."""
    pairs, lo = 0, n
    for t in sorted({0, T - 1}):
        p = n - T + t
        hi = min(n, p + 1) if c["causal"] else n
        first = max(0, p - c["window"] + 1) if c["window"] > 0 else 0
        lo = min(lo, first)
        got = max(0, hi - first) + (min(c["n_first"], first, max(0, hi)) if c["window"] > 0 else 0)
        pairs += got * T / (2.0 if T > 1 else 1.0)
    return max(0, n - lo) + (min(c["n_first"], lo) if c["window"] > 0 else 0), pairs


def work(c):
    # lengths that a seed spreads count by what they are expected to be
    stored = c["hd"] + 1.0 if c["bits"] == 8 else 2.0 * c["hd"]  # bytes of a row of one head
    if c["op"] == "gather":
        rows = 2.0 * c["batch"] * c["n_kv_h"] * c["rows"]
        return {"bytes": rows * (stored + 2.0 * c["hd"]), "flops": rows * c["hd"]}
    new = _new_tokens(c)
    tokens = sum(new)
    if c["op"] == "append":
        rows = 2.0 * tokens * c["n_kv_h"]
        return {"bytes": rows * (stored + 2.0 * c["hd"]) + 4.0 * c["batch"], "flops": 3.0 * rows * c["hd"]}
    seen = [_visible((T + c["cap"]) / 2.0 if c["ragged"] else c["cap"] - 1, T, c) for T in new]
    keys, pairs = sum(x[0] for x in seen), sum(x[1] for x in seen)
    rows = tokens * c["n_h"]
    return {"bytes": keys * c["n_kv_h"] * 2.0 * stored + rows * (4.0 * c["hd"] + 4), "flops": 4.0 * pairs * c["n_h"] * c["hd"]}


# ---------------------------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _key_gain(gen, heads, hd):
    """Channels of K: a few several times as large as the others, as trained models have them."""
    return 1.0 + 3.0 * (torch.rand((heads, 1, hd), generator=gen, device=DEV) > 0.96)


def _table(c, seed, lens):
    """(number of pages, block table): each sequence's pages anywhere in the pool, -1 behind its end."""
    page, width = c["page"], c["cap"] // c["page"]
    need = [-(-n // page) for n in lens]
    total = c["batch"] * width + 3
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 5)).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(order[at : at + n] + [-1] * (width - n))
        at += n
    return total, rows


def _given_back(rows, c, lens, new):
    """The pages of a windowed sequence that no row attends any more are given back."""
    for row, n, T in zip(rows, lens, new):
        first = n - T - c["window"] + 1
        for i in range(-(-c["n_first"] // c["page"]), len(row)):
            if (i + 1) * c["page"] <= first:
                row[i] = -1


def _to_pages(gen, c, total, gain):
    """A pool of pages that earlier tokens have filled: (pages, scale bytes or None)."""
    shape = (c["n_kv_h"], c["page"], c["hd"])
    pages = torch.empty((total, *shape), dtype=torch.uint8 if c["bits"] == 8 else torch.bfloat16, device=DEV)
    scales = torch.empty((total, *shape[:2]), dtype=torch.uint8, device=DEV) if c["bits"] == 8 else None
    step = max(1, (1 << 26) // (shape[0] * shape[1] * shape[2]))
    for i in range(0, total, step):
        x = _normal(gen, min(step, total - i), *shape)
        x = (x if gain is None else x * gain).to(torch.bfloat16)
        if scales is None:
            pages[i : i + step] = x
        else:
            pages[i : i + step], scales[i : i + step] = _quantise(x)
    return pages, scales


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    b, hk, hd, page = c["batch"], c["n_kv_h"], c["hd"], c["page"]
    s = {"c": c}
    if c["op"] == "gather":
        lens = [c["rows"]] * b
    else:
        new = _new_tokens(c)
        order = torch.randperm(b, generator=torch.Generator().manual_seed(seed + 33)).tolist()
        new = [new[i] for i in order]
        s["new"], s["most"] = new, max(new)
        if c["ragged_q"]:
            at = [0]
            for n in new:
                at.append(at[-1] + n)
            s["total"] = at[-1] + c.get("pad", 0)  # rows behind the last sequence are no tokens
            s["cu_q"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        if c["op"] == "append":
            g = torch.Generator().manual_seed(seed + 77)
            start = [int(x * (c["cap"] - n + 0.999)) for x, n in zip(torch.rand(b, generator=g).tolist(), new)]
            s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
            lens = [x + n for x, n in zip(start, new)]
        else:
            lens = _lens(c, seed, new)
    total, rows = _table(c, seed, lens)
    if c["op"] == "attend" and c["window"] > 0:
        _given_back(rows, c, lens, new)
    s["block_table"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["host_lens"] = lens
    gain = _key_gain(gen, hk, hd)
    s["k_scales"] = s["v_scales"] = None
    if c["op"] == "append":
        if c["ragged_q"]:  # K and V rows lie in the rows of a projection, behind the query heads
            wide = _normal(gen, s["total"], 4 * hk, hd)
            wide[:, 2 * hk : 3 * hk] *= gain.transpose(0, 1)
            wide = wide.to(torch.bfloat16)
            s["k"], s["v"] = wide[:, 2 * hk : 3 * hk], wide[:, 3 * hk :]
        else:
            s["k"] = (_normal(gen, b, hk, c["T"], hd) * gain).to(torch.bfloat16)
            s["v"] = _normal(gen, b, hk, c["T"], hd).to(torch.bfloat16)
        for name in ("k", "v"):
            s[name + "_pages"] = torch.zeros((total, hk, page, hd), dtype=torch.uint8 if c["bits"] == 8 else torch.bfloat16, device=DEV)
            if c["bits"] == 8:
                s[name + "_scales"] = torch.zeros((total, hk, page), dtype=torch.uint8, device=DEV)
        return s
    s["k_pages"], s["k_scales"] = _to_pages(gen, c, total, gain)
    s["v_pages"], s["v_scales"] = _to_pages(gen, c, total, None)
    if c["op"] == "gather":
        s["k"] = torch.zeros((b, hk, c["rows"], hd), dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.zeros_like(s["k"])
        return s
    shape = (s["total"], c["n_h"], hd) if c["ragged_q"] else (b, c["n_h"], c["T"], hd)
    s["q"] = _normal(gen, *shape).to(torch.bfloat16)
    s["o"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(shape[:-1], dtype=torch.float32, device=DEV)
    s["sink"] = _normal(gen, c["n_h"]) if c["sink"] else None
    return s


# ------------------------------------------------------------------------------------------------------------ plain forms


def _quantise(x):
    """(E4M3 codes as bytes, scale bytes) of bf16 rows: the smallest power of two that brings a row's largest value to 448 or less."""
    y = x.float()
    most = y.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(most)
    e = e - 9 + (m > 0.875).to(e.dtype)  # 448 = 0.875 * 2^9
    e = torch.where(most > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    return torch.ldexp(y, -e).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8).squeeze(-1)


def _values(rows, scales):
    """fp32 rows from bf16 rows, or from codes and scale bytes."""
    if scales is None:
        return rows.float()
    return torch.ldexp(rows.view(torch.float8_e4m3fn).float(), (scales.int() - 127)[..., None])


def _append(s):
    c = s["c"]
    if c["ragged_q"]:
        seq = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["cu_q"].diff().long(), output_size=s["total"])
        pos = s["start"].long()[seq] + torch.arange(s["total"], device=DEV) - s["cu_q"].long()[seq]
    else:
        seq = torch.arange(c["batch"], device=DEV)[:, None].expand(-1, c["T"])
        pos = s["start"].long()[:, None] + torch.arange(c["T"], device=DEV)
    page, row = s["block_table"].long()[seq, pos // c["page"]], pos % c["page"]
    for name in ("k", "v"):
        x = s[name] if c["ragged_q"] else s[name].transpose(1, 2)
        if c["bits"] == 8:
            x, scale = _quantise(x)
            s[name + "_scales"][page, :, row] = scale
        s[name + "_pages"][page, :, row] = x
    return _appended(s)


def _appended(s):
    if s["c"]["bits"] == 16:
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"k_codes": s["k_pages"].view(torch.float8_e4m3fn), "v_codes": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _gather(s):
    c = s["c"]
    pos = torch.arange(c["rows"], device=DEV)
    page, row = s["block_table"].long()[:, pos // c["page"]], pos % c["page"]  # [b, rows]
    there = ((page >= 0) & (pos < s["lens"].long()[:, None]))[:, None, :, None]
    page = page.clamp(min=0)
    for name in ("k", "v"):
        scales = s[name + "_scales"]
        x = _values(s[name + "_pages"][page, :, row], None if scales is None else scales[page, :, row])
        s[name].copy_(torch.where(there, x.transpose(1, 2).to(torch.bfloat16), s[name]))
    return {"k": s["k"], "v": s["v"]}


def _paged_rows(s, name):
    """fp32 [b, n_kv_h, keys, hd]: every row of the block table's pages."""
    at = s["block_table"].long().clamp(min=0)
    scales = s[name + "_scales"]
    x = _values(s[name + "_pages"][at], None if scales is None else scales[at])
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s):
    c, q = s["c"], s["q"]
    b, nh, hk, hd, T, n = c["batch"], c["n_h"], c["n_kv_h"], c["hd"], s["most"], c["cap"]
    new = s["cu_q"].long().diff() if c["ragged_q"] else torch.full((b,), T, device=DEV)
    if c["ragged_q"]:
        at = s["cu_q"].long()[:-1, None] + torch.arange(T, device=DEV)
        at = torch.where(torch.arange(T, device=DEV) < new[:, None], at, s["total"])  # one row more takes what is no token
        q = torch.cat([q, torch.zeros_like(q[:1])])[at].transpose(1, 2)
    j = torch.arange(n, device=DEV)[None, None]
    p = (s["lens"].long() - new)[:, None, None] + torch.arange(T, device=DEV)[:, None]
    seen = (j < s["lens"].long()[:, None, None]) & (s["block_table"] >= 0).repeat_interleave(c["page"], 1)[:, None]
    if c["causal"]:
        seen = seen & (j <= p)
    if c["window"] > 0:
        seen = seen & ((j > p - c["window"]) | (j < c["n_first"]))
    k, v = _paged_rows(s, "k"), _paged_rows(s, "v")
    x = (q.float().reshape(b, hk, nh // hk * T, hd) @ k.transpose(-1, -2)).mul_(hd ** -0.5)
    x = x.view(b, hk, nh // hk, T, n).masked_fill_(~seen.view(b, 1, 1, -1, n), -math.inf)
    top = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        extra = s["sink"].view(1, hk, nh // hk, 1, 1)
        top = torch.maximum(top, extra)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = x.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(extra - top)
    o = (w.flatten(2, 3) @ v).view(b, hk, nh // hk, T, hd)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(b, nh, T, hd)
    lse = (top + torch.log(total)).reshape(b, nh, T)
    if c["ragged_q"]:
        out = torch.cat([s["o"], s["o"][:1]])
        out[at] = o.transpose(1, 2).to(torch.bfloat16)
        s["o"].copy_(out[:-1])
        out = torch.cat([s["lse"], s["lse"][:1]])
        out[at] = lse.transpose(1, 2)
        s["lse"].copy_(out[:-1])
    else:
        s["o"].copy_(o)
        s["lse"].copy_(lse)
    return {"o": s["o"], "lse": s["lse"]}


def run(s):
    c = s["c"]
    if own:
        from head_attention_forward_fmha_gb300 import binding

        cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if c["op"] == "append":
            binding.fmha_paged_append(s["k"], s["v"], *cache, s["block_table"], s["start"], cu_q=s.get("cu_q"))
            return _appended(s)
        if c["op"] == "gather":
            k, v = binding.fmha_paged_gather(*cache, s["block_table"], s["lens"], c["rows"], k=s["k"], v=s["v"])
            return {"k": k, "v": v}
        o, lse = binding.fmha_fwd_paged(s["q"], *cache, s["block_table"], s["lens"], cu_q=s.get("cu_q"), max_q=s["most"], o=s["o"], lse=s["lse"],
                                        window=c["window"], n_first=c["n_first"], causal=c["causal"], sink=s["sink"])
        return {"o": o, "lse": lse}
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "gather":
        return _gather(s)
    return _attend(s)


# ------------------------------------------------------------------------------------------------------- 64-bit definition


def _exact_codes(x):
    """(64-bit values of the E4M3 codes, 64-bit scales) of rows: nearest code, ties to the even one, under the row's power of two."""
    x = x.double()
    most = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((most / 448.0).clamp(min=2.0 ** -127)))
    e = torch.where(most > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(most <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-127.0)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e)


def _exact_rows(s, name, i, n):
    """64-bit K or V rows [n_kv_h, n, hd] of sequence i, straight from the bits of its pages; NaN where there is no page."""
    c = s["c"]
    pages = s[name + "_pages"]
    out = torch.full((c["n_kv_h"], n, c["hd"]), math.nan, dtype=torch.float64, device=DEV)
    for slot, at in enumerate(s["block_table"][i].tolist()):
        lo, hi = slot * c["page"], min(n, (slot + 1) * c["page"])
        if at < 0 or hi <= lo:
            continue
        if c["bits"] == 16:
            out[:, lo:hi] = pages[at, :, : hi - lo].double()
            continue
        code = pages[at, :, : hi - lo].long()
        expo, man = (code >> 3) & 15, (code & 7).double()
        mag = torch.where(expo == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(expo.double() - 10))
        scale = torch.exp2(s[name + "_scales"][at, :, : hi - lo].double() - 127)
        out[:, lo:hi] = torch.where(code >= 128, -mag, mag) * scale[..., None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    b, page = c["batch"], c["page"]
    if c["op"] == "gather":
        return {n: torch.stack([_exact_rows(s, n, i, c["rows"]) for i in range(b)]) for n in ("k", "v")}
    if c["op"] == "append":
        out = {}
        for name in ("k", "v"):
            pages = torch.zeros(s[name + "_pages"].shape, dtype=torch.float64, device=DEV)
            first = 0
            for i, (n, at) in enumerate(zip(s["new"], s["start"].tolist())):
                rows = s[name][first : first + n].transpose(0, 1) if c["ragged_q"] else s[name][i]
                first += n
                rows = rows.double() if c["bits"] == 16 else _exact_codes(rows)[0]
                table = s["block_table"][i].tolist()
                done = 0
                while done < n:
                    slot, off = divmod(at + done, page)
                    take = min(page - off, n - done)
                    pages[table[slot], :, off : off + take] = rows[:, done : done + take]
                    done += take
            out[name + ("_pages" if c["bits"] == 16 else "_codes")] = pages
            if c["bits"] == 8:
                out[name + "_scales"] = None
        return out
    nh, hk = c["n_h"], c["n_kv_h"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for i, (n, T) in enumerate(zip(s["host_lens"], s["new"])):
        k, v = _exact_rows(s, "k", i, n), _exact_rows(s, "v", i, n)
        behind = torch.arange(n - T, n, device=DEV)[:, None] - torch.arange(n, device=DEV)  # how far behind the row a key is
        hide = torch.zeros_like(behind, dtype=torch.bool)
        if c["window"]:
            hide = behind >= c["window"]
            hide[:, : c["n_first"]] = False
        if c["causal"]:
            hide |= behind < 0
        hide |= torch.isnan(k[0, :, 0])
        q = s["q"][first : first + T].transpose(0, 1) if c["ragged_q"] else s["q"][i]
        for head in range(hk):
            rows = slice(head * (nh // hk), (head + 1) * (nh // hk))
            x = torch.einsum("gtd,nd->gtn", q[rows].double(), torch.nan_to_num(k[head])) / math.sqrt(c["hd"])
            x = x.masked_fill(hide, -math.inf)
            whole = torch.logsumexp(x, -1)
            if s["sink"] is not None:
                whole = torch.logaddexp(whole, s["sink"][rows].double()[:, None].expand_as(whole))
            y = torch.einsum("gtn,nd->gtd", torch.nan_to_num(torch.exp(x - whole[..., None]), nan=0.0), torch.nan_to_num(v[head]))
            if c["ragged_q"]:
                o[first : first + T, rows], lse[first : first + T, rows] = y.transpose(0, 1), whole.transpose(0, 1)
            else:
                o[i, rows], lse[i, rows] = y, whole
        first += T
    return {"o": o, "lse": lse}
