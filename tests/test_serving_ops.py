"""The serving operators on the GPU against 64-bit plain implementations (tests/serving_ref.py,
which derives the bounds)."""
import math

import numpy as np
import pytest
import torch

import oracle
import serving_ref as ref
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    binding.fmha_check_device_status()


# ------------------------------------------------------------------ norm and rotation
def table(max_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def check_norm_rope(q, k, v, qkv, n_h, n_kv, hd, qw, kw, eps, tab, pos, inter):
    b, T = qkv.shape[:2]
    x = qkv.double().reshape(b, T, n_h + 2 * n_kv, hd).transpose(1, 2)
    cos = sin = None
    if tab is not None:
        row = tab.double()[pos.long()][:, None]
        cos, sin = row[..., : tab.shape[1] // 2], row[..., tab.shape[1] // 2 :]
    for name, got, lo, hi, w in (("q", q, 0, n_h, qw), ("k", k, n_h, n_h + n_kv, kw)):
        want, tol = ref.norm_rope(x[:, lo:hi], None if w is None else w.double(), eps, cos, sin, inter)
        off = (got.double() - want).abs() - tol
        assert (off <= 0).all(), "%s off by %.3e beyond its bound" % (name, off.max().item())
    assert torch.equal(v, x[:, n_h + n_kv :].to(torch.bfloat16))


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("b,T,n_h,n_kv,rot_of,inter,pad", [
    (1, 1, 1, 1, 1.0, False, 0), (3, 5, 6, 2, 1.0, True, 8), (2, 7, 5, 1, 0.5, False, 64), (1, 33, 8, 8, 0.375, True, 0),
    (2, 3, 3, 3, 0.25, False, 24), (4, 257, 40, 8, 1.0, False, 0), (5, 129, 64, 8, 0.5, True, 16), (2, 1, 4, 2, 0.0, False, 0)])
def test_norm_rope(hd, b, T, n_h, n_kv, rot_of, inter, pad):
    g = gen(hd + T)
    wide = normal(g, b, T, (n_h + 2 * n_kv) * hd + pad)
    qkv = wide[..., : (n_h + 2 * n_kv) * hd]
    rot = int(hd * rot_of)
    tab = table(5000, rot) if rot else None
    pos = torch.randint(0, 5000, (b, T), generator=g, device=DEV).to(torch.int32) if rot else None
    qw, kw = 1 + 0.3 * torch.randn(hd, generator=g, device=DEV), 1 + 0.3 * torch.randn(hd, generator=g, device=DEV)
    q, k, v = binding.fmha_qk_norm_rope(qkv, tab, pos, n_h, n_kv, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    check_norm_rope(q, k, v, qkv, n_h, n_kv, hd, qw, kw, 1e-5, tab, pos, inter)
    # one side without a norm
    q, k, v = binding.fmha_qk_norm_rope(qkv, tab, pos, n_h, n_kv, k_weight=kw, eps=1e-5, interleaved=inter)
    check_norm_rope(q, k, v, qkv, n_h, n_kv, hd, None, kw, 1e-5, tab, pos, inter)


def test_norm_rope_padding_and_placement():
    """Padding tokens and rows outside k and v are left as they were; sequences may lie at any stride."""
    g = gen(1)
    b, T, n_h, n_kv, hd, rows = 3, 4, 4, 2, 128, 9
    qkv = normal(g, b, 2 * T, (n_h + 2 * n_kv) * hd)[:, ::2]  # every other row: token stride twice the width
    tab = table(100, hd)
    pos = torch.tensor([[0, 1, 2, 99], [-1, 5, 100, 7], [3, 2 ** 31 - 1, -(2 ** 31), 50]], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 7, -2], dtype=torch.int32, device=DEV)
    q = torch.full((b, n_h, T, hd), 3.0, dtype=torch.bfloat16, device=DEV)
    k = torch.full((b, n_kv, rows, hd), 5.0, dtype=torch.bfloat16, device=DEV)
    v = torch.full((b, n_kv, rows, hd), 7.0, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(hd, device=DEV)
    binding.fmha_qk_norm_rope(qkv, tab, pos, n_h, n_kv, q_weight=w, k_weight=w, q=q, k=k, v=v, kv_start=start)
    safe = pos.clamp(0, 99)
    q2, k2, v2 = binding.fmha_qk_norm_rope(qkv, tab, safe, n_h, n_kv, q_weight=w, k_weight=w)
    check_norm_rope(q2, k2, v2, qkv, n_h, n_kv, hd, w, w, 1e-6, tab, safe, False)
    wq, wk, wv = torch.full_like(q, 3.0), torch.full_like(k, 5.0), torch.full_like(v, 7.0)
    for i in range(b):
        for t in range(T):
            if 0 <= int(pos[i, t]) < 100:
                wq[i, :, t] = q2[i, :, t]
                r = int(start[i]) + t
                if 0 <= r < rows:
                    wk[i, :, r], wv[i, :, r] = k2[i, :, t], v2[i, :, t]
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(v, wv)


def test_norm_rope_extremes():
    """Rows of zeros (eps carries them), tiny and huge rows; infinities stay in their own row, and out of V's way."""
    g = gen(2)
    hd = 64
    qkv = normal(g, 1, 5, 3 * hd)
    qkv[0, 0] = 0
    qkv[0, 1] *= 1e-15
    qkv[0, 2] *= 1e15
    tab, pos = table(16, 32), torch.arange(5, dtype=torch.int32, device=DEV)[None]
    w = torch.ones(hd, device=DEV)
    q, k, v = binding.fmha_qk_norm_rope(qkv, tab, pos, 1, 1, q_weight=w, k_weight=w)
    check_norm_rope(q, k, v, qkv, 1, 1, hd, w, w, 1e-6, tab, pos, False)
    for inter in (False, True):  # an infinity past the rotated columns does not reach the rest of an unnormalised row
        bad = qkv.clone()
        bad[0, 3, hd - 1] = float("inf")
        bad[0, 3, 2 * hd + 1] = float("nan")
        q, k, v = binding.fmha_qk_norm_rope(bad, tab, pos, 1, 1, interleaved=inter)
        want, tol = ref.norm_rope(qkv.double()[:, :, :hd][:, None], None, 0.0, tab.double()[pos.long()][:, None, :, :16],
                                  tab.double()[pos.long()][:, None, :, 16:], inter)
        assert ((q.double() - want).abs() <= tol)[0, 0, :, : hd - 1].all() and q[0, 0, 3, hd - 1] == float("inf")
        assert torch.isnan(v[0, 0, 3, 1]) and torch.isnan(v).sum() == 1


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("b,n_kv,T,g", [(1, 1, 1, 1.0), (3, 2, 5, 0.25), (2, 8, 33, 3.0), (7, 1, 100, 0.7)])
def test_append_matches_the_oracle_bit_for_bit(hd, b, n_kv, T, g):
    r = gen(hd + T)
    cap = 128
    k, v = normal(r, b, n_kv, T, hd) * 3, normal(r, b, n_kv, T, hd)
    k[0, 0, 0, :16] = 0
    k[0, 0, T - 1, 16:32] = float("inf")
    v[0, 0, 0, 5] = 1e30
    v[-1, 0, 0] *= 1e-30
    cache = [torch.full_like(t, 0xA5) for t in binding.fmha_kv4_cache(b, n_kv, cap, hd)]
    start = torch.randint(0, cap - T + 1, (b,), generator=r, device=DEV).to(torch.int32)
    start[0] = cap - T
    k_out, v_out = torch.zeros_like(k), torch.zeros_like(v)
    binding.fmha_kv4_append(k, v, *cache, start, k_global=g, v_global=2 * g, k_out=k_out, v_out=v_out)
    for x, codes, scales, gg, out in ((k, cache[0], cache[1], g, k_out), (v, cache[2], cache[3], 2 * g, v_out)):
        # From 448 * 6 * gg on both codes saturate, whatever the size.  The oracle compares distances in double, where
        # those of huge values to 4 and to 6 round to the same number (for an infinity they are both infinite): it is
        # asked about 10^6 in their place.
        c_ref, s_ref = oracle.quantize_nvfp4(x.float().clamp(-1e6, 1e6).cpu().numpy().reshape(-1, hd), gg)
        c_ref = torch.from_numpy(np.ascontiguousarray(c_ref)).reshape(b, n_kv, T, hd // 2)
        s_ref = torch.from_numpy(np.ascontiguousarray(s_ref)).reshape(b, n_kv, T, hd // 16)
        want_c, want_s = torch.full_like(codes.cpu(), 0xA5), torch.full_like(scales.cpu(), 0xA5)
        for i in range(b):
            at = int(start[i])
            want_c[i, :, at : at + T], want_s[i, :, at : at + T] = c_ref[i], s_ref[i]
        assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
        values = ref.dequantise(c_ref, s_ref, 1.0).float() * torch.tensor(gg, dtype=torch.float32)
        assert torch.equal(out.cpu(), values.to(torch.bfloat16))


def test_append_leaves_rows_outside_the_cache_out():
    r = gen(4)
    b, n_kv, T, cap, hd = 5, 2, 4, 32, 64
    k, v = normal(r, b, n_kv, T, hd), normal(r, b, n_kv, T, hd)
    start = torch.tensor([-2, 30, -100, 2 ** 31 - 1, 32], dtype=torch.int32, device=DEV)
    cache = [torch.full_like(t, 0x5A) for t in binding.fmha_kv4_cache(b, n_kv, cap, hd)]
    out = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    binding.fmha_kv4_append(k, v, *cache, start, k_out=out[0], v_out=out[1])
    whole = binding.fmha_kv4_cache(b, n_kv, cap, hd)
    binding.fmha_kv4_append(k, v, *whole, torch.zeros_like(start))
    for t, w in zip(cache, whole):
        want = torch.full_like(t, 0x5A)
        want[0, :, 0:2] = w[0, :, 2:4]
        want[1, :, 30:32] = w[1, :, 0:2]
        assert torch.equal(t, want)
    written = torch.zeros((b, T), dtype=torch.bool)
    written[0, 2:] = written[1, :2] = True
    for o in out:
        same = (o == 9.0).all(-1).all(1).cpu()
        assert torch.equal(same, ~written)


# ------------------------------------------------------------------ attention over the 4-bit cache
@pytest.fixture(params=[1, 2], ids=["rows8", "rows128"])
def kernel(request):
    """Both kernels of the 4-bit attention."""
    binding.fmha_set_kernel_path(request.param)
    yield
    binding.fmha_set_kernel_path(0)


def filled(r, b, n_kv, cap, hd, g=1.0):
    k, v = normal(r, b, n_kv, cap, hd), normal(r, b, n_kv, cap, hd)
    k[..., 3] *= 6
    cache = binding.fmha_kv4_cache(b, n_kv, cap, hd)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(b, dtype=torch.int32, device=DEV), k_global=g, v_global=2 * g)
    return list(cache)


def spoil(cache, lens):
    """Rows behind each sequence's end: code and scale bytes of all ones (NaN scales)."""
    for t in cache:
        for i, n in enumerate(lens):
            t[i, :, n:] = 0xFF


def check_kv4(hd, n_h, n_kv, T, cap, lens, window=0, n_first=0, causal=False, sink=False, g=1.0, kv_chunk=0, s_k=None, seed=0, scale=None,
              q_mult=1.0):
    r = gen(seed + hd)
    b = len(lens)
    cache = filled(r, b, n_kv, cap, hd, g)
    spoil(cache, lens)
    q = normal(r, b, n_h, T, hd) * q_mult
    sg = torch.randn(n_h, generator=r, device=DEV) * 2 if sink else None
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = binding.fmha_fwd_kv4(q, *cache, ln, s_k=s_k, k_global=g, v_global=2 * g, scale=scale, window=window, n_first=n_first, causal=causal,
                               sink=sg, kv_chunk=kv_chunk)
    zero = [t.clone() for t in cache]
    for t in zero:
        for i, n in enumerate(lens):
            t[i, :, n:] = 0
    want = ref.attend(q, ref.dequantise(zero[0], zero[1], g), ref.dequantise(zero[2], zero[3], 2 * g), lens,
                      hd ** -0.5 if scale is None else scale, window, n_first, causal, sg)
    ref.assert_attention(got, want, "kv4 hd %d" % hd)
    return got


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("n_h,n_kv", [(1, 1), (8, 1), (6, 2), (10, 2), (24, 1), (64, 2)])
def test_kv4_decode_lengths(hd, n_h, n_kv, kernel):
    check_kv4(hd, n_h, n_kv, 1, 352, [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 352, 351])


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("T,causal", [(2, True), (5, True), (5, False), (37, True)])
def test_kv4_more_rows(hd, T, causal, kernel):
    """Rows before their sequence's first key attend nothing (causal, T > length)."""
    check_kv4(hd, 6, 2, T, 128, [0, 1, 3, 36, 100, 128], causal=causal)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("window,n_first", [(1, 0), (1, 1), (17, 4), (64, 33), (100, 64), (300, 16), (1000, 7), (5, 200)])
@pytest.mark.parametrize("T,causal", [(1, False), (9, True), (3, False)])
def test_kv4_window_and_first_keys(hd, window, n_first, T, causal, kernel):
    check_kv4(hd, 4, 2, T, 400, [0, 4, 40, 111, 256, 400, 399], window=window, n_first=n_first, causal=causal)


@pytest.mark.parametrize("kv_chunk", [16, 32, 64, 100, 512])
@pytest.mark.parametrize("hd,window,n_first,sink", [(128, 0, 0, False), (128, 150, 40, True), (64, 0, 0, True), (256, 70, 5, False), (512, 99, 17, True)])
def test_kv4_splits(hd, kv_chunk, window, n_first, sink, kernel):
    check_kv4(hd, 8, 2, 3, 512, [0, 1, 130, 511, 512], window=window, n_first=n_first, causal=True, sink=sink, kv_chunk=kv_chunk)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_kv4_sink_scales_and_bounds(hd, kernel):
    check_kv4(hd, 8, 2, 1, 256, [0, 7, 256], sink=True, g=0.25)
    check_kv4(hd, 8, 2, 2, 256, [0, 7, 200], g=3.0, s_k=200)
    check_kv4(hd, 8, 2, 1, 256, [0, 7, 256], scale=-0.2)          # a negative scale turns the order round
    check_kv4(hd, 8, 2, 1, 256, [0, 7, 256], scale=0.0)           # every key the same weight
    check_kv4(hd, 8, 2, 2, 256, [0, 7, 256], g=2.0 ** -40, kv_chunk=64)   # tiny and huge values through partials
    check_kv4(hd, 8, 2, 2, 256, [0, 7, 256], g=2.0 ** 30, scale=2.0 ** -34, kv_chunk=64)
    check_kv4(hd, 8, 2, 1, 256, [5, 256], q_mult=2.0 ** 60, scale=2.0 ** -63)
    check_kv4(hd, 8, 2, 1, 256, [5, 256], q_mult=2.0 ** -70, scale=2.0 ** 67)


def test_kv4_lengths_beyond_bounds_are_clamped(kernel):
    r = gen(9)
    cache = filled(r, 4, 1, 128, 64)
    q = normal(r, 4, 2, 1, 64)
    given = torch.tensor([-5, 2 ** 31 - 1, 101, -(2 ** 31)], dtype=torch.int32, device=DEV)
    o, lse = binding.fmha_fwd_kv4(q, *cache, given, s_k=100)
    o2, lse2 = binding.fmha_fwd_kv4(q, *cache, torch.tensor([0, 100, 100, 0], dtype=torch.int32, device=DEV), s_k=100)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = binding.fmha_fwd_kv4(q, *cache, s_k=100)
    assert torch.equal(o3[1:3], o[1:3]) and torch.equal(lse3[1:3], lse[1:3])
    assert (o[0] == 0).all() and torch.isinf(lse[0]).all()


def test_kv4_one_dominant_key_and_rising_scores(kernel):
    """Scores that rise along the keys (the running reference moves often) and one key far above the rest."""
    hd, n = 128, 1024
    r = gen(11)
    k = normal(r, 1, 1, n, hd) * 0.1
    v = normal(r, 1, 1, n, hd)
    q = normal(r, 1, 8, 1, hd)
    q[..., 0] = 8
    k[0, 0, :, 0] = torch.linspace(0, 48, n, device=DEV).to(torch.bfloat16)
    cache = binding.fmha_kv4_cache(1, 1, n, hd)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    for chunk in (0, 1024):
        got = binding.fmha_fwd_kv4(q, *cache, kv_chunk=chunk)
        want = ref.attend(q, ref.dequantise(cache[0], cache[1], 1.0), ref.dequantise(cache[2], cache[3], 1.0), [n], hd ** -0.5)
        ref.assert_attention(got, want)


def test_kv4_long_cache_past_32_bit_offsets(kernel):
    """The last sequence's rows lie more than 2^32 bytes into the cache."""
    b, n_kv, cap, hd = 5, 8, 1 << 19, 512
    cache = [torch.zeros((b, n_kv, cap, hd // w), dtype=torch.uint8, device=DEV) for w in (2, 16, 2, 16)]
    assert cache[0].numel() > 1 << 32
    r = gen(12)
    T = 3
    k, v = normal(r, b, n_kv, T, hd), normal(r, b, n_kv, T, hd)
    start = torch.full((b,), cap - T, dtype=torch.int32, device=DEV)
    binding.fmha_kv4_append(k, v, *cache, start)
    q = normal(r, b, n_kv, 1, hd)
    o, lse = binding.fmha_fwd_kv4(q, *cache, window=T)
    small = [t[:, :, -16:].contiguous() for t in cache]
    want = ref.attend(q, ref.dequantise(small[0], small[1], 1.0), ref.dequantise(small[2], small[3], 1.0), [16] * b, hd ** -0.5, window=T)
    ref.assert_attention((o, lse), want)


# ------------------------------------------------------------------ window with first keys
@pytest.fixture
def path():
    yield binding.fmha_set_kernel_path
    binding.fmha_set_kernel_path(0)


def check_first(hd, b, n_h, n_kv, T, s_k, window, n_first, causal, sink=False, seed=0):
    r = gen(seed + hd)
    q, k, v = normal(r, b, n_h, T, hd), normal(r, b, n_kv, s_k, hd) * 2, normal(r, b, n_kv, s_k, hd)
    sg = torch.randn(n_h, generator=r, device=DEV) * 2 if sink else None
    # keys that no row attends hold NaN and infinities
    lo = max(0, s_k - T - window + 1)
    if window < s_k and n_first < lo:
        k[:, :, n_first:lo] = float("nan")
        v[:, :, n_first:lo] = float("inf")
    got = binding.fmha_fwd_first(q, k, v, n_first, window=window, causal=causal, sink=sg)
    if window < s_k and n_first < lo:
        k[:, :, n_first:lo] = 0
        v[:, :, n_first:lo] = 0
    want = ref.attend(q, k, v, [s_k] * b, hd ** -0.5, window, n_first, causal, sg, p_bits=8)
    ref.assert_attention(got, want, "first hd %d T %d s_k %d window %d n_first %d" % (hd, T, s_k, window, n_first))


@pytest.mark.parametrize("which", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("n_h,n_kv,T,s_k,window,n_first,causal,sink", [
    (8, 1, 1, 700, 200, 4, False, False), (6, 2, 1, 333, 64, 70, False, True), (4, 4, 1, 513, 1, 1, True, False),
    (4, 2, 9, 400, 100, 130, True, False), (2, 2, 33, 300, 280, 17, True, True), (16, 1, 40, 500, 37, 4, True, False),
    (8, 2, 128, 600, 150, 16, True, False), (3, 1, 100, 450, 30, 300, False, True), (4, 1, 64, 64, 5, 3, True, False),
    (2, 1, 5, 90, 90, 4, True, False), (2, 1, 5, 90, 1000, 4, False, False), (2, 1, 3, 200, 199, 200, False, False),
    (1, 1, 1, 1, 1, 4, True, False), (32, 1, 8, 1500, 900, 128, True, True)])
def test_first_keys(hd, n_h, n_kv, T, s_k, window, n_first, causal, sink, which, path):
    path(which)
    check_first(hd, 2, n_h, n_kv, T, s_k, window, n_first, causal, sink)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("T,n_first", [(1, 4), (16, 200), (128, 64)])
def test_first_keys_split(hd, T, n_first):
    """Long windows on few heads: the plan splits the key axis, the first keys among its chunks."""
    n_h = 2 if T > 1 else 8
    assert binding.fmha_fwd_first_workspace_bytes(1, n_h, 1, T, 20000, hd, 9000, n_first, True) > 0
    check_first(hd, 1, n_h, 1, T, 20000, 9000, n_first, True, sink=True)


def test_first_keys_without_any_is_the_windowed_forward():
    r = gen(50)
    q, k, v = normal(r, 2, 8, 3, 128), normal(r, 2, 2, 500, 128), normal(r, 2, 2, 500, 128)
    for window in (0, 77, 500):
        a = binding.fmha_fwd_first(q, k, v, 0, window=window, causal=True)
        b = binding.fmha_fwd(q, k, v, window=window, causal=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = binding.fmha_fwd_first(q, k, v, 9, window=0)
    b = binding.fmha_fwd(q, k, v)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_first_keys_captured_twice_on_one_stream():
    """Two graphs of split calls captured on one stream and replayed at once keep their workspaces apart."""
    r = gen(51)
    sets, graphs, st = [], [], torch.cuda.Stream()
    for i in range(2):
        q, k, v = normal(r, 1, 8, 1, 128), normal(r, 1, 1, 9000, 128), normal(r, 1, 1, 9000, 128)
        o, lse = binding.fmha_fwd_first(q, k, v, 4, window=8000)
        sets.append((q, k, v, o, lse))
    torch.cuda.synchronize()
    for q, k, v, o, lse in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            binding.fmha_fwd_first(q, k, v, 4, window=8000, o=o, lse=lse)
        graphs.append(graph)
    for s in sets:
        s[0].copy_(normal(r, 1, 8, 1, 128))
    torch.cuda.synchronize()
    lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for graph, lane in zip(graphs, lanes):
            with torch.cuda.stream(lane):
                graph.replay()
    torch.cuda.synchronize()
    for q, k, v, o, lse in sets:
        ref.assert_attention((o, lse), ref.attend(q, k, v, [9000], 128 ** -0.5, 8000, 4, p_bits=8))


# ------------------------------------------------------------------ together, streams and graphs
def step(s, stream=None):
    """One decode step: projection rows -> norm and rotation -> append -> attention."""
    q, k, v = binding.fmha_qk_norm_rope(s["qkv"], s["tab"], s["pos"], s["n_h"], s["n_kv"], q_weight=s["w"], k_weight=s["w"], q=s["q"],
                                        k=s["k"], v=s["v"], stream=stream)
    binding.fmha_kv4_append(k, v, *s["cache"], s["start"], stream=stream)
    return binding.fmha_fwd_kv4(q, *s["cache"], s["lens"], window=64, n_first=4, causal=True, o=s["o"], lse=s["lse"], stream=stream)


def state(seed, b=3, T=2, n_h=8, n_kv=2, hd=128, cap=256):
    r = gen(seed)
    lens = torch.randint(T, cap - T, (b,), generator=r, device=DEV).to(torch.int32)
    return dict(n_h=n_h, n_kv=n_kv, qkv=normal(r, b, T, (n_h + 2 * n_kv) * hd), tab=table(512, hd), w=1 + 0.1 * torch.randn(hd, generator=r, device=DEV),
                pos=(lens[:, None] - T + torch.arange(T, device=DEV)).to(torch.int32), start=(lens - T).to(torch.int32), lens=lens,
                cache=filled(r, b, n_kv, cap, hd), q=torch.empty(b, n_h, T, hd, dtype=torch.bfloat16, device=DEV),
                k=torch.empty(b, n_kv, T, hd, dtype=torch.bfloat16, device=DEV), v=torch.empty(b, n_kv, T, hd, dtype=torch.bfloat16, device=DEV),
                o=torch.empty(b, n_h, T, hd, dtype=torch.bfloat16, device=DEV), lse=torch.empty(b, n_h, T, device=DEV))


def check_step(s):
    cache = s["cache"]
    want = ref.attend(s["q"], ref.dequantise(cache[0], cache[1], 1.0), ref.dequantise(cache[2], cache[3], 1.0), s["lens"].tolist(), 128 ** -0.5,
                      window=64, n_first=4, causal=True)
    ref.assert_attention((s["o"], s["lse"]), want, "step")
    check_norm_rope(s["q"], s["k"], s["v"], s["qkv"], s["n_h"], s["n_kv"], 128, s["w"], s["w"], 1e-6, s["tab"], s["pos"], False)


def test_decode_step():
    s = state(20)
    step(s)
    check_step(s)


def test_decode_step_captured_and_replayed():
    """Two graphs captured on one stream, replayed at the same time on two others, after their inputs changed."""
    a, c = state(21), state(22)
    step(a), step(c)
    graphs, st = [], torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for s in (a, c):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step(s)
        graphs.append(graph)
    fresh = [state(23), state(24)]
    for s, f in zip((a, c), fresh):
        for n in ("qkv", "pos", "start", "lens"):
            s[n].copy_(f[n])
        s["o"].zero_()
    torch.cuda.synchronize()
    lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for graph, lane in zip(graphs, lanes):
            with torch.cuda.stream(lane):
                graph.replay()
    torch.cuda.synchronize()
    check_step(a)
    check_step(c)


def test_two_streams_at_once():
    states, lanes = [state(30 + i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, lane in zip(states, lanes):
            step(s, stream=lane)
    torch.cuda.synchronize()
    for s in states:
        check_step(s)
    with pytest.raises(TypeError):
        binding.fmha_fwd_kv4(states[0]["q"].transpose(1, 2), *states[0]["cache"])
    with pytest.raises(ValueError):
        binding.fmha_fwd_kv4(states[0]["q"], *states[0]["cache"], states[0]["lens"][:2].contiguous())


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_kv4_many_rows(hd):
    """Prompt chunks and shared heads: whole and part row tiles, the automatic choice of kernel."""
    check_kv4(hd, 16, 2, 40, 512, [0, 7, 39, 300, 512], causal=True, window=200, n_first=4)
    check_kv4(hd, 128, 1, 1, 512, [1, 511, 64], sink=True)
    check_kv4(hd, 3, 1, 100, 256, [100, 256, 30], causal=True, kv_chunk=64)


def test_threads_on_one_stream_keep_their_partials_apart():
    """Four threads run split calls on the same (default) stream at once; each checks its own results."""
    import threading

    sets = [state(60 + i, b=1, T=1, n_h=8, n_kv=1, cap=8192) for i in range(4)]
    for s in sets:
        s["lens"].fill_(8100)
    torch.cuda.synchronize()
    assert binding.fmha_fwd_kv4_plan(1, 8, 1, 1, 8192, 128)[0] > 1

    def work(s):
        for _ in range(50):
            binding.fmha_fwd_kv4(s["q"], *s["cache"], s["lens"], o=s["o"], lse=s["lse"])

    for s in sets:
        s["q"].copy_(normal(gen(70), *s["q"].shape))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(s,)) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for s in sets:
        c = s["cache"]
        ref.assert_attention((s["o"], s["lse"]), ref.attend(s["q"], ref.dequantise(c[0], c[1], 1.0), ref.dequantise(c[2], c[3], 1.0),
                                                            [8100], 128 ** -0.5))
    binding.fmha_release()
    assert not binding._workspaces


def test_kv4_same_call_twice_is_bitwise_the_same():
    r = gen(40)
    cache = filled(r, 2, 2, 4096, 128)
    q = normal(r, 2, 16, 1, 128)
    a = [t.clone() for t in binding.fmha_fwd_kv4(q, *cache)]
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    b = binding.fmha_fwd_kv4(q, *cache, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_torch_ops():
    """The custom ops run the same calls, and trace under fake tensors."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    from head_attention_forward_fmha_gb300 import torch_op  # noqa: F401  (registers them)

    r = gen(80)
    q, k, v = normal(r, 1, 8, 2, 128), normal(r, 1, 2, 400, 128), normal(r, 1, 2, 400, 128)
    a = torch.ops.fmha_gb300.fwd_first(q, k, v, 4, 128 ** -0.5, 100, True)
    b = binding.fmha_fwd_first(q, k, v, 4, window=100, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cache = filled(r, 1, 2, 256, 128)
    lens = torch.tensor([200], dtype=torch.int32, device=DEV)
    a = torch.ops.fmha_gb300.fwd_kv4(q, *cache, lens, 1.0, 2.0, 128 ** -0.5, 100, 4, True)
    b = binding.fmha_fwd_kv4(q, *cache, lens, v_global=2.0, window=100, n_first=4, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with FakeTensorMode() as mode:
        f = [mode.from_tensor(t) for t in (q, *cache, lens)]
        o, lse = torch.ops.fmha_gb300.fwd_kv4(*f, 1.0, 2.0, 128 ** -0.5, 100, 4, True)
        assert o.shape == q.shape and o.dtype == torch.bfloat16 and lse.shape == (1, 8, 2) and lse.dtype == torch.float32
        o, lse = torch.ops.fmha_gb300.fwd_first(*[mode.from_tensor(t) for t in (q, k, v)], 4, 128 ** -0.5, 100, True)
        assert o.shape == q.shape and lse.shape == (1, 8, 2)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_long_chunks_of_queries(hd):
    """More query rows than a tile holds, several times over, and odd counts."""
    check_kv4(hd, 6, 2, 301, 640, [301, 640, 5], causal=True, window=123, n_first=9)
    check_first(hd, 1, 3, 1, 301, 640, 123, 9, True, sink=True)


def test_no_rows_and_no_keys():
    r = gen(81)
    cache = filled(r, 2, 1, 64, 64)
    o, lse = binding.fmha_fwd_kv4(torch.empty(2, 4, 0, 64, dtype=torch.bfloat16, device=DEV), *cache)
    assert o.numel() == 0 and lse.numel() == 0
    empty = binding.fmha_kv4_cache(2, 1, 0, 64)
    sink = torch.tensor([1.0, -2.0, 0.5, 3.0], device=DEV)
    o, lse = binding.fmha_fwd_kv4(normal(r, 2, 4, 3, 64), *empty, sink=sink)
    assert (o == 0).all() and torch.equal(lse, sink[None, :, None].expand(2, 4, 3))
    o, lse = binding.fmha_fwd_first(normal(r, 1, 2, 2, 64), torch.empty(1, 1, 0, 64, dtype=torch.bfloat16, device=DEV),
                                    torch.empty(1, 1, 0, 64, dtype=torch.bfloat16, device=DEV), 4, window=8)
    assert (o == 0).all() and torch.isinf(lse).all()
    binding.fmha_kv4_append(*[torch.empty(2, 1, 0, 64, dtype=torch.bfloat16, device=DEV)] * 2, *cache,
                            torch.zeros(2, dtype=torch.int32, device=DEV))
    q, k, v = binding.fmha_qk_norm_rope(torch.empty(2, 0, 192, dtype=torch.bfloat16, device=DEV), None, None, 1, 1)
    assert q.shape == (2, 1, 0, 64)


@pytest.mark.parametrize("b", [2, 7, 32, 33])
def test_kv4_order_of_lengths(b, kernel):
    """Sequences in rising, falling and mixed order of length, with equal ones and empty ones; more of them than lanes."""
    rising = [3 * i for i in range(b)]
    mixed = [(37 * i) % 5 * 20 for i in range(b)]
    for lens in (rising, rising[::-1], mixed, [50] * b, [0] * b):
        check_kv4(64, 4, 2, 3, 112, lens, causal=True, window=40, n_first=2)
    check_kv4(128, 4, 1, 2, 512, [(131 * i) % 513 for i in range(b)], kv_chunk=128)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("kv_chunk", [128, 256])
def test_kv4_chunks_without_keys_are_not_read(hd, kv_chunk, kernel):
    """8 or 4 chunks, most of them empty, over a workspace of NaN: empty chunks reach no result, whatever lies there."""
    lens = [0, 1, 130, 300, 1024, 640]
    want = check_kv4(hd, 4, 2, 2, 1024, lens, sink=True, kv_chunk=kv_chunk, causal=True)
    r = gen(hd)
    cache = filled(r, len(lens), 2, 1024, hd)
    spoil(cache, lens)
    q = normal(r, len(lens), 4, 2, hd)
    sink = torch.randn(4, generator=r, device=DEV) * 2
    n, _ = binding.fmha_fwd_kv4_plan(len(lens), 4, 2, 2, 1024, hd, causal=True, kv_chunk=kv_chunk)
    assert n == 1024 // kv_chunk
    ws = torch.full((binding.fmha_workspace_bytes(len(lens), 4, 2, hd, n),), 0xFF, dtype=torch.uint8, device=DEV)
    got = binding.fmha_fwd_kv4(q, *cache, torch.tensor(lens, dtype=torch.int32, device=DEV), v_global=2.0, sink=sink, kv_chunk=kv_chunk,
                               causal=True, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
