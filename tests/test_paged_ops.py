"""The cache in pages on the GPU against 64-bit plain implementations (tests/paged_ref.py, which derives the bounds)."""
import math

import pytest
import torch

import paged_ref as ref
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [torch.bfloat16, torch.float8_e4m3fn]
HD = [64, 128, 256, 512]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    binding.fmha_check_device_status()


@pytest.fixture(params=[1, 2], ids=["rows8", "rows128"])
def kernel(request):
    """Both kernels of the attention."""
    binding.fmha_set_kernel_path(request.param)
    yield
    binding.fmha_set_kernel_path(0)


def blank(n_pages, n_kv, page, hd, form):
    """A pool in which nothing is written: every byte all ones (NaN rows, NaN scales)."""
    cache = list(binding.fmha_paged_cache(n_pages, n_kv, page, hd, dtype=form))
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(0xFF)
    return cache


def pool(g, lens, n_kv, page, hd, form, width=None, spare=3, k_mult=1.0):
    """(cache, block table) of sequences that have lens[i] rows on pages in random order; whatever else the pool holds is NaN."""
    need = [-(-n // page) for n in lens]
    width = max(need + [1]) if width is None else width
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at : at + n] + [-1] * (width - n))
        at += n
    cache, table = blank(sum(need) + spare, n_kv, page, hd, form), ints(table)
    total = sum(lens)
    k, v = normal(g, total, n_kv, hd) * k_mult, normal(g, total, n_kv, hd)
    k[..., 3] *= 6
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    binding.fmha_paged_append(k, v, *cache, table, ints([0] * len(lens)), cu_q=ints(cu))
    return cache, table


def check(g, hd, n_h, n_kv, T, lens, page, form, new=None, pad=(0, 0), window=0, n_first=0, causal=False, sink=False, n_splits=0, s_k=None,
          scale=None, q_mult=1.0, k_mult=1.0, gone=None, max_q=None):
    """new: ragged new tokens (with pad[0] rows before and pad[1] behind); gone: a function of the table that takes pages away."""
    cache, table = pool(g, lens, n_kv, page, hd, form, k_mult=k_mult)
    if gone:
        gone(table)
    sg = torch.randn(n_h, generator=g, device=DEV) * 2 if sink else None
    cu = None
    if new is None:
        q = normal(g, len(lens), n_h, T, hd) * q_mult
    else:
        cu = [pad[0] + sum(new[:i]) for i in range(len(new) + 1)]
        q = normal(g, cu[-1] + pad[1], n_h, hd) * q_mult
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device=DEV)
    binding.fmha_fwd_paged(q, *cache, table, ints(lens), cu_q=None if cu is None else ints(cu), max_q=max_q, o=o, lse=lse, s_k=s_k, scale=scale,
                           window=window, n_first=n_first, causal=causal, sink=sg, n_splits=n_splits)
    want = ref.attend(q, cache, table, lens, page, cu, scale, window, n_first, causal, sg)
    if cu is not None:
        for a, b in ((0, cu[0]), (cu[-1], q.shape[0])):
            assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
            o[a:b], lse[a:b] = 0, 0
    ref.assert_attention((o, lse), want, "hd %d page %d %s" % (hd, page, form))


# ------------------------------------------------------------------ append
def special_rows(hd):
    """Rows at the ends of the number range."""
    rows = torch.zeros(16, hd)
    rows[1, 5] = 448.0                       # the largest that 2^0 holds
    rows[2, 5] = -450.0                      # the next bf16 above it
    rows[3] = torch.linspace(-3e38, 3e38, hd)
    rows[4, 0] = 9.2e-41                     # the smallest bf16
    rows[5] = torch.linspace(-1e-38, 1e-38, hd)
    rows[6, 1], rows[6, 2] = float("nan"), 1.0
    rows[7, 3], rows[7, 4] = -float("inf"), 2.0
    rows[8] = 2.0 ** -133
    rows[9] = torch.arange(hd) * 2.0 ** -9 / 4   # halves of the smallest codes: ties
    rows[9, -1] = 448.0
    rows[10] = torch.arange(hd).float() - hd / 2
    rows[11] = -0.0
    rows[12, 0], rows[12, 1] = 3.3e38, 1e-3
    rows[13, 7] = 1.75 * 2.0 ** -119         # the largest that 2^-127 holds
    rows[14, 7] = 1.7578125 * 2.0 ** -119
    rows[15] = torch.tensor([17.0, 19.0, 21.0, 23.0] * (hd // 4))   # between neighbouring codes
    rows[15, 0] = 447.0
    return rows.to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("hd", HD)
def test_append_codes_are_the_definitions(hd):
    g = gen(hd)
    k, v = normal(g, 40, 2, hd), (normal(g, 40, 2, hd) * 2.0 ** torch.randint(-60, 60, (40, 2, 1), generator=g, device=DEV)).to(torch.bfloat16)
    k[:16, 1], v[16:32, 0] = special_rows(hd), special_rows(hd)
    cache = blank(4, 2, 16, hd, FORMS[1])
    binding.fmha_paged_append(k, v, *cache, ints([[2, 0, 3]]), ints([3]), cu_q=ints([0, 40]))
    got = binding.fmha_paged_gather(*cache, ints([[2, 0, 3]]), ints([43]), 40, start=ints([3]))
    for x, pages, scales, back in ((k, cache[0], cache[2], got[0]), (v, cache[1], cache[3], got[1])):
        codes, byte = ref.quantise(x)
        want_c, want_s = torch.full(pages.shape, 0xFF, dtype=torch.uint8), torch.full(scales.shape, 0xFF, dtype=torch.uint8)
        for t in range(40):
            p, r = (2, 0, 3)[(t + 3) // 16], (t + 3) % 16
            want_c[p, :, r], want_s[p, :, r] = codes[t], byte[t]
        assert torch.equal(scales.cpu(), want_s) and torch.equal(pages.cpu(), want_c)
        want = ref.values(codes, byte).to(torch.bfloat16)
        fine = ~torch.isnan(want)
        back = back[0].transpose(0, 1).cpu()
        assert torch.equal(torch.isnan(back), ~fine) and torch.equal(back[fine], want[fine])
        # what a row stands for is off by half a code step at most
        exact = x.double().cpu()
        off = (ref.values(codes, byte) - exact).abs()
        tol = exact.abs() * 2.0 ** -4 + (torch.exp2(byte.double() - 127) * 2.0 ** -10)[..., None]
        ok = torch.isfinite(exact).all(-1, keepdim=True).expand_as(off)
        assert (off <= tol)[ok].all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("heads,page,T", [(1, 16, 1), (3, 16, 37), (8, 64, 5), (2, 256, 130)])
def test_append_uniform_and_ragged_write_the_same_rows(hd, heads, page, T, form):
    """[b, heads, T, hd], strided or not, and token rows of a projection: the same pages; rows outside are left out."""
    g = gen(hd + T)
    b, width = 5, -(-2 * T // page) + 1
    wide = normal(g, b, T, 3 * heads + 1, hd)   # q, k, v heads and padding
    k, v = wide[:, :, heads : 2 * heads], wide[:, :, 2 * heads : 3 * heads]
    table = torch.randperm(b * width, generator=g, device=DEV).reshape(b, width).to(torch.int32)
    start = ints([0, -2, width * page - 1, 7, 2 ** 31 - 1])
    table[3, 0] = -1                            # a page that is not there
    table[0, 0] = b * width + 5                 # nor is this one
    pools = [blank(b * width, heads, page, hd, form) for _ in range(4)]
    binding.fmha_paged_append(k.transpose(1, 2), v.transpose(1, 2), *pools[0], table, start)
    binding.fmha_paged_append(k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), *pools[1], table, start)
    flat = wide.reshape(b * T, 3 * heads + 1, hd)
    rows = flat[:, heads : 2 * heads], flat[:, 2 * heads : 3 * heads]
    binding.fmha_paged_append(*rows, *pools[2], table, start, cu_q=ints([i * T for i in range(b + 1)]))
    # with padding before and behind
    more = torch.cat([normal(g, 3, *flat.shape[1:]), flat, normal(g, 9, *flat.shape[1:])])
    binding.fmha_paged_append(more[:, heads : 2 * heads], more[:, 2 * heads : 3 * heads], *pools[3], table, start, cu_q=ints([3 + i * T for i in range(b + 1)]))
    want = [t.clone() if t is not None else None for t in blank(b * width, heads, page, hd, form)]
    for x, i in ((k, 0), (v, 1)):
        stored, scale = (x, None) if form == FORMS[0] else ref.quantise(x)
        for s in range(b):
            for t in range(T):
                pos = int(start[s]) + t
                p = int(table[s, pos // page]) if 0 <= pos < width * page else -1
                if 0 <= p < b * width:
                    want[i][p, :, pos % page] = stored[s, t].to(DEV)
                    if scale is not None:
                        want[2 + i][p, :, pos % page] = scale[s, t].to(DEV)
    for got in pools:
        for a, w in zip(got, want):
            assert (a is None and w is None) or torch.equal(a.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("b", [1, 31, 33, 70])
def test_append_and_attend_of_many_ragged_sequences(b):
    """More sequences than a warp has lanes, some without a token."""
    g = gen(b)
    new = [(i * 7) % 4 for i in range(b)]
    lens = [n + (i * 13) % 40 for i, n in enumerate(new)]
    for form in FORMS:
        check(g, 64, 4, 2, 0, lens, 16, form, new=new, pad=(2, 5), causal=True, max_q=3)
        check(g, 64, 12, 1, 0, lens, 32, form, new=[n * 9 for n in new], pad=(0, 1), causal=True)


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("heads,page,rows", [(1, 16, 1), (2, 16, 50), (3, 128, 300)])
def test_gather(hd, heads, page, rows, form):
    g = gen(rows)
    lens = [0, 1, rows, rows + 20, 17]
    cache, table = pool(g, lens, heads, page, hd, form)
    table[3, 0] = -7
    for start in (None, [0, 0, 3, rows, -4]):
        k, v = (torch.full((5, heads, rows, hd), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        binding.fmha_paged_gather(*cache, table, ints(lens), rows, start=None if start is None else ints(start), k=k, v=v)
        for got, pages, scales in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
            want = torch.full_like(got, 7.0)
            for i, n in enumerate(lens):
                x, there = ref.sequence(pages, scales, table[i], n, page)
                for r in range(rows):
                    pos = r + (0 if start is None else start[i])
                    if 0 <= pos < n and there[pos]:
                        want[i, :, r] = x[:, pos].to(torch.bfloat16)
            assert torch.equal(got, want)
    k, v = binding.fmha_paged_gather(*cache, table, ints(lens), rows)
    assert (k[0] == 0).all() and (v[0] == 0).all()


# ------------------------------------------------------------------ attention
LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 129, 352, 351]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("n_h,n_kv,page", [(1, 1, 16), (8, 1, 32), (6, 2, 64), (10, 2, 16), (24, 1, 256), (64, 2, 16)])
def test_decode_lengths(hd, n_h, n_kv, page, form, kernel):
    check(gen(hd), hd, n_h, n_kv, 1, LENS, page, form)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("T,causal,page", [(2, True, 16), (5, True, 64), (5, False, 16), (37, True, 32), (150, True, 16)])
def test_more_rows(hd, T, causal, page, form, kernel):
    """Rows before their sequence's first key attend nothing (causal, T above the length)."""
    check(gen(T), hd, 6, 2, T, [0, 1, 3, 36, 100, 200], page, form, causal=causal)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("new,lens,page", [([1, 0, 5, 130, 1, 2], [300, 9, 5, 260, 1, 40], 16), ([64, 200], [64, 201], 128),
                                           ([3, 3, 3], [0, 2, 3], 32), ([0, 0], [5, 0], 16)])
def test_ragged_tokens(hd, new, lens, page, form, kernel):
    check(gen(hd), hd, 8, 2, 0, lens, page, form, new=new, pad=(2, 3), causal=True, sink=True)
    check(gen(hd), hd, 3, 1, 0, lens, page, form, new=new, causal=False, max_q=1)     # more tokens than said


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("window,n_first", [(1, 0), (1, 1), (17, 4), (64, 33), (100, 64), (300, 16), (1000, 7), (5, 200), (2 ** 31 - 1, 3)])
@pytest.mark.parametrize("T,causal,page", [(1, False, 16), (9, True, 64), (3, False, 16), (140, True, 32)])
def test_window_and_first_keys(hd, window, n_first, T, causal, page, form, kernel):
    check(gen(window % 1000), hd, 4, 2, T, [0, 4, 40, 111, 256, 400, 399], page, form, window=window, n_first=n_first, causal=causal)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("T,page", [(1, 16), (7, 32), (130, 16), (3, 128)])
def test_pages_that_are_not_there(hd, T, page, form, kernel):
    """Given back behind a window, in the middle, the first, the last, all: their keys are attended by no row."""
    lens = [400, 399, 200, 300, 130, 16]

    def gone(table):
        table[0, 0] = -1
        table[1, 1] = 10 ** 6
        table[2, (200 - 1) // page] = -(2 ** 31)
        table[3, :] = -5
        table[4, : table.shape[1] // 2] = 2 ** 31 - 1

    check(gen(T), hd, 4, 2, T, lens, page, form, causal=True, gone=gone)
    check(gen(T), hd, 4, 2, T, lens, page, form, causal=True, gone=gone, sink=True, n_splits=3)
    check(gen(T), hd, 4, 2, T, lens, page, form, causal=True, gone=gone, window=90, n_first=5)


@pytest.mark.parametrize("n_splits", [1, 2, 3, 5, 64])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd,window,n_first,sink", [(128, 0, 0, False), (128, 150, 40, True), (64, 0, 0, True), (256, 70, 5, False), (512, 99, 17, True)])
def test_splits(hd, n_splits, window, n_first, sink, form, kernel):
    check(gen(hd), hd, 8, 2, 3, [0, 1, 130, 511, 1024], 16, form, window=window, n_first=n_first, causal=True, sink=sink, n_splits=n_splits)
    check(gen(hd), hd, 8, 2, 0, [0, 60, 130, 511, 700], 32, form, new=[0, 33, 2, 1, 3], pad=(1, 2), window=window, n_first=n_first, causal=True,
          sink=sink, n_splits=n_splits, max_q=33)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
def test_scales_and_bounds(hd, form, kernel):
    g = gen(hd)
    lens = [0, 7, 256]
    check(g, hd, 8, 2, 2, [0, 7, 200], 16, form, s_k=200)
    check(g, hd, 8, 2, 1, lens, 16, form, scale=-0.2)          # a negative scale turns the order round
    check(g, hd, 8, 2, 1, lens, 16, form, scale=0.0)           # every key the same weight
    check(g, hd, 8, 2, 2, lens, 16, form, scale=0.0, causal=True, window=30, n_first=3)
    check(g, hd, 8, 2, 1, lens, 16, form, scale=2.0 ** -140)
    check(g, hd, 8, 2, 2, lens, 16, form, k_mult=2.0 ** 60, scale=2.0 ** -63, n_splits=2)    # scale bytes far above 127
    check(g, hd, 8, 2, 2, lens, 16, form, k_mult=2.0 ** -60, scale=2.0 ** 57, n_splits=2)
    check(g, hd, 8, 2, 1, lens, 16, form, q_mult=2.0 ** 60, scale=2.0 ** -63)
    check(g, hd, 8, 2, 1, lens, 16, form, q_mult=2.0 ** -70, scale=2.0 ** 67)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("mult", [1.0, 2.0 ** 40, 2.0 ** 100, 2.0 ** -100])
def test_values_of_every_size(hd, mult, form, kernel):
    """V's scale bytes from one end to the other, row by row."""
    g = gen(hd)
    n, page = 300, 32
    cache, table = blank(12, 2, page, hd, form), ints([list(range(10))])
    k, v = normal(g, n, 2, hd), normal(g, n, 2, hd) * mult * 2.0 ** torch.randint(-12, 13, (n, 2, 1), generator=g, device=DEV)
    binding.fmha_paged_append(k, v.to(torch.bfloat16), *cache, table, ints([0]), cu_q=ints([0, n]))
    q = normal(g, 1, 8, 5, hd)
    got = binding.fmha_fwd_paged(q, *cache, table, ints([n]), causal=True, n_splits=2)
    ref.assert_attention(got, ref.attend(q, cache, table, [n], page, causal=True))


def test_lengths_and_bounds_beyond_what_there_is_are_cut(kernel):
    g = gen(9)
    cache, table = pool(g, [128] * 4, 1, 16, 64, FORMS[0])
    q = normal(g, 4, 2, 1, 64)
    o, lse = binding.fmha_fwd_paged(q, *cache, table, ints([-5, 2 ** 31 - 1, 101, -(2 ** 31)]), s_k=100)
    o2, lse2 = binding.fmha_fwd_paged(q, *cache, table, ints([0, 100, 100, 0]), s_k=100)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o, lse = binding.fmha_fwd_paged(q, *cache, table, ints([128, 2 ** 31 - 1, 129, 500]))
    o2, lse2 = binding.fmha_fwd_paged(q, *cache, table, ints([128] * 4))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # bounds past the tensor's end, negative ones, and ones that fall: what is left of them is computed, nothing else written
    x = normal(g, 6, 2, 64)
    o, lse = torch.full_like(x, 7.0), torch.full((6, 2), 7.0, device=DEV)
    binding.fmha_fwd_paged(x, *cache, table, ints([128] * 4), cu_q=ints([-3, 2, 1, 5, 900]), o=o, lse=lse, n_splits=1)
    good, glse = binding.fmha_fwd_paged(x, *cache, table, ints([128] * 4), cu_q=ints([0, 2, 2, 2, 6]), n_splits=1)
    assert torch.equal(o[:1], good[:1]) and torch.equal(lse[:1], glse[:1])
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("form", FORMS)
def test_pages_shared_by_sequences(form, kernel):
    """A common prefix on the same pages, and sequences that go on on pages of their own."""
    g = gen(5)
    cache, table = pool(g, [200, 130, 90], 2, 16, 128, form)
    table = table.clone()
    table[1, :4] = table[0, :4]
    table[2, :5] = table[0, :5]
    lens = [200, 130, 90]
    q = normal(g, 3, 8, 2, 128)
    got = binding.fmha_fwd_paged(q, *cache, table, ints(lens), causal=True)
    ref.assert_attention(got, ref.attend(q, cache, table, lens, 16, causal=True))


@pytest.mark.parametrize("form", FORMS)
def test_pool_past_32_bit_offsets(form, kernel):
    """Pages that lie more than 2^32 bytes into the pool, under a table that names them."""
    n_kv, page, hd = 8, 256, 512
    n_pages = (9 if form == FORMS[1] else 5) * (1 << 32) // ((1 if form == FORMS[1] else 2) * n_kv * page * hd) // 2
    cache = binding.fmha_paged_cache(n_pages, n_kv, page, hd, dtype=form)
    assert cache[0].numel() * cache[0].element_size() > 1 << 32
    g = gen(12)
    lens = [300, 20]
    table = ints([[n_pages - 1, n_pages - 3, 0], [n_pages - 2, 5, 1]])
    k, v = normal(g, 320, n_kv, hd), normal(g, 320, n_kv, hd)
    binding.fmha_paged_append(k, v, *cache, table, ints([0, 0]), cu_q=ints([0, 300, 320]))
    q = normal(g, 2, n_kv, 1, hd)
    got = binding.fmha_fwd_paged(q, *cache, table, ints(lens))
    ref.assert_attention(got, ref.attend(q, cache, table, lens, page))
    back, _ = binding.fmha_paged_gather(*cache, table, ints(lens), 300)
    want, _ = ref.sequence(cache[0], cache[2], table[0], 300, page)
    assert torch.equal(back[0], want.to(torch.bfloat16))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
def test_scores_that_rise(hd, form, kernel):
    """Far above the reference of the first tile, in every tile, for some rows of a warp and not for others; and one dominant key."""
    n, rows, page = 1024, 40, 64
    g = gen(93)
    k, v, q = normal(g, n, 1, hd) * 0.1, normal(g, n, 1, hd), normal(g, 1, rows, 1, hd)
    k[:, 0, 0] = torch.linspace(0, 96, n, device=DEV).to(torch.bfloat16)
    q[0, :, 0, 0] = torch.linspace(-4, 3 * hd ** 0.5, rows, device=DEV).to(torch.bfloat16)
    cache, table = blank(16, 1, page, hd, form), ints([list(range(15, -1, -1))])
    binding.fmha_paged_append(k, v, *cache, table, ints([0]), cu_q=ints([0, n]))
    want = ref.attend(q, cache, table, [n], page)
    for n_splits in (1, 0):
        ref.assert_attention(binding.fmha_fwd_paged(q, *cache, table, ints([n]), n_splits=n_splits), want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", HD)
@pytest.mark.parametrize("n_splits", [1, 2, 8])
@pytest.mark.parametrize("sink", [False, True])
def test_nan_scores_show_whatever_the_chunks(hd, n_splits, sink, form, kernel):
    """A NaN in a query row or in an attended K row: NaN in O and LSE of the rows that meet it, and only there."""
    g = gen(hd)
    lens, n_h, n_kv, T, page = [1024, 700, 100, 0], 4, 2, 2, 16
    cache, table = pool(g, lens, n_kv, page, hd, form)
    q = normal(g, 4, n_h, T, hd)
    sg = torch.randn(n_h, generator=g, device=DEV) * 2 if sink else None
    ro, rl, o_tol, l_tol = ref.attend(q, cache, table, lens, page, causal=True, sink=sg)
    bad = torch.zeros((4, n_h, T), dtype=torch.bool, device=DEV)
    q[1, 2, 1, 5] = float("nan")
    q[2, 1, 0] = float("nan")
    p, r = int(table[0, 1023 // page]), 1023 % page
    if form == FORMS[0]:
        cache[0][p, 1, r, 2] = float("nan")
    else:
        cache[2][p, 1, r] = 255
    bad[1, 2, 1] = bad[2, 1, 0] = True
    bad[0, 2:, 1] = True                        # the last key: causal hides it from the first row
    o, lse = binding.fmha_fwd_paged(q, *cache, table, ints(lens), causal=True, sink=sg, n_splits=n_splits)
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    keep = ~bad
    assert ((o.double() - ro).abs() <= o_tol)[keep].all()
    fin = keep & torch.isfinite(rl)
    assert torch.equal(torch.isinf(lse[keep]), torch.isinf(rl[keep])) and ((lse.double() - rl).abs() <= l_tol)[fin].all()


@pytest.mark.parametrize("form", FORMS)
def test_strided_queries(form, kernel):
    """Query heads in the rows of a projection, of other layouts, broadcast."""
    g = gen(2)
    lens, page, hd, n_h = [130, 64, 20], 16, 128, 6
    cache, table = pool(g, lens, 2, page, hd, form)
    wide = normal(g, 3, 4, n_h + 5, hd)
    for q in (wide[:, :, 2 : 2 + n_h].transpose(1, 2), wide[:, :1, :n_h].transpose(1, 2), wide[:1, :, :n_h].transpose(1, 2).expand(3, n_h, 4, hd)):
        ref.assert_attention(binding.fmha_fwd_paged(q, *cache, table, ints(lens), causal=True), ref.attend(q, cache, table, lens, page, causal=True))
    flat = wide.reshape(12, n_h + 5, hd)[:, 1 : 1 + n_h]
    cu = [0, 5, 6, 12]
    ref.assert_attention(binding.fmha_fwd_paged(flat, *cache, table, ints(lens), cu_q=ints(cu), causal=True),
                         ref.attend(flat, cache, table, lens, page, cu, causal=True))


def test_no_rows_and_no_keys(kernel):
    g = gen(1)
    for form in FORMS:
        cache = binding.fmha_paged_cache(2, 2, 16, 64, dtype=form)
        for b, T in ((0, 1), (2, 0)):
            o, lse = binding.fmha_fwd_paged(normal(g, b, 4, T, 64), *cache, torch.zeros((b, 1), dtype=torch.int32, device=DEV), ints([1] * b))
            assert o.shape == (b, 4, T, 64) and lse.shape == (b, 4, T)
        binding.fmha_paged_append(normal(g, 2, 2, 0, 64), normal(g, 2, 2, 0, 64), *cache, ints([[0], [1]]), ints([0, 0]))
        q, sink = normal(g, 2, 4, 3, 64), torch.randn(4, device=DEV)
        for pages, table in ((binding.fmha_paged_cache(0, 2, 16, 64, dtype=form), ints([[0], [1]])), (cache, torch.zeros((2, 0), dtype=torch.int32, device=DEV))):
            o, lse = binding.fmha_fwd_paged(q, *pages, table, ints([5, 5]), sink=sink)
            assert (o == 0).all() and torch.equal(lse, sink[None, :, None].expand_as(lse))
            binding.fmha_paged_append(normal(g, 2, 2, 1, 64), normal(g, 2, 2, 1, 64), *pages, table, ints([0, 0]))
            k, _ = binding.fmha_paged_gather(*pages, table, ints([5, 5]), 4)
            assert (k == 0).all()
        o, lse = binding.fmha_fwd_paged(q[:, :, :0].reshape(0, 4, 64), *cache, ints([[0], [1]]), ints([1, 1]), cu_q=ints([0, 0, 0]))
        assert o.shape == (0, 4, 64)


# ------------------------------------------------------------------ together, as a serving loop runs them
def serving_step(state, qkv, cu, start, lens, outputs=None):
    """Projection rows of a ragged batch -> norm and rotation -> append -> attention."""
    n_h, n_kv, cache, table, cos_sin, weight = state
    total = qkv.shape[0]
    seq = torch.bucketize(torch.arange(total, device=DEV, dtype=torch.int32), cu[1:], right=True, out_int32=True).clamp(max=len(start) - 1).long()
    positions = (start[seq] + torch.arange(total, device=DEV, dtype=torch.int32) - cu[seq]).to(torch.int32)
    q, k, v = binding.fmha_qk_norm_rope(qkv[None], cos_sin, positions[None].contiguous(), n_h, n_kv, q_weight=weight, k_weight=weight)
    q, k, v = (x[0].transpose(0, 1) for x in (q, k, v))
    binding.fmha_paged_append(k, v, *cache, table, start, cu_q=cu)
    return (q, k, v) + binding.fmha_fwd_paged(q, *cache, table, lens, cu_q=cu, causal=True, **(outputs or {}))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", [64, 128])
def test_a_batch_grows_step_by_step(hd, form):
    """Prompts in chunks and single tokens in one batch, three steps; at the end each sequence's last rows agree with fmha_fwd over
    what gather brings back."""
    g = gen(4)
    n_h, n_kv, page, b = 8, 2, 16, 3
    cache = blank(40, n_kv, page, hd, form)
    table = torch.randperm(40, generator=g, device=DEV)[:36].reshape(b, 12).to(torch.int32)
    angle = torch.arange(192, device=DEV)[:, None] * 10000.0 ** (-torch.arange(0, hd, 2, device=DEV) / hd)
    state = (n_h, n_kv, cache, table, torch.cat([angle.cos(), angle.sin()], 1).float().contiguous(), torch.ones(hd, device=DEV))
    have = [0, 0, 0]
    for new in ([100, 1, 30], [1, 70, 40], [1, 1, 1]):
        cu = [sum(new[:i]) for i in range(b + 1)]
        lens = [a + n for a, n in zip(have, new)]
        q, k, v, o, lse = serving_step(state, normal(g, cu[-1], (n_h + 2 * n_kv) * hd), ints(cu), ints(have), ints(lens))
        ref.assert_attention((o, lse), ref.attend(q, cache, table, lens, page, cu, causal=True))
        have = lens
    kc, vc = binding.fmha_paged_gather(*cache, table, ints(have), max(have))
    for i, n in enumerate(have):
        o2, lse2 = binding.fmha_fwd(q[cu[i] : cu[i + 1]].transpose(0, 1)[None].contiguous(), kc[i : i + 1, :, :n].contiguous(),
                                    vc[i : i + 1, :, :n].contiguous(), causal=True)
        # both are within a bf16 rounding of P and of O of the same value
        assert (o2[0].transpose(0, 1).float() - o[cu[i] : cu[i + 1]].float()).abs().max() <= 6 * 2.0 ** -8 * vc.abs().max()
        assert (lse2[0].transpose(0, 1) - lse[cu[i] : cu[i + 1]]).abs().max() <= 1e-3


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n_h", [8, 64])
def test_steps_captured_and_replayed(n_h, form):
    """Append, gather and (split) attention in one graph, replayed on other lengths, bounds and pages."""
    g = gen(6)
    n_kv, page, hd, b = 2, 16, 128, 3
    cache = blank(64, n_kv, page, hd, form)
    table = torch.randperm(64, generator=g, device=DEV)[:60].reshape(b, 20).to(torch.int32)
    k, v, q = normal(g, 9, n_kv, hd), normal(g, 9, n_kv, hd), normal(g, 9, n_h, hd)
    cu, start, lens = ints([0, 3, 4, 9]), ints([0, 0, 0]), ints([3, 1, 5])

    def step():
        binding.fmha_paged_append(k, v, *cache, table, start, cu_q=cu)
        return binding.fmha_fwd_paged(q, *cache, table, lens, cu_q=cu, causal=True, n_splits=3) + binding.fmha_paged_gather(*cache, table, lens, 64)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    for bounds, first in (([0, 3, 4, 9], [0, 0, 0]), ([0, 1, 8, 9], [3, 1, 60]), ([0, 4, 4, 8], [290, 100, 17])):
        for t in cache:
            if t is not None:
                t.view(torch.uint8).random_(0, 64)   # finite rows of any kind
        for x in (q, k, v):
            x.copy_(normal(g, *x.shape))
        table.copy_(torch.randperm(64, generator=g, device=DEV)[:60].reshape(b, 20))
        cu.copy_(ints(bounds))
        start.copy_(ints(first))
        ends = [f + bounds[i + 1] - bounds[i] for i, f in enumerate(first)]
        lens.copy_(ints(ends))
        outs[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.attend(q, cache, table, ends, page, bounds, causal=True)
        n = bounds[-1]
        ref.assert_attention((outs[0][:n], outs[1][:n]), tuple(x[:n] for x in want))
        for i, e in enumerate(ends):
            x, _ = ref.sequence(cache[0], cache[2], table[i], min(e, 64), page)
            assert torch.equal(outs[2][i, :, : min(e, 64)], x.to(torch.bfloat16))


def test_two_streams_at_once():
    """Split calls on two streams keep their partials apart."""
    g = gen(8)
    cache, table = pool(g, [3000, 2000], 2, 16, 128, FORMS[0])
    q = [normal(g, 2, 8, 1, 128) for _ in range(2)]
    lens = ints([3000, 2000])
    want = [binding.fmha_fwd_paged(x, *cache, table, lens, n_splits=8) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [binding.fmha_fwd_paged(x, *cache, table, lens, n_splits=8, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        for (o, lse), (ro, rl) in zip(got, want):
            assert torch.equal(o, ro) and torch.equal(lse, rl)
    ws = torch.empty(binding.fmha_workspace_bytes(1, 8, 2, 128, 8), dtype=torch.uint8, device=DEV)
    o, lse = binding.fmha_fwd_paged(q[0], *cache, table, lens, n_splits=8, workspace=ws)
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    with pytest.raises(binding.FmhaError):
        binding.fmha_fwd_paged(q[0], *cache, table, lens, n_splits=8, workspace=ws[:-16])


def test_refusals_of_tensors():
    cache = binding.fmha_paged_cache(4, 2, 16, 64)
    codes = binding.fmha_paged_cache(4, 2, 16, 64, dtype=FORMS[1])
    table, lens, q, kv = ints([[0, 1]]), ints([5]), torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device=DEV)
    ok = binding.fmha_fwd_paged(q, *cache, table, lens)[0]
    assert ok.shape == q.shape
    for bad in (lambda: binding.fmha_fwd_paged(q.float(), *cache, table, lens), lambda: binding.fmha_fwd_paged(q, *cache, table.long(), lens),
                lambda: binding.fmha_fwd_paged(q, *cache, table, lens.float()), lambda: binding.fmha_fwd_paged(q, cache[0].float(), cache[1], None, None, table, lens),
                lambda: binding.fmha_fwd_paged(q.cpu(), *cache, table, lens), lambda: binding.fmha_fwd_paged(q, *cache, table, lens.cpu()),
                lambda: binding.fmha_fwd_paged(q, *cache, table.expand(2, 2)[:, ::2], ints([5, 5])),
                lambda: binding.fmha_paged_append(kv, kv.float(), *cache, table, lens), lambda: binding.fmha_paged_append(kv, kv, *cache, table, lens.cpu())):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: binding.fmha_fwd_paged(q, cache[0], cache[1], codes[2], codes[3], table, lens),   # scales beside bf16 pages
                lambda: binding.fmha_fwd_paged(q, codes[0], codes[1], None, None, table, lens),
                lambda: binding.fmha_fwd_paged(q, codes[0], codes[1], codes[2], None, table, lens),
                lambda: binding.fmha_fwd_paged(q, *codes[:2], codes[2][:3], codes[3], table, lens),
                lambda: binding.fmha_fwd_paged(q, *cache, table, ints([5, 5])), lambda: binding.fmha_fwd_paged(q, *cache, table, lens, cu_q=ints([0, 1])),
                lambda: binding.fmha_fwd_paged(q[:, :, 0], *cache, table, lens, cu_q=ints([0])),
                lambda: binding.fmha_fwd_paged(q[..., :32], *cache, table, lens), lambda: binding.fmha_fwd_paged(q, *cache, table[0], lens),
                lambda: binding.fmha_fwd_paged(q, *cache, table, lens, o=torch.empty(1, 4, 2, 64, dtype=torch.bfloat16, device=DEV)),
                lambda: binding.fmha_fwd_paged(q, *cache, table, lens, lse=torch.empty(1, 4, 2, device=DEV)),
                lambda: binding.fmha_paged_append(kv, kv[:, :1], *cache, table, lens), lambda: binding.fmha_paged_append(kv[0], kv[0], *cache, table, lens),
                lambda: binding.fmha_paged_append(kv, kv.expand(1, 2, 2, 64), *cache, table, lens),
                lambda: binding.fmha_paged_gather(*cache, table, lens, 4, k=kv), lambda: binding.fmha_paged_gather(*cache, table, lens, 4, k=kv, v=kv),
                lambda: binding.fmha_fwd_paged(torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16, device=DEV)[..., ::2], *cache, table, lens)):
        with pytest.raises((ValueError, binding.FmhaError)):
            bad()
    wide = torch.zeros(2, 4, 3, 68, dtype=torch.bfloat16, device=DEV)[..., :64]   # token rows 68 elements apart
    with pytest.raises(binding.FmhaError):
        binding.fmha_fwd_paged(wide, *cache, table.expand(2, 2).contiguous(), ints([5, 5]))


def test_same_call_twice_is_bitwise_the_same(kernel):
    g = gen(3)
    for form in FORMS:
        cache, table = pool(g, [2000, 700, 40], 2, 32, 128, form)
        q = normal(g, 3, 16, 9, 128)
        runs = [binding.fmha_fwd_paged(q, *cache, table, ints([2000, 700, 40]), causal=True) for _ in range(3)]
        for o, lse in runs[1:]:
            assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
