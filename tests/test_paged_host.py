"""Refusals of the calls on a cache in pages, without a GPU: the C entry points' argument checks (nothing is
launched on an error), the plan, the argument structs and the binding's own checks; and the 8-bit form's reference."""
import math
import os
import struct
import subprocess

import pytest
import torch

import paged_ref as ref
from head_attention_forward_fmha_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


P = 4096  # an aligned address that is never read: every call below is refused or has nothing to do

APPEND = dict(k=P, v=P, kp=P, vp=P, ks=None, vs=None, table=P, start=P, cu=None, stream=None, k0=1024, k1=128, k2=128, v0=1024, v1=128, v2=128,
              batch=2, T=1, total=0, n_kv=8, hd=128, page=16, n_pages=8, width=4)
GATHER = dict(kp=P, vp=P, ks=None, vs=None, table=P, lens=P, start=None, k=P, v=P, stream=None, batch=2, rows=4, n_kv=8, hd=128, page=16,
              n_pages=8, width=4, reserved=0)
FWD = dict(q=P, kp=P, vp=P, ks=None, vs=None, table=P, lens=P, cu=None, o=P, lse=P, sink=None, ws=None, wsb=0, stream=None, q0=8192, q1=128,
           q2=128, scale=0.1, batch=2, T=1, total=0, n_h=64, n_kv=8, hd=128, page=16, n_pages=8, width=4, s_k=64, window=0, n_first=0, causal=1,
           n_splits=1, reserved=0)
FORMATS = {"fmha_paged_append": "=10Q6q8i", "fmha_paged_gather": "=10Q8i", "fmha_fwd_paged": "=14Q3qf15i"}


def call(lib, name, base, change):
    return getattr(lib, name)(struct.pack(FORMATS[name], *[0 if x is None else x for x in {**base, **change}.values()]))


COMMON = [
    (dict(hd=96), -3), (dict(hd=32), -3), (dict(n_kv=0), -4), (dict(batch=-1), -5), (dict(page=8), -5), (dict(page=24), -5), (dict(page=0), -5),
    (dict(page=131072), -5), (dict(page=-16), -5), (dict(n_pages=-1), -5), (dict(width=-1), -5), (dict(n_pages=1 << 24), -5), (dict(kp=None), -1),
    (dict(vp=None), -1), (dict(table=None), -1), (dict(ks=P), -1), (dict(vs=P), -1), (dict(kp=P + 8), -2), (dict(ks=P + 4, vs=P), -2),
    (dict(table=P + 2), -2), (dict(batch=0), 0),
]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(T=-1), -5), (dict(cu=P, total=-1), -5), (dict(k0=4), -5), (dict(k1=-128), -5), (dict(v2=12), -5), (dict(batch=1 << 15, T=1 << 15), -5),
    (dict(k=None), -1), (dict(start=None), -1), (dict(k=P + 8), -2), (dict(start=P + 1), -2), (dict(cu=P + 2, total=3), -2), (dict(T=0), 0),
    (dict(cu=P, total=0), 0), (dict(n_pages=0), 0), (dict(width=0), 0),
])
def test_append_refusals(lib, change, code):
    assert call(lib, "fmha_paged_append", APPEND, change) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(rows=-1), -5), (dict(rows=1 << 28), -5), (dict(lens=None), -1), (dict(k=None), -1), (dict(v=P + 8), -2), (dict(start=P + 2), -2),
    (dict(rows=0), 0), (dict(n_pages=0), 0), (dict(width=0), 0),
])
def test_gather_refusals(lib, change, code):
    assert call(lib, "fmha_paged_gather", GATHER, change) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(n_h=12), -4), (dict(n_h=0), -4), (dict(T=-1), -5), (dict(cu=P, total=-2), -5), (dict(s_k=-1), -5), (dict(s_k=(1 << 30) + 1), -5),
    (dict(window=-1), -5), (dict(n_first=-1), -5), (dict(causal=2), -5), (dict(n_splits=-1), -5), (dict(scale=math.nan), -5), (dict(scale=3e38), -5),
    (dict(q1=4), -5), (dict(q0=-8), -5), (dict(batch=1 << 14, T=1 << 14), -5), (dict(q=None), -1), (dict(lens=None), -1), (dict(o=None), -1),
    (dict(lse=None), -1), (dict(q=P + 8), -2), (dict(o=P + 2), -2), (dict(lse=P + 2), -2), (dict(sink=P + 1), -2), (dict(cu=P + 1, total=2), -2),
    (dict(T=0), 0), (dict(cu=P, total=0), 0), (dict(s_k=1024, width=64, n_splits=4), -6), (dict(s_k=1024, width=64, n_splits=4, ws=P, wsb=100), -6),
    (dict(s_k=1024, width=64, n_splits=4, ws=P + 8, wsb=1 << 30), -2),
])
def test_attention_refusals(lib, change, code):
    assert call(lib, "fmha_fwd_paged", FWD, change) == code
    if code < 0:
        assert binding.fmha_get_last_error()


def test_null_arguments(lib):
    for name in FORMATS:
        assert getattr(lib, name)(None) == -1


def test_argument_structs_are_laid_out_as_packed_here(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    last = {"fmha_paged_append": "table_width", "fmha_paged_gather": "reserved", "fmha_fwd_paged": "reserved"}
    lines = "".join('printf("%%zu %%zu ", offsetof(struct %s_args, %s), sizeof(struct %s_args));' % (n, f, n) for n, f in last.items())
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fmha.h"\nint main(void) {%s return 0;}\n' % lines)
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [x for n in last for x in (struct.calcsize(FORMATS[n]) - 4, struct.calcsize(FORMATS[n]))]
    kinds = {**dict.fromkeys("BFIUbfiuS", "Q"), "q": "q", "n": "i", "r": "f"}
    for entries in (binding._PAGED_APPEND, binding._PAGED_GATHER, binding._PAGED_FWD):
        for name, layout, tensors in entries.values():
            fields = "".join(kinds[c] for c in layout.decode())
            assert struct.calcsize("=" + fields) == struct.calcsize(FORMATS[name]) <= 248
            assert sum(c in "BFIUbfiuS" for c in layout.decode()) == len(tensors)


def test_plan():
    plan = binding.fmha_fwd_paged_plan
    assert plan(1, 1, 64, 8, 128, 16, 8192) > 1                       # one user: the keys are divided
    assert plan(64, 1, 64, 8, 128, 16, 100) == 1                      # nothing to divide
    assert plan(4, 2048, 64, 8, 128, 16, 8192, causal=True) == 1      # enough rows
    assert plan(1, 1, 64, 8, 128, 16, 0) == 1 and plan(0, 1, 64, 8, 128, 16, 64) == 1 and plan(1, 0, 64, 8, 128, 16, 64) == 1
    for n in (1, 2, 3, 7, 64, 1000):
        for s_k in (1, 100, 8192):
            assert 1 <= plan(1, 1, 64, 8, 128, 16, s_k, n_splits=n) <= min(n, 64)
    # a short window has few keys to divide, however long the sequences are
    assert plan(1, 1, 8, 1, 128, 16, 1 << 20, window=256, n_first=4) <= 8
    assert plan(3, 40, 8, 2, 128, 16, 4096, total=50) >= 1
    for bad in (dict(hd=100), dict(page=20), dict(n_h=9), dict(s_k=-1), dict(n_splits=-1)):
        with pytest.raises(binding.FmhaError):
            plan(**{**dict(batch=1, T=1, n_h=8, n_kv_h=2, hd=128, page=16, s_k=64), **bad})
    # a call's partials stay within a GiB
    n = plan(512, 1, 128, 8, 128, 16, 1 << 20, n_splits=64)
    assert n * 512 * 128 * 129 * 4 <= 1 << 30


def test_binding_refusals():
    bf = torch.zeros(1, 8, 1, 128, dtype=torch.bfloat16)
    cache = binding.fmha_paged_cache(4, 2, 16, 128, device="cpu")
    assert [None if t is None else (tuple(t.shape), t.dtype) for t in cache] == [((4, 2, 16, 128), torch.bfloat16)] * 2 + [None] * 2
    codes = binding.fmha_paged_cache(4, 2, 16, 128, dtype=torch.float8_e4m3fn, device="cpu")
    assert [tuple(t.shape) for t in codes] == [(4, 2, 16, 128)] * 2 + [(4, 2, 16)] * 2 and all(t.dtype == torch.uint8 for t in codes)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (lambda: binding.fmha_fwd_paged(bf, *cache, table, lens), lambda: binding.fmha_paged_append(bf, bf, *cache, table, lens),
                lambda: binding.fmha_paged_gather(*cache, table, lens, 4)):   # host tensors
        with pytest.raises(TypeError):
            bad()
    for bad in (dict(hd=96), dict(page=8), dict(page=48), dict(dtype=torch.float16), dict(page=1 << 17)):
        with pytest.raises(ValueError):
            binding.fmha_paged_cache(**{**dict(n_pages=1, n_kv_h=1, page=16, hd=64, device="cpu"), **bad})


# ------------------------------------------------------------------ the reference of the 8-bit form
def test_reference_codes_agree_with_torchs_cast():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(200, 64, generator=g) * 2.0 ** torch.randint(-100, 100, (200, 1), generator=g)).to(torch.bfloat16)
    x[0] = 0
    x[1, 3], x[2, 3], x[3, 3] = 448.0, 450.0, -449.0
    codes, byte = ref.quantise(x)
    cast = torch.ldexp(x.float(), 127 - byte.int()[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(codes, cast.view(torch.uint8))
    assert torch.equal(ref.values(codes, byte), torch.ldexp(cast.double(), (byte.int() - 127)[:, None]))
    # the scale is the smallest that fits
    top = x.double().abs().amax(-1)
    s = torch.exp2(byte.double() - 127)
    assert (top <= 448 * s).all() and ((top > 224 * s) | (byte == 0)).all()
    for table in (ref.E4M3[:127], [-v for v in ref.E4M3[128:255]]):
        assert table == torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().tolist()


def test_reference_marks_rows_that_are_not_finite():
    x = torch.ones(3, 64, dtype=torch.bfloat16)
    x[0, 5], x[1, 6] = math.nan, -math.inf
    codes, byte = ref.quantise(x)
    assert byte.tolist()[:2] == [255, 255] and (codes[:2] == 0).all() and torch.isnan(ref.values(codes, byte)[:2]).all()


def test_reference_attention_is_torchs_softmax():
    g = torch.Generator().manual_seed(2)
    pages = [torch.randn(5, 2, 16, 64, generator=g).to(torch.bfloat16) for _ in range(2)]
    table, n = torch.tensor([[3, 0, 4]]), 41
    q = torch.randn(1, 4, 7, 64, generator=g).to(torch.bfloat16)
    o, lse, _, _ = ref.attend(q, (*pages, None, None), table, [n], 16, causal=True)
    k, v = (p[[3, 0, 4]].transpose(0, 1).reshape(2, 48, 64)[:, :n].double().repeat_interleave(2, 0) for p in pages)
    x = q[0].double() @ k.transpose(1, 2) / 8.0
    x = x.masked_fill(torch.arange(n) > n - 7 + torch.arange(7)[:, None], -math.inf)
    assert torch.allclose(o[0], torch.softmax(x, -1) @ v, atol=1e-12) and torch.allclose(lse[0], torch.logsumexp(x, -1), atol=1e-12)
    # pages that are not there are as if their keys were not, and the order of pages is the table's
    o2, _, _, _ = ref.attend(q, (*pages, None, None), torch.tensor([[3, -1, 4]]), [n], 16)
    keep = torch.cat([torch.arange(16), torch.arange(32, n)])
    x = q[0].double() @ k[:, keep].transpose(1, 2) / 8.0
    assert torch.allclose(o2[0], torch.softmax(x, -1) @ v[:, keep], atol=1e-12)
