"""Refusals of the serving operators, without a GPU: the C entry points' argument
checks (nothing is launched on an error), the 4-bit plan, and the binding's own checks."""
import re
import struct

import pytest
import torch

from head_attention_forward_fmha_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


P = 4096  # an aligned address that is never read: every call below is refused

NORM = dict(qkv=P, bs=0, ts=1280, qw=None, kw=None, eps=1e-6, cs=P, pos=P, max_pos=64, rot=128, inter=0, q=P, k=P, v=P, start=None,
            rows=1, b=1, T=1, n_h=8, n_kv=1, hd=128, stream=None)
APPEND = dict(k=P, v=P, kc=P, ks=P, vc=P, vs=P, start=P, kg=1.0, vg=1.0, ko=None, vo=None, b=1, n_kv=1, T=1, cap=64, hd=128, stream=None)
KV4 = dict(q=P, kc=P, ks=P, vc=P, vs=P, lens=None, o=P, lse=P, sink=None, kg=1.0, vg=1.0, b=1, n_h=8, n_kv=1, T=1, s_k=64, cap=64,
           hd=128, scale=0.1, window=0, n_first=0, causal=0, chunk=0, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(hd=96), -3), (dict(n_h=3, n_kv=2), -4), (dict(n_kv=0), -4), (dict(b=-1), -5), (dict(T=-1), -5), (dict(rows=-1), -5),
    (dict(rot=4), -5), (dict(rot=136), -5), (dict(rot=-8), -5), (dict(max_pos=0), -5), (dict(inter=2), -5), (dict(eps=-1.0), -5),
    (dict(eps=float("nan")), -5), (dict(ts=1272), -5), (dict(ts=1284), -5), (dict(bs=4), -5), (dict(bs=-8), -5), (dict(qkv=None), -1),
    (dict(cs=None), -1), (dict(pos=None), -1), (dict(q=None), -1), (dict(v=None), -1), (dict(qkv=P + 8), -2), (dict(k=P + 2), -2),
    (dict(qw=P + 4), -2), (dict(start=P + 1), -2), (dict(b=0), 0), (dict(T=0), 0),
])
def test_norm_rope_refusals(lib, change, code):
    assert lib.fmha_qk_norm_rope(*{**NORM, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(hd=32), -3), (dict(n_kv=0), -4), (dict(b=-1), -5), (dict(cap=40), -5), (dict(cap=-16), -5), (dict(kg=0.0), -5),
    (dict(vg=float("inf")), -5), (dict(k=None), -1), (dict(start=None), -1), (dict(ko=P), -1), (dict(vc=P + 8), -2), (dict(k=P + 8), -2),
    (dict(b=0), 0), (dict(T=0), 0), (dict(cap=0), 0), (dict(b=1 << 20, n_kv=1 << 8, T=1 << 12), -5),
])
def test_append_refusals(lib, change, code):
    assert lib.fmha_kv4_append(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    (dict(hd=80), -3), (dict(n_h=6, n_kv=4), -4), (dict(T=-1), -5), (dict(s_k=-1), -5), (dict(s_k=65), -5), (dict(cap=72), -5),
    (dict(window=-1), -5), (dict(n_first=-1), -5), (dict(causal=2), -5), (dict(scale=float("nan")), -5), (dict(kg=-1.0), -5),
    (dict(chunk=-1), -5), (dict(b=70000), -5), (dict(q=None), -1), (dict(vs=None), -1), (dict(lse=None), -1), (dict(q=P + 4), -2),
    (dict(kc=P + 8), -2), (dict(lens=P + 2), -2), (dict(T=0), 0), (dict(b=0), 0),
    (dict(s_k=1024, cap=1024, chunk=256), -6), (dict(s_k=1024, cap=1024, chunk=256, ws=P, wsb=16), -6),
    (dict(s_k=1024, cap=1024, chunk=256, ws=P + 8, wsb=1 << 20), -2),
])
def test_kv4_refusals(lib, change, code):
    assert lib.fmha_fwd_kv4(*{**KV4, **change}.values()) == code
    if code < 0:
        assert binding.fmha_get_last_error()


FIRST = dict(q=P, k=P, v=P, o=P, lse=P, sink=None, b=1, n_h=8, n_kv=1, T=1, s_k=64, hd=128, scale=0.1, window=16, n_first=4, causal=0,
             ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(hd=80), -3), (dict(n_h=6, n_kv=4), -4), (dict(T=-1), -5), (dict(s_k=-1), -5), (dict(window=-1), -5), (dict(n_first=-1), -5),
    (dict(causal=2), -5), (dict(causal=1, T=65), -5), (dict(scale=float("inf")), -5), (dict(q=None), -1), (dict(v=None), -1), (dict(o=None), -1),
    (dict(q=P + 8), -2), (dict(sink=P + 1), -2), (dict(T=0), 0), (dict(b=0), 0), (dict(s_k=1 << 30 | 1), -5),
    (dict(s_k=65536, window=65000), -6), (dict(s_k=65536, window=65000, ws=P, wsb=100), -6),
    (dict(s_k=65536, window=65000, ws=P + 4, wsb=1 << 30), -2),
])
def test_first_refusals(lib, change, code):
    assert lib.fmha_fwd_first(*{**FIRST, **change}.values()) == code


def test_argument_structs_are_laid_out_as_packed_here(tmp_path):
    """The binding packs the structs of include/fmha.h itself: sizes and the offsets of the last fields."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    last = [("qk_norm_rope", "hd", "=10Q2qf9i"), ("kv4_append", "reserved", "=10Q2f6i"), ("fwd_kv4", "kv_chunk", "=12Q3f11i"),
            ("fwd_first", "causal", "=9Qf9i")]
    lines = "".join('printf("%%zu ", offsetof(struct fmha_%s_args, %s));' % (n, f) for n, f, _ in last)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fmha.h"\nint main(void) {%s return 0;}\n' % lines)
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [struct.calcsize(f) - 4 for _, _, f in last]
    # the binding's layouts have the same fields (a pointer for each tensor)
    for (name, layout, tensors), (n, _, f) in zip((binding._NORM_ROPE, binding._APPEND, binding._KV4, binding._FIRST), last):
        kinds = {**dict.fromkeys("BFIUbfiuS", "Q"), "q": "q", "n": "i", "r": "f"}
        fields = "".join(kinds[c] for c in layout.decode())
        assert name == "fmha_" + n and struct.calcsize("=" + fields) == struct.calcsize(f)
        assert sum(c in "BFIUbfiuS" for c in layout.decode()) == len(tensors)
        assert fields.replace("q", "Q") == "".join((c * int(k or 1)).replace("q", "Q") for k, c in re.findall(r"(\d*)([Qqfi])", f))


def test_packed_calls_refuse_like_the_others(lib):
    assert lib.fmha_fwd_kv4_packed(None) == -1 and lib.fmha_fwd_first_packed(None) == -1
    assert lib.fmha_qk_norm_rope_packed(None) == -1 and lib.fmha_kv4_append_packed(None) == -1
    assert lib.fmha_fwd_kv4_packed(struct.pack("=12Q3f11i", *[P] * 5, 0, P, P, 0, 0, 0, 0, 1.0, 1.0, 0.1, 1, 8, 1, 1, 64, 64, 80, 0, 0, 0, 0)) == -3
    assert lib.fmha_fwd_first_packed(struct.pack("=9Qf9i", *[P] * 5, 0, 0, 0, 0, 0.1, 1, 8, 1, 1, 64, 128, 16, -1, 0)) == -5
    assert lib.fmha_kv4_append_packed(struct.pack("=10Q2f6i", *[P] * 7, 0, 0, 0, 1.0, 1.0, 1, 1, 1, 40, 128, 0)) == -5
    assert lib.fmha_qk_norm_rope_packed(struct.pack("=10Q2qf9i", *[P] * 8, 0, 0, 0, 1280, 1e-6, 64, 4, 0, 1, 1, 1, 8, 1, 128)) == -5


def test_first_workspace():
    f = binding.fmha_fwd_first_workspace_bytes
    assert f(1, 8, 1, 1, 64, 128, 16, 4) == 0          # one chunk
    assert f(1, 8, 1, 1, 65536, 128, 65000, 4) > 0
    assert f(1, 8, 3, 1, 65536, 128, 65000, 4) == 0    # refused by the call
    # a window that holds every key is none: fmha_fwd's plan
    n, _ = binding.fmha_fwd_plan(1, 8, 1, 1, 4096, 128)
    assert f(1, 8, 1, 1, 4096, 128, 4096, 4) == binding.fmha_workspace_bytes(1, 8, 1, 128, n)


def test_kv4_plan():
    n, chunk = binding.fmha_fwd_kv4_plan(1, 64, 8, 1, 8192, 128)
    assert n > 1 and chunk % 32 == 0 and n * chunk >= 8192
    assert binding.fmha_fwd_kv4_plan(1, 64, 8, 1, 8192, 128, kv_chunk=1000) == (8, 1024)
    # a window shorter than the sequence: the first keys' tile and the window's keys
    assert binding.fmha_fwd_kv4_plan(1, 8, 1, 1, 8192, 128, window=512, n_first=4, kv_chunk=32) == (18, 32)
    assert binding.fmha_fwd_kv4_plan(1, 8, 1, 1, 0, 128)[0] == 1
    with pytest.raises(binding.FmhaError):
        binding.fmha_fwd_kv4_plan(1, 8, 3, 1, 64, 128)
    # chunks cover the longest axis whatever the sequences' lengths are taken to be
    for ragged in (False, True):
        for T in (1, 128):
            n, chunk = binding.fmha_fwd_kv4_plan(32, 64, 8, T, 32768, 128, ragged=ragged)
            assert n * chunk >= 32768 > (n - 1) * chunk


def test_binding_refusals():
    bf = torch.zeros(1, 8, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # host tensors
        binding.fmha_qk_norm_rope(torch.zeros(1, 1, 1280, dtype=torch.bfloat16), None, None, 8, 1)
    cache = binding.fmha_kv4_cache(1, 1, 64, 128, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(1, 1, 64, 64), (1, 1, 64, 8)] * 2
    with pytest.raises(TypeError):
        binding.fmha_fwd_kv4(bf, *cache, s_k=64)
    with pytest.raises(TypeError):
        binding.fmha_kv4_append(bf[:, :1], bf[:, :1], *cache, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        binding.fmha_fwd_first(bf, bf, bf, 4, window=8)
    with pytest.raises(ValueError):
        binding.fmha_kv4_cache(1, 1, 40, 128, device="cpu")


def test_kv4_refuses_what_its_arithmetic_does_not_hold(lib):
    """Positions len - T - window and the factor scale * k_global * log2(e) past 32 bits."""
    big = (1 << 31) - 8192
    assert lib.fmha_fwd_kv4(*{**KV4, **dict(T=8192, s_k=big, cap=big, window=big - 1)}.values()) == -5
    assert lib.fmha_fwd_kv4_plan(1, 8, 1, 8192, big, 128, big - 1, 0, 1, 1, None) == -5
    assert lib.fmha_fwd_kv4_plan(1, 8, 1, 8192, big, 128, big, 0, 1, 1, None) > 0  # holds every key: no window
    assert lib.fmha_fwd_kv4(*{**KV4, **dict(scale=1e30, kg=1e30)}.values()) == -5


def test_plans_are_kept_within_bounds():
    plans = {}
    for i in range(10000):
        assert binding._remember(plans, i, -i) == -i and plans[i] == -i
    assert len(plans) <= 4096


def test_argument_packer():
    """What the packer refuses, and the bytes that it passes on (read back by a callback)."""
    import ctypes

    from head_attention_forward_fmha_gb300 import _tensor_args

    got = []

    @ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p)
    def entry(p):
        got.append(ctypes.string_at(p, 32))
        return 7

    fn = ctypes.cast(entry, ctypes.c_void_p).value
    call = _tensor_args.call
    assert call(fn, b"bqnrnn", ("x",), 0, None, None, -5, 1 << 30, 0.25, -1, True) == 7
    assert got[0] == struct.pack("=Qqifii", 0, -5, 1 << 30, 0.25, -1, 1)
    t = torch.zeros(2, 3, dtype=torch.bfloat16)
    for bad, err in ((("B", ("x",), t, (2, 3)), TypeError),             # not on a GPU
                     (("B", ("x",), None, (2, 3)), TypeError),          # needed
                     (("S", ("x",), "text"), TypeError),
                     (("n", (), 1 << 31), ValueError), (("n", (), -(1 << 31) - 1), ValueError), (("q", (), 1 << 63), ValueError),
                     (("n", (), 1.5), TypeError), (("r", (), "1"), TypeError), (("n", ()), TypeError), (("n", (), 1, 2), TypeError),
                     (("z", (), 1), TypeError), (("b", (), None, None), TypeError), (("n" * 70, (), *range(70)), TypeError)):
        with pytest.raises(err):
            call(fn, bad[0].encode(), bad[1], 0, *bad[2:])
    assert len(got) == 1


def test_argument_packer_refuses_bad_numbers_of_bytes():
    """A number of bytes in a workspace's place goes with a stream's handle, and only there."""
    from head_attention_forward_fmha_gb300 import _tensor_args

    for layout, value, stream, err in ((b"uq", -1, 0, ValueError), (b"uq", 1 << 70, 0, OverflowError), (b"uq", 4096, None, TypeError),
                                       (b"uq", True, 0, TypeError), (b"Uq", 4096, 0, TypeError), (b"fq", 4096, 0, TypeError)):
        with pytest.raises(err):
            _tensor_args.call(1, layout, ("workspace",), 0, value, stream, 0)


@pytest.mark.parametrize("name", ["kv4", "first"])
def test_plans_are_those_of_the_tensors_device(name, monkeypatch):
    """Two devices of which the second plans twice the chunks: each call asks with its device current, and a plan kept for one
    is not taken on the other."""
    state = {"current": 0}

    class On:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.old, state["current"] = state["current"], self.dev

        def __exit__(self, *_):
            state["current"] = self.old

    got = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(binding, "_run", lambda entry, dev, *values: got.append((dev, values)))
    monkeypatch.setattr(binding, "_handle", lambda stream, dev: 0)
    monkeypatch.setattr(binding, "fmha_fwd_kv4_plan", lambda *a: (2 * (1 + state["current"]), 512))
    monkeypatch.setattr(binding, "fmha_fwd_first_workspace_bytes", lambda *a: 1000 * (1 + state["current"]))
    monkeypatch.setattr(binding, "_kv4_plans", {})
    monkeypatch.setattr(binding, "_first_plans", {})
    q, o, lse = torch.zeros(1, 8, 1, 128), torch.zeros(1, 8, 1, 128), torch.zeros(1, 8, 1)
    kv, cache = torch.zeros(1, 1, 64, 128), torch.zeros(1, 1, 64, 64)
    for dev in (0, 1, 0, 1):
        monkeypatch.setattr(binding, "_device", lambda t, name: dev)
        if name == "kv4":
            binding.fmha_fwd_kv4(q, cache, cache, cache, cache, o=o, lse=lse)
            need = binding.fmha_workspace_bytes(1, 8, 1, 128, 2 * (1 + dev))
        else:
            binding.fmha_fwd_first(q, kv, kv, 4, o=o, lse=lse, window=16)
            need = 1000 * (1 + dev)
        assert got[-1][0] == dev and need in [x for x in got[-1][1] if isinstance(x, int)]
        assert state["current"] == 0
    kept = binding._kv4_plans if name == "kv4" else binding._first_plans
    assert len(kept) == 2


def test_older_calls_need_no_argument_packer():
    """Without the packer the library loads and its other calls work; the serving calls say what is missing."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys
sys.modules["head_attention_forward_fmha_gb300._tensor_args"] = None  # importing it raises ImportError
import torch
from head_attention_forward_fmha_gb300 import binding
assert binding.fmha_fwd_plan(1, 8, 1, 1, 4096, 128)[0] >= 1 and binding.fmha_fwd_kv4_plan(1, 8, 1, 1, 4096, 128)[0] >= 1
torch._C._cuda_getDevice = lambda: 0
for entry in (binding._NORM_ROPE, binding._APPEND, binding._KV4, binding._FIRST):
    try:
        binding._run(entry, 0)
        raise SystemExit("no error")
    except ImportError as e:
        assert "_tensor_args" in str(e) and "build" in str(e), e
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


def test_libraries_are_built_without_a_host_compiler(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "ARGS_PATH", str(tmp_path / "_tensor_args.so"))
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.warns(UserWarning, match="packer was not built"):
        assert build.build() == build.LIB_PATH
    with pytest.raises(RuntimeError):
        build.build_args()


def test_index_check_sites_are_named_and_used():
    """Every site code stands at some check of a kernel and has a description; the serving kernels check what they access."""
    import glob
    import os

    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    text = {os.path.basename(p): open(p).read() for p in glob.glob(os.path.join(csrc, "*.cu*"))}
    enum = text["ptx.cuh"][text["ptx.cuh"].index("enum CheckSite") :]
    enum = enum[: enum.index("};")]
    sites = re.findall(r"^\s*(kSite\w+) = 0x", enum, re.M)
    assert len(sites) == len(set(sites)) > 40
    elsewhere = "".join(text.values()).replace(enum, "").replace(text["status.cu"], "")
    for site in sites:
        assert "case %s:" % site in text["status.cu"], site + " has no description"
        if site != "kSiteSelfTest":  # its check stands in status.cu
            assert re.search(r"\b%s\b" % site, elsewhere), site + " is checked nowhere"
    kv4 = {"Copy", "Key", "Comb", "Out", "Q"}
    for name, want in (("kv4_kernel.cu", kv4), ("kv4_tc_kernel.cu", kv4 | {"Tmem", "Desc", "Range"}), ("kv4_append_kernel.cu", {"Append"})):
        have = set(re.findall(r"kSiteKv4(\w+)", text[name] + text["kv4_common.cuh"]))
        assert want <= have, "%s: no check for %s" % (name, want - have)
    assert {"Col", "Row", "Table"} <= set(re.findall(r"kSiteNr(\w+)", text["qk_norm_rope_kernel.cu"]))
