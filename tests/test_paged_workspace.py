"""The workspace of the attention over a cache in pages: as many bytes as fmha_fwd_paged_plan's chunks need are enough for the
call with the same arguments, however many keys its block table holds and however many tokens a ragged batch has."""
import struct

import pytest
import torch

import paged_ref as ref
import test_paged_host as host
import test_paged_ops as ops
from head_attention_forward_fmha_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


kernel = ops.kernel  # fixture: both kernels of the attention


def planned(lib, c):
    """Chunks and workspace bytes by the plan, for arguments named as in test_paged_host.FWD."""
    ragged = c["cu"] is not None
    n = lib.fmha_fwd_paged_plan(c["batch"], c["T"], c["total"], c["n_h"], c["n_kv"], c["hd"], c["page"], c["s_k"], c["window"], c["n_first"],
                                c["causal"], int(ragged), int(c["ks"] is not None), c["n_splits"])
    assert n >= 1
    return n, lib.fmha_workspace_bytes(1, c["n_h"], c["total"] if ragged else c["batch"] * c["T"], c["hd"], n) if n > 1 else 0


# Calls whose bound on the keys is above what the table holds, by more than one chunk each: with a workspace of the planned size that
# is not aligned they are refused for that, not for its size.
@pytest.mark.parametrize("change", [
    dict(s_k=1088, page=64, width=16, n_splits=16), dict(s_k=1088, page=64, width=16, n_splits=16, ks=host.P, vs=host.P),
    dict(batch=1, hd=64, s_k=8192, width=64, window=1024, n_splits=0), dict(batch=1, n_h=8, hd=512, s_k=1 << 30, width=64, window=1000, n_splits=0),
    dict(batch=3, T=5, s_k=4000, page=64, width=48, window=2048, n_first=4, n_splits=64), dict(batch=2, cu=host.P, total=7, T=7, s_k=1088, page=64, width=16, n_splits=16),
    dict(batch=2, T=5, hd=256, n_h=256, n_kv=2, s_k=8192, page=256, width=16, window=4096, n_first=4, n_splits=64),
])
def test_planned_workspace_is_enough_under_a_short_table(lib, change):
    c = {**host.FWD, **change}
    n, need = planned(lib, c)
    assert n > 1
    assert host.call(lib, "fmha_fwd_paged", c, dict(ws=host.P + 8, wsb=need)) == -2, binding.fmha_get_last_error()


def run(lib, q, cache, table, lens, c, workspace):
    """fmha_fwd_paged through its C entry."""
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device=ops.DEV)
    at = [0 if t is None else t.data_ptr() for t in (q, *cache, table, lens)]
    x = {**c, **dict(zip(("q", "kp", "vp", "ks", "vs", "table", "lens"), at)), "o": o.data_ptr(), "lse": lse.data_ptr(),
         "q0": q.stride(0), "q1": q.stride(2), "q2": q.stride(1), "scale": c["hd"] ** -0.5, "ws": workspace.data_ptr(), "wsb": workspace.numel(),
         "stream": torch.cuda.current_stream().cuda_stream}
    rc = lib.fmha_fwd_paged(struct.pack(host.FORMATS["fmha_fwd_paged"], *[0 if v is None else v for v in x.values()]))
    assert rc == 0, binding.fmha_get_last_error()
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("form", ops.FORMS)
@pytest.mark.parametrize("s_k,window,n_splits", [(400, 0, 0), (1088, 0, 16), (8192, 0, 0), (8192, 300, 0), (1 << 30, 500, 0), (1088, 700, 64), (1 << 30, 0, 64)])
@pytest.mark.parametrize("T,hd", [(1, 64), (1, 128), (9, 512), (40, 128)])
def test_calls_with_a_planned_workspace(lib, T, hd, s_k, window, n_splits, form, kernel):
    """Bounds below and above the 400 keys that the table holds: the call runs, writes nothing behind the workspace, and is right."""
    g = ops.gen(T + hd)
    lens, n_h, n_kv, page = [400, 33, 0], 8, 2, 16
    cache, table = ops.pool(g, lens, n_kv, page, hd, form)
    q = ops.normal(g, 3, n_h, T, hd)
    c = {**host.FWD, "batch": 3, "T": T, "n_h": n_h, "n_kv": n_kv, "hd": hd, "n_pages": cache[0].shape[0], "width": table.shape[1], "s_k": s_k,
         "window": window, "n_splits": n_splits, "ks": None if cache[2] is None else 1}
    _, need = planned(lib, c)
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=ops.DEV)
    got = run(lib, q, cache, table, ops.ints(lens), c, room[:need])
    assert (room[need:] == 0xA5).all()
    ref.assert_attention(got, ref.attend(q, cache, table, lens, page, window=window, causal=True))


@pytest.mark.gpu
@pytest.mark.parametrize("s_k,window", [(1088, 0), (8192, 300)])
def test_binding_takes_a_planned_workspace(s_k, window, kernel):
    g = ops.gen(3)
    lens, page = [400, 33], 16
    cache, table = ops.pool(g, lens, 2, page, 128, ops.FORMS[0])
    q, n = ops.normal(g, 2, 8, 1, 128), ops.ints(lens)
    for splits in (0, 16):
        chunks = binding.fmha_fwd_paged_plan(2, 1, 8, 2, 128, page, s_k, window, 0, True, n_splits=splits)
        ws = torch.empty(binding.load().fmha_workspace_bytes(1, 8, 2, 128, chunks), dtype=torch.uint8, device=ops.DEV)
        for w in (ws, None):
            got = binding.fmha_fwd_paged(q, *cache, table, n, s_k=s_k, window=window, causal=True, n_splits=splits, workspace=w)
            ref.assert_attention(got, ref.attend(q, cache, table, lens, page, window=window, causal=True))


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("n_h,n_kv,hd", [(64, 8, 128), (8, 8, 64), (32, 4, 256), (128, 1, 512)])
def test_no_sequence_counts_more_tokens_than_there_are(n_h, n_kv, hd, codes):
    """max_q above the rows of q: the plan is that of the call, which cuts it to them."""
    for total in (1, 2, 7, 40):
        for window in (0, 1000):
            want = binding.fmha_fwd_paged_plan(3, total, n_h, n_kv, hd, 16, 8192, window, 4, True, total, codes)
            for T in (total + 1, 512, 1 << 20):
                assert binding.fmha_fwd_paged_plan(3, T, n_h, n_kv, hd, 16, 8192, window, 4, True, total, codes) == want


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [2, 3, 512])
def test_binding_takes_a_workspace_planned_for_max_q(max_q):
    """Two sequences of one token: a workspace planned for max_q tokens of a sequence."""
    g = ops.gen(4)
    lens, page = [4000, 33], 16
    cache, table = ops.pool(g, lens, 2, page, 128, ops.FORMS[0])
    q, n, cu = ops.normal(g, 2, 8, 128), ops.ints(lens), [0, 1, 2]
    chunks = binding.fmha_fwd_paged_plan(2, max_q, 8, 2, 128, page, 4000, causal=True, total=2)
    ws = torch.empty(binding.load().fmha_workspace_bytes(1, 8, 2, 128, chunks), dtype=torch.uint8, device=ops.DEV)
    got = binding.fmha_fwd_paged(q, *cache, table, n, cu_q=ops.ints(cu), max_q=max_q, s_k=4000, causal=True, workspace=ws)
    ref.assert_attention(got, ref.attend(q, cache, table, lens, page, cu, causal=True))
