"""Edges of the serving operators on the GPU: the ends of the number range, NaN, other streams, memory
that outlives a call.  64-bit references and bounds are those of tests/serving_ref.py."""
import pytest
import torch

import serving_ref as ref
import test_serving_ops as ops
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
kernel, _status = ops.kernel, ops._status  # fixtures: both 4-bit kernels; the status word after each test


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("g", [1e-4, 2.0 ** -10, 2.0 ** -80, 2.0 ** -120, 1.0, 2.0 ** 100])
def test_append_of_values_far_above_saturation(hd, g):
    """Codes, scales and values are those of the block quantiser where x / (g s) passes fp32's range: -6 stays -6."""
    r = ops.gen(hd)
    T, cap = 8, 16
    k, v = ops.normal(r, 1, 2, T, hd), ops.normal(r, 1, 2, T, hd)
    for t, big in enumerate((3e38, 2e38, 1e30, 1e20, 1e10)):
        k[0, 0, t, 3], k[0, 0, t, 17], k[0, 0, t, 18] = -big, big, -big
        v[0, 1, t, :16] *= -big
    k[0, 1, 0], k[0, 1, 1] = -3e38, 3e38
    k[0, 1, 2, ::2], k[0, 1, 3] = -float("inf"), float("inf")
    k[0, 1, 4, 5], k[0, 1, 5] = float("nan"), float("nan")
    k[0, 1, 6], k[0, 1, 7] = (k[0, 1, 6].float() * 700 * g).to(k.dtype), -2688 * g  # around the largest scale, and at it
    cache = binding.fmha_kv4_cache(1, 2, cap, hd)
    out = torch.zeros_like(k), torch.zeros_like(v)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(1, dtype=torch.int32, device=DEV), k_global=g, v_global=g, k_out=out[0], v_out=out[1])
    for x, codes, scales, o in ((k, cache[0], cache[1], out[0]), (v, cache[2], cache[3], out[1])):
        c, s = binding.fmha_quantize_nvfp4(x.float(), global_scale=g)
        assert torch.equal(codes[:, :, :T], c) and torch.equal(scales[:, :, :T], s)
        values = ref.dequantise(c, s, 1.0).float() * torch.tensor(g, dtype=torch.float32, device=DEV)
        assert torch.equal(o, values.to(torch.bfloat16))
    assert (cache[0][0, 1, 0] == 0xFF).all() and (cache[0][0, 1, 1] == 0x77).all()


# ------------------------------------------------------------------ NaN in attended places
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("kv_chunk", [1024, 512, 256, 128])
@pytest.mark.parametrize("sink", [False, True])
def test_kv4_nan_scores_show_whatever_the_chunks(hd, kv_chunk, sink, kernel):
    """A NaN in a query row, or in the scale of an attended key: NaN in O and in LSE of the rows that meet it, and only
    there, with 1, 2, 4 and 8 chunks.  Sequences of one chunk beside it leave the others empty."""
    r = ops.gen(hd)
    lens, cap, n_h, n_kv, T = [1024, 700, 100, 0], 1024, 4, 2, 2
    cache = ops.filled(r, len(lens), n_kv, cap, hd)
    q = ops.normal(r, len(lens), n_h, T, hd)
    sg = torch.randn(n_h, generator=r, device=DEV) * 2 if sink else None
    want = ref.attend(q, ref.dequantise(cache[0], cache[1], 1.0), ref.dequantise(cache[2], cache[3], 2.0), lens, hd ** -0.5, causal=True, sink=sg)
    ops.spoil(cache, lens)
    bad = torch.zeros((len(lens), n_h, T), dtype=torch.bool, device=DEV)
    q[1, 2, 1, 5] = float("nan")
    q[2, 1, 0] = float("nan")
    cache[1][0, 1, 300, 2] = 0x7F
    bad[1, 2, 1] = bad[2, 1, 0] = bad[0, 2:] = True
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    n, _ = binding.fmha_fwd_kv4_plan(len(lens), n_h, n_kv, T, cap, hd, causal=True, kv_chunk=kv_chunk)
    assert n == cap // kv_chunk
    o, lse = binding.fmha_fwd_kv4(q, *cache, ln, v_global=2.0, causal=True, sink=sg, kv_chunk=kv_chunk)
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    keep = ~bad
    (ro, rl, o_tol, l_tol) = want
    assert ((o.double() - ro).abs() <= o_tol)[keep].all()
    fin = keep & torch.isfinite(rl)
    assert torch.equal(torch.isinf(lse[keep]), torch.isinf(rl[keep])) and ((lse.double() - rl).abs() <= l_tol)[fin].all()


# ------------------------------------------------------------------ factors of the scores at the ends of fp32
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("kv_chunk", [0, 64])
def test_kv4_score_factors_past_the_range_of_fp32(hd, kv_chunk, kernel):
    """Rows so small that their factor underflows (every key weighs the same then), masked keys beside them; and products of
    scale and global scale below fp32's smallest number."""
    lens = [0, 7, 200, 256]
    ops.check_kv4(hd, 8, 2, 2, 256, lens, g=2.0 ** -40, q_mult=2.0 ** -100, causal=True, kv_chunk=kv_chunk)
    ops.check_kv4(hd, 8, 2, 2, 256, lens, g=2.0 ** -40, q_mult=2.0 ** -100, window=50, n_first=3, kv_chunk=kv_chunk)
    ops.check_kv4(hd, 8, 2, 2, 256, lens, g=2.0 ** -40, scale=2.0 ** -130, causal=True, sink=True, kv_chunk=kv_chunk)
    ops.check_kv4(hd, 8, 2, 2, 256, lens, g=2.0 ** -40, scale=2.0 ** -115, q_mult=2.0 ** 110, causal=True, kv_chunk=kv_chunk)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_kv4_keys_of_zero_under_a_factor_past_fp32(hd, kernel):
    """K is zero and every score 0, however large Q, scale and global scale are: the mean of V."""
    r = ops.gen(hd)
    lens = [5, 256, 130]
    cache = ops.filled(r, 3, 2, 256, hd)
    cache[0].zero_()
    q = ops.normal(r, 3, 8, 2, hd) * 2.0 ** 110
    got = binding.fmha_fwd_kv4(q, *cache, torch.tensor(lens, dtype=torch.int32, device=DEV), k_global=2.0 ** 60, v_global=2.0, scale=2.0 ** 20)
    want = ref.attend(q, torch.zeros(3, 2, 256, hd, device=DEV), ref.dequantise(cache[2], cache[3], 2.0), lens, 1.0)
    ref.assert_attention(got, want)


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
def test_kv4_scores_that_rise_within_every_tile(hd, kernel):
    """The reference moves in every tile after its weights have been written once, for some rows of a warp and not for others."""
    n, rows = 1024, 40
    r = ops.gen(93)
    k, v, q = ops.normal(r, 1, 1, n, hd) * 0.1, ops.normal(r, 1, 1, n, hd), ops.normal(r, 1, rows, 1, hd)
    k[0, 0, :, 0] = torch.linspace(0, 96, n, device=DEV).to(torch.bfloat16)
    q[0, :, 0, 0] = torch.linspace(-4, 0.5 * hd ** 0.5 * 4, rows, device=DEV).to(torch.bfloat16)
    cache = binding.fmha_kv4_cache(1, 1, n, hd)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    want = ref.attend(q, ref.dequantise(cache[0], cache[1], 1.0), ref.dequantise(cache[2], cache[3], 1.0), [n], hd ** -0.5)
    for chunk in (0, 1024):
        ref.assert_attention(binding.fmha_fwd_kv4(q, *cache, kv_chunk=chunk), want)


# ------------------------------------------------------------------ other streams
def _calls(r, hd=128):
    """Calls that allocate their outputs, each as a function of the stream: (name, outputs)."""
    q, k, v = ops.normal(r, 2, 8, 1, hd), ops.normal(r, 2, 2, 600, hd), ops.normal(r, 2, 2, 600, hd)
    cache = ops.filled(r, 2, 2, 608, hd)
    qkv, tab = ops.normal(r, 2, 1, 12 * hd), ops.table(16, hd)
    pos = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    parts = binding.fmha_fwd_splitkv(q, k, v, 200)
    q5, k5, v5 = ops.normal(r, 1, 64, 1, 512), ops.normal(r, 1, 1, 600, 512), ops.normal(r, 1, 1, 600, 512)
    parts16 = binding.fmha_fwd_splitkv_f16(q5, k5, v5, 256)
    return {
        "norm_rope": lambda s: binding.fmha_qk_norm_rope(qkv, tab, pos, 8, 2, stream=s),
        "kv4": lambda s: binding.fmha_fwd_kv4(q, *cache, stream=s),
        "first": lambda s: binding.fmha_fwd_first(q, k, v, 4, window=500, stream=s),
        "fwd": lambda s: binding.fmha_fwd(q, k, v, stream=s),
        "nvfp4": lambda s: binding.fmha_fwd_nvfp4(q, k, v, stream=s),
        "splitkv": lambda s: binding.fmha_fwd_splitkv(q, k, v, 200, stream=s),
        "merge": lambda s: binding.fmha_merge(*parts, stream=s),
        "splitkv_f16": lambda s: binding.fmha_fwd_splitkv_f16(q5, k5, v5, 256, stream=s),
        "merge_f16": lambda s: binding.fmha_merge_f16(*parts16, stream=s),
        "quantize": lambda s: binding.fmha_quantize_nvfp4(parts[0], stream=s),
    }


CALLS = ["norm_rope", "kv4", "first", "fwd", "nvfp4", "splitkv", "merge", "splitkv_f16", "merge_f16", "quantize"]
STREAMS = ["stream", "handle", "default handle"]


def _lanes(how):
    """(the current stream of the test, what a call is given as its stream, that as a Stream)"""
    if how == "default handle":
        return torch.cuda.Stream(), 0, torch.cuda.default_stream()
    side = torch.cuda.Stream()
    return torch.cuda.default_stream(), side if how == "stream" else side.cuda_stream, side


def _bits(out):
    return [t.clone().view(torch.uint8) for t in out]


@pytest.mark.parametrize("how", STREAMS)
@pytest.mark.parametrize("name", CALLS)
def test_outputs_do_not_take_memory_that_the_current_stream_still_uses(name, how):
    """Blocks freed on the current stream, which copies from them later, beside a call on another stream that allocates."""
    here, given, side = _lanes(how)
    call = _calls(ops.gen(90))[name]
    sizes = [t.shape + (t.element_size(),) for t in call(None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        olds = [torch.full(s, 7, dtype=torch.uint8, device=DEV) for s in sizes]
        news = [torch.empty_like(t) for t in olds]
        here.synchronize()
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
        for o, n in zip(olds, news):
            n.copy_(o)
        del o, olds
        outs = call(given)
    side.synchronize()
    torch.cuda.synchronize()
    assert len(outs) == len(news) and all((n == 7).all() for n in news)


@pytest.mark.parametrize("how", STREAMS)
@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_kept_for_the_current_stream_too(name, how):
    """Outputs of a call on another stream, read on the current one, dropped before that has happened, and the same call again."""
    here, given, side = _lanes(how)
    call = _calls(ops.gen(91))[name]
    want = _bits(call(None))
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        outs = call(given)
        here.wait_stream(side)
        torch.cuda._sleep(200_000_000)
        got = _bits(outs)
        del outs
        with torch.cuda.stream(side):
            other = [torch.full_like(w, 9) for w in want]  # takes such blocks if they are free
        side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and all((t == 9).all() for t in other)


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_a_stream_that_a_capture_forks(name):
    """Captured on a side stream that joins the capture, outputs and workspaces allocated by the calls; replayed twice."""
    call = _calls(ops.gen(97))[name]
    want = _bits(call(None))
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        outs = [call(side) for _ in range(2)]
        here.wait_stream(side)
    for _ in range(2):
        for out in outs:
            for t in out:
                t.view(torch.uint8).fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(g, w) for g, w in zip(_bits(out), want))


# ------------------------------------------------------------------ memory that outlives a call
@pytest.mark.parametrize("name", ["kv4", "first"])
def test_split_calls_keep_no_memory(name):
    """Partials belong to the call: threads and streams that come and go leave nothing behind, nor does a call whose
    allocations go to a pool of their own, as in a compiled program's graph mode."""
    import threading

    r = ops.gen(92)
    q, o, lse = ops.normal(r, 1, 8, 1, 128), torch.empty(1, 8, 1, 128, dtype=torch.bfloat16, device=DEV), torch.empty(1, 8, 1, device=DEV)
    k, v = ops.normal(r, 1, 1, 8192, 128), ops.normal(r, 1, 1, 8192, 128)
    cache = ops.filled(r, 1, 1, 8192, 128)
    assert binding.fmha_fwd_kv4_plan(1, 8, 1, 1, 8192, 128, ragged=False)[0] > 1
    assert binding.fmha_fwd_first_workspace_bytes(1, 8, 1, 1, 8192, 128, 8000, 4) > 0

    def call(stream=None):
        if name == "kv4":
            binding.fmha_fwd_kv4(q, *cache, o=o, lse=lse, stream=stream)
        else:
            binding.fmha_fwd_first(q, k, v, 4, window=8000, o=o, lse=lse, stream=stream)

    call()
    torch.cuda.synchronize()
    binding.fmha_release()
    before = torch.cuda.memory_allocated()

    def work():
        side = torch.cuda.Stream()
        torch.cuda.synchronize()  # this thread's context
        call()
        call(side)
        with torch.cuda.stream(side):
            call()
        side.synchronize()

    for _ in range(3):
        threads = [threading.Thread(target=work) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    pool = torch.cuda.MemPool()
    with torch.cuda.use_mem_pool(pool):
        call()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


def test_split_calls_in_a_compiled_program_with_graphs():
    """torch.compile's graph mode (a warm-up in its own memory pool, a capture, replays), eager calls in between."""
    from head_attention_forward_fmha_gb300 import torch_op  # noqa: F401  (registers the ops)

    r = ops.gen(94)
    cache, k, v = ops.filled(r, 1, 1, 8192, 128), ops.normal(r, 1, 1, 8192, 128), ops.normal(r, 1, 1, 8192, 128)
    lens = torch.tensor([8100], dtype=torch.int32, device=DEV)

    def program(q):
        a = torch.ops.fmha_gb300.fwd_kv4(q * 1.0, *cache, lens, 1.0, 2.0, 128 ** -0.5, 0, 0, False)
        b = torch.ops.fmha_gb300.fwd_first(q * 1.0, k, v, 4, 128 ** -0.5, 8000, False)
        return a[0] * 1.0, a[1], b[0] * 1.0, b[1]

    compiled = torch.compile(program, mode="reduce-overhead", fullgraph=True)
    for _ in range(6):
        q = ops.normal(r, 1, 8, 1, 128)
        torch.compiler.cudagraph_mark_step_begin()
        got = [t.clone() for t in compiled(q)]
        want = program(q)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_a_workspace_that_does_not_fit_is_torchs_error():
    """More partials than the device has memory for: torch.OutOfMemoryError, nothing launched, and the next call works."""
    r = ops.gen(96)
    q, cache = ops.normal(r, 1, 8, 1, 128), ops.filled(r, 1, 1, 256, 128)
    entry, names = binding._packed["fmha_fwd_kv4"], binding._KV4[2]
    binding.fmha_fwd_kv4(q, *cache)
    o, lse = torch.zeros_like(q), torch.zeros(1, 8, 1, device=DEV)
    with pytest.raises(torch.OutOfMemoryError):
        binding._call(entry, binding._KV4[1], names, 0, q, None, *[x for t in cache for x in (t, None)], None, None, o, None, lse, None,
                      None, None, 1 << 45, 0, 1 << 45, 0, 1.0, 1.0, 0.1, 1, 8, 1, 1, 256, 256, 128, 0, 0, 0, 0)
    torch.cuda.synchronize()
    assert (o == 0).all() and (lse == 0).all()
    a, b = binding.fmha_fwd_kv4(q, *cache), binding.fmha_fwd_kv4(q, *cache)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("name", ["norm_rope", "append", "kv4", "first", "fwd", "splitkv", "noalloc", "nvfp4"])
def test_first_call_of_a_fresh_thread(name):
    """A thread that has made no CUDA call yet."""
    import threading

    r = ops.gen(95)
    q, k, v = ops.normal(r, 1, 8, 1, 128), ops.normal(r, 1, 1, 8192, 128), ops.normal(r, 1, 1, 8192, 128)
    o, lse, cache = torch.empty_like(q), torch.empty(1, 8, 1, device=DEV), ops.filled(r, 1, 1, 8192, 128)
    qkv, pos, tab = ops.normal(r, 1, 1, 10 * 128), torch.zeros(1, 1, dtype=torch.int32, device=DEV), ops.table(16, 128)
    start, ws = torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
    k1, v1 = (torch.empty(1, 1, 1, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    parts = torch.empty(8, 1, 8, 1, 128, device=DEV), torch.empty(8, 1, 8, 1, device=DEV)
    codes = [torch.empty(1, 8, 1, 128 // w, dtype=torch.uint8, device=DEV) for w in (2, 16)]
    here = torch.cuda.current_stream().cuda_stream
    calls = {
        "norm_rope": lambda: binding.fmha_qk_norm_rope(qkv, tab, pos, 8, 1, q=q, k=k1, v=v1, stream=here),
        "append": lambda: binding.fmha_kv4_append(k, v, *cache, start, stream=here),
        "kv4": lambda: binding.fmha_fwd_kv4(q, *cache, o=o, lse=lse, workspace=ws, stream=here),
        "first": lambda: binding.fmha_fwd_first(q, k, v, 4, window=8000, o=o, lse=lse, workspace=ws, stream=here),
        "fwd": lambda: binding.fmha_fwd(q, k, v, o=o, lse=lse, stream=here),
        "splitkv": lambda: binding.fmha_fwd_splitkv(q, k, v, 1024, *parts, stream=here),
        "noalloc": lambda: binding.fmha_fwd_noalloc(q, k, v, o, lse, stream=here),
        "nvfp4": lambda: binding.fmha_fwd_nvfp4(q, k, v, *codes, lse, stream=here),
    }
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            calls[name]()
        except Exception as e:  # shown by the test
            raised.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised, raised


def test_smoke_runs_a_kernel_with_first_keys(monkeypatch):
    """The smoke run's call with first keys has a window that hides some of them."""
    import __graft_entry__ as entry

    seen, real = [], binding.fmha_fwd_first

    def record(q, k, v, n_first, **kw):
        seen.append(0 < n_first < k.shape[2] - q.shape[2] - kw.get("window", 0) + 1 and kw.get("window", 0) > 0)
        return real(q, k, v, n_first, **kw)

    monkeypatch.setattr(binding, "fmha_fwd_first", record)
    entry.smoke()
    assert seen and all(seen)
