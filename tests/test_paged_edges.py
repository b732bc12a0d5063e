"""Calls of the cache in pages in the ways a program makes them: as custom ops, on other streams, in captures that fork,
from fresh threads, and the memory that they leave.  64-bit references and bounds are those of tests/paged_ref.py."""
import threading

import pytest
import torch

import paged_ref as ref
import test_paged_ops as ops
import test_serving_edges as edges
from head_attention_forward_fmha_gb300 import binding, torch_op  # noqa: F401  (registers the ops)

DEV = "cuda"
FORMS = ops.FORMS
kernel = ops.kernel  # fixture: both kernels of the attention


@pytest.fixture(autouse=True)
def _status(request):
    yield
    if request.node.get_closest_marker("gpu"):
        torch.cuda.synchronize()
        binding.fmha_check_device_status()


# ------------------------------------------------------------------ custom ops
@pytest.mark.parametrize("codes", [False, True])
def test_ops_have_fake_shapes(codes):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        pages = torch.empty((9, 2, 16, 128), dtype=torch.uint8 if codes else torch.bfloat16)
        scales = torch.empty((9, 2, 16), dtype=torch.uint8) if codes else None
        table, lens = torch.empty((3, 4), dtype=torch.int32), torch.empty(3, dtype=torch.int32)
        q, new = torch.empty((3, 8, 5, 128), dtype=torch.bfloat16), torch.empty((7, 2, 128), dtype=torch.bfloat16)
        o, lse = torch.ops.fmha_gb300.fwd_paged(q, pages, pages, scales, scales, table, lens, None, None, 0.1, 0, 0, True)
        r, rl = torch.ops.fmha_gb300.fwd_paged(q[0].transpose(0, 1), pages, pages, scales, scales, table, lens, torch.empty(4, dtype=torch.int32), 2, 0.1, 8, 1, True, torch.empty(8))
        k, v = torch.ops.fmha_gb300.paged_gather(pages, pages, scales, scales, table, lens, 33)
        other = torch.empty_like(pages), None if scales is None else torch.empty_like(scales)
        assert torch.ops.fmha_gb300.paged_append(new, new, pages, other[0], scales, other[1], table, lens, torch.empty(4, dtype=torch.int32)) is None
    assert o.shape == (3, 8, 5, 128) and lse.shape == (3, 8, 5) and r.shape == (5, 8, 128) and rl.shape == (5, 8) and k.shape == v.shape == (3, 2, 33, 128)
    assert r.is_contiguous() and {o.dtype, r.dtype, k.dtype, v.dtype} == {torch.bfloat16} and lse.dtype == rl.dtype == torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_ops_eager_and_compiled_match(form):
    """A step (append, attend, gather) under torch.compile: the same cache and outputs as eagerly."""
    g = ops.gen(41)
    lens = [40, 7, 90]
    cache, table = ops.pool(g, lens, 2, 16, 128, form, width=8)
    for i, n in enumerate(lens):   # a page more for each
        table[i, -(-n // 16)] = 10 + i
    n = max(13, int(table.max()) + 1)
    cache = [None if t is None else torch.cat([t, torch.zeros_like(t)])[: n + 4].contiguous() for t in cache]
    start, end, cu = ops.ints(lens), ops.ints([x + 3 for x in lens]), ops.ints([0, 3, 6, 9])
    k, v, q = ops.normal(g, 9, 2, 128), ops.normal(g, 9, 2, 128), ops.normal(g, 9, 8, 128)

    def step(q, k, v, *cache):
        torch.ops.fmha_gb300.paged_append(k, v, *cache, table, start, cu)
        o, lse = torch.ops.fmha_gb300.fwd_paged(q * 1.0, *cache, table, end, cu, 3, 128 ** -0.5, 0, 0, True)
        kk, vv = torch.ops.fmha_gb300.paged_gather(*cache, table, end, 96)
        return o * 1.0, lse, kk, vv

    one, two = ([None if t is None else t.clone() for t in cache] for _ in range(2))
    a = step(q, k, v, *one)
    b = torch.compile(step, backend="aot_eager", fullgraph=True)(q, k, v, *two)
    torch.cuda.synchronize()
    for x, y in zip(list(a) + one, list(b) + two):
        assert (x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert not torch.equal(one[0].view(torch.uint8), cache[0].view(torch.uint8))
    ends = [x + 3 for x in lens]
    ref.assert_attention(a[:2], ref.attend(q, one, table, ends, 16, [0, 3, 6, 9], causal=True))


# ------------------------------------------------------------------ padded batches
@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hd", ops.HD)
@pytest.mark.parametrize("T,window", [(9, 0), (9, 3), (40, 0), (300, 100)])
def test_more_tokens_than_keys(hd, T, window, form, kernel):
    """Sequences with fewer keys than new tokens: the first rows stand before the first key and attend nothing."""
    ops.check(ops.gen(50), hd, 8, 2, T, [4, 0, T, 2 * T, 1, T + 1], 16, form, window=window, n_first=min(window, 2), causal=True)
    ops.check(ops.gen(51), hd, 8, 2, T, [4, 0, T - 1, 200], 16, form, window=window, n_first=min(window, 2), sink=True, n_splits=2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("b,pad", [(64, (0, 0)), (65, (3, 2)), (200, (0, 5)), (1100, (130, 1))])
def test_batches_on_both_sides_of_the_search(b, pad, form, kernel):
    """Ragged batches whose sequences a block looks through and such in which it searches, some of them empty."""
    new = [(i * 7) % 11 if i % 5 else 0 for i in range(b)]
    new[b // 2], new[-1] = 300, 0
    ops.check(ops.gen(54), 64, 4, 1, None, [n + (i * 13) % 50 for i, n in enumerate(new)], 16, form, new=new, pad=pad, causal=True)
    new = [1 + (i % 17 == 0) * 40 for i in range(b)]
    ops.check(ops.gen(55), 128, 8, 2, None, [n + i % 70 for i, n in enumerate(new)], 16, form, new=new, pad=pad, causal=True, n_splits=2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_subnormal_queries(form, kernel):
    """Query rows whose largest magnitude is a subnormal bf16 over keys large enough for it to count."""
    ops.check(ops.gen(52), 128, 8, 2, 1, [100, 37], 16, form, q_mult=2.0 ** -129, k_mult=2.0 ** 121)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_appended_tokens_that_share_a_row_leave_the_others_alone(form):
    """Two sequences that write the same row of the pool: that row is undefined, every other one is as it was or as written."""
    g = ops.gen(53)
    cache = ops.blank(4, 2, 16, 64, form)
    before = [None if t is None else t.clone() for t in cache]
    table, k = ops.ints([[1], [1], [2]]), ops.normal(g, 3, 2, 1, 64)
    binding.fmha_paged_append(k, k, *cache, table, ops.ints([5, 5, 3]))
    one = ops.blank(4, 2, 16, 64, form)
    binding.fmha_paged_append(k[2:], k[2:], *one, table[2:].contiguous(), ops.ints([3]))
    for a, b, c in zip(cache, one, before):
        if a is not None:
            a, b, c = (x.view(torch.uint8) for x in (a, b, c))
            b[1, :, 5] = a[1, :, 5]
            assert torch.equal(a, b) and not torch.equal(b[2], c[2])


# ------------------------------------------------------------------ streams
CALLS = ["attend", "attend split", "attend codes", "attend rows", "gather", "gather codes"]


def _calls(g):
    """Calls that allocate their outputs (and partials), as functions of the stream."""
    lens = [600, 350]
    bf, table = ops.pool(g, lens, 2, 16, 128, FORMS[0])
    codes, table8 = ops.pool(g, lens, 2, 16, 128, FORMS[1])
    q, rows, n = ops.normal(g, 2, 8, 1, 128), ops.normal(g, 2, 8, 40, 128), ops.ints(lens)
    return {
        "attend": lambda s: binding.fmha_fwd_paged(q, *bf, table, n, n_splits=1, stream=s),
        "attend split": lambda s: binding.fmha_fwd_paged(q, *bf, table, n, n_splits=4, stream=s),
        "attend codes": lambda s: binding.fmha_fwd_paged(q, *codes, table8, n, n_splits=4, stream=s),
        "attend rows": lambda s: binding.fmha_fwd_paged(rows, *codes, table8, n, causal=True, n_splits=2, stream=s),
        "gather": lambda s: binding.fmha_paged_gather(*bf, table, n, 610, stream=s),
        "gather codes": lambda s: binding.fmha_paged_gather(*codes, table8, n, 610, stream=s),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("how", edges.STREAMS)
@pytest.mark.parametrize("name", CALLS)
def test_outputs_on_another_stream(name, how):
    """Blocks freed on the current stream, which copies from them later, are not taken; outputs read on the current stream and
    dropped before that has happened are not given away."""
    here, given, side = edges._lanes(how)
    call = _calls(ops.gen(90))[name]
    want = edges._bits(call(None))
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        olds = [torch.full_like(w, 7) for w in want]
        news = [torch.empty_like(t) for t in olds]
        here.synchronize()
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
        for o, n in zip(olds, news):
            n.copy_(o)
        del o, olds
        outs = call(given)
        here.wait_stream(side)
        got = edges._bits(outs)
        del outs
        with torch.cuda.stream(side):
            other = [torch.full_like(w, 9) for w in want]
        side.synchronize()
    torch.cuda.synchronize()
    assert all((n == 7).all() for n in news) and all((t == 9).all() for t in other)
    assert all(torch.equal(x, w) for x, w in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_calls_on_a_stream_that_a_capture_forks(name):
    call = _calls(ops.gen(97))[name]
    want = edges._bits(call(None))
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
            assert all(torch.equal(x, w) for x, w in zip(edges._bits(out), want))


@pytest.mark.gpu
def test_two_graphs_of_split_calls_replayed_together():
    """Two captures on two streams, each with its own partials, their replays in flight at once."""
    g = ops.gen(98)
    lens = [3000, 2000]
    cache, table = ops.pool(g, lens, 2, 16, 128, FORMS[1])
    n, qs = ops.ints(lens), [ops.normal(g, 2, 8, 1, 128) for _ in range(2)]
    want = [edges._bits(binding.fmha_fwd_paged(q, *cache, table, n, n_splits=8)) for q in qs]
    torch.cuda.synchronize()
    graphs, streams, outs = [torch.cuda.CUDAGraph() for _ in qs], [torch.cuda.Stream() for _ in qs], []
    for graph, stream, q in zip(graphs, streams, qs):
        with torch.cuda.graph(graph, stream=stream):
            outs.append(binding.fmha_fwd_paged(q, *cache, table, n, n_splits=8))
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(edges._bits(out), w))


# ------------------------------------------------------------------ memory that outlives a call, threads
@pytest.mark.gpu
def test_split_calls_keep_no_memory():
    g = ops.gen(92)
    cache, table = ops.pool(g, [8000], 1, 64, 128, FORMS[0])
    q, o, lse, n = ops.normal(g, 1, 8, 1, 128), torch.empty(1, 8, 1, 128, dtype=torch.bfloat16, device=DEV), torch.empty(1, 8, 1, device=DEV), ops.ints([8000])
    assert binding.fmha_fwd_paged_plan(1, 1, 8, 1, 128, 64, 8000) > 1

    def call(stream=None):
        binding.fmha_fwd_paged(q, *cache, table, n, o=o, lse=lse, stream=stream)

    call()
    torch.cuda.synchronize()
    binding.fmha_release()
    before = torch.cuda.memory_allocated()

    def work():
        side = torch.cuda.Stream()
        torch.cuda.synchronize()  # this thread's context
        call()
        call(side)
        side.synchronize()

    for _ in range(3):
        threads = [threading.Thread(target=work) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["append", "gather", "attend", "attend rows"])
def test_first_call_of_a_fresh_thread(name):
    g = ops.gen(95)
    cache, table = ops.pool(g, [8000], 1, 64, 128, FORMS[1])
    q, rows, n, k = ops.normal(g, 1, 8, 1, 128), ops.normal(g, 1, 8, 40, 128), ops.ints([8000]), ops.normal(g, 1, 1, 1, 128)
    out, ws = torch.empty(1, 1, 64, 128, dtype=torch.bfloat16, device=DEV), torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
    o, lse, here = torch.empty_like(rows), torch.empty(1, 8, 40, device=DEV), torch.cuda.current_stream().cuda_stream
    o1, lse1 = torch.empty_like(q), torch.empty(1, 8, 1, device=DEV)
    calls = {
        "append": lambda: binding.fmha_paged_append(k, k, *cache, table, n, stream=here),
        "gather": lambda: binding.fmha_paged_gather(*cache, table, n, 64, k=out, v=torch.empty_like(out), stream=here),
        "attend": lambda: binding.fmha_fwd_paged(q, *cache, table, n, o=o1, lse=lse1, workspace=ws, stream=here),
        "attend rows": lambda: binding.fmha_fwd_paged(rows, *cache, table, n, o=o, lse=lse, workspace=ws, stream=here),
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


@pytest.mark.gpu
def test_a_workspace_that_does_not_fit_is_torchs_error(monkeypatch):
    """More partials than the device has memory for: torch.OutOfMemoryError, nothing launched, and the next call works."""
    g = ops.gen(96)
    cache, table = ops.pool(g, [256], 1, 16, 128, FORMS[0])
    q, n = ops.normal(g, 1, 8, 1, 128), ops.ints([256])
    o, lse = torch.zeros_like(q), torch.zeros(1, 8, 1, device=DEV)
    want = binding.fmha_fwd_paged(q, *cache, table, n, n_splits=2)
    binding._paged_plans.clear()
    monkeypatch.setattr(binding, "_paged_plan", lambda *a: (2, 1 << 45))
    with pytest.raises(torch.OutOfMemoryError):
        binding.fmha_fwd_paged(q, *cache, table, n, n_splits=2, o=o, lse=lse)
    monkeypatch.undo()
    binding._paged_plans.clear()
    torch.cuda.synchronize()
    assert (o == 0).all() and (lse == 0).all()
    got = binding.fmha_fwd_paged(q, *cache, table, n, n_splits=2)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
def test_smoke_runs_both_kernels_and_forms(monkeypatch):
    import __graft_entry__ as entry

    seen, real = set(), binding.fmha_fwd_paged

    def record(q, k_pages, v_pages, k_scales, *a, **kw):
        seen.add((q.shape[1] * q.shape[2] // k_pages.shape[1] > 40, k_scales is not None))
        return real(q, k_pages, v_pages, k_scales, *a, **kw)

    monkeypatch.setattr(binding, "fmha_fwd_paged", record)
    entry.smoke()
    assert len(seen) == 4
