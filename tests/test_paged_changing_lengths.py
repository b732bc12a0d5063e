"""Lengths, bounds and pages of the attention over a cache in pages that another stream rewrites while calls run: what such a call gives is
any value, but it ends, leaves the rows outside its batch alone, and the next call is right.  (A block's rows and keys are read by one
warp for all.)"""
import pytest
import torch

import paged_ref as ref
import test_paged_ops as ops
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu
_status, kernel = ops._status, ops.kernel  # fixtures: device status after each test, both kernels


@pytest.mark.parametrize("form", ops.FORMS)
@pytest.mark.parametrize("hd", ops.HD)
@pytest.mark.parametrize("n_splits", [1, 3])
def test_calls_end_while_their_lengths_change(hd, n_splits, form, kernel):
    g = ops.gen(hd)
    lens, new, page = [700, 0, 300, 1, 450], [40, 0, 1, 1, 130], 16
    cu = [2, 42, 42, 43, 44, 174]
    cache, table = ops.pool(g, lens, 2, page, hd, form)
    q = ops.normal(g, 180, 8, hd)
    n, at, pages = ops.ints(lens), ops.ints(cu), table.clone()
    states = [(ops.ints(x), ops.ints(y), t) for x, y, t in (
        (lens, cu, table), ([0, 700, 0, 2 ** 31 - 1, -5], [2, 2, 2, 174, 174, 174], torch.full_like(table, -1)),
        ([5, 5, 700, 700, 0], [2, 3, 170, 170, 171, 174], table.flip(0).contiguous()))]
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device=ops.DEV)

    def call():
        binding.fmha_fwd_paged(q, *cache, pages, n, cu_q=at, max_q=130, o=o, lse=lse, causal=True, n_splits=n_splits)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(60):
        with torch.cuda.stream(side):
            for x, y, t in states:
                n.copy_(x), at.copy_(y), pages.copy_(t)
        call()
    torch.cuda.synchronize()
    for a, b in ((0, 2), (174, 180)):
        assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
    n.copy_(states[0][0]), at.copy_(states[0][1]), pages.copy_(table)
    call()
    o[:2], o[174:], lse[:2], lse[174:] = 0, 0, 0, 0
    ref.assert_attention((o, lse), ref.attend(q, cache, table, lens, page, cu, causal=True))
