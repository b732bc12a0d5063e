"""Scores that rise above a row's first ones over large values: O is summed in fp32 before its division, and what |V| times the number
of keys times 2^8 (the most by which a score may pass its row's reference before that moves) leaves below 2^128 comes out finite, on
both kernels of the attention over a cache in pages.  64-bit references and bounds are those of tests/paged_ref.py."""
import pytest
import torch

import paged_ref as ref
import test_paged_ops as ops
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu
_status, kernel = ops._status, ops.kernel  # fixtures: device status after each test, both kernels


@pytest.mark.parametrize("form", ops.FORMS)
@pytest.mark.parametrize("hd", ops.HD)
@pytest.mark.parametrize("T", [1, 20, 40])  # rows of one row tile, of two at hd 64 and 128
@pytest.mark.parametrize("rise", [7.5, 9.0, 38.0, 39.9, 200.0])  # log2 of a later weight over the first ones
@pytest.mark.parametrize("size", [90, 108])  # log2 of V
def test_large_values_under_rising_scores(hd, T, rise, size, form, kernel):
    g = ops.gen(hd + T)
    n, page = 500, 32
    cache, table = ops.blank(17, 2, page, hd, form), ops.ints([list(range(16, 0, -1))])
    k, v = ops.normal(g, n, 2, hd) * 0.1, (ops.normal(g, n, 2, hd) * 2.0 ** size)
    k[:, :, 0] = 0.0
    k[150:, :, 0] = 1.0  # the first tile, or two, and later keys that weigh 2^rise as much
    q = ops.normal(g, 1, 8, T, hd)
    q[..., 0] = rise * 0.6931471805599453
    binding.fmha_paged_append(k, v, *cache, table, ops.ints([0]), cu_q=ops.ints([0, n]))
    for n_splits in (1, 0):
        got = binding.fmha_fwd_paged(q, *cache, table, ops.ints([n]), scale=1.0, n_splits=n_splits)
        assert torch.isfinite(got[0]).all()
        ref.assert_attention(got, ref.attend(q, cache, table, [n], page, scale=1.0))
