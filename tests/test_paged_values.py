"""The ends of the number range in the attention over a cache in pages: values as large as O's fp32 sum allows (|V| times the number of
keys times 2^8, the most by which a weight may pass its row's reference, below 2^128), and scores of ordinary size from factors that are
far from it, on both kernels.  64-bit references and bounds are those of tests/paged_ref.py."""
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


@pytest.mark.parametrize("form", ops.FORMS)
@pytest.mark.parametrize("hd", ops.HD)
@pytest.mark.parametrize("q_mult,k_mult,scale", [(2.0 ** -100, 2.0 ** -12, 2.0 ** 111), (1.0, 2.0 ** 100, 2.0 ** -103), (2.0 ** -90, 2.0 ** 90, 0.2),
                                                 (2.0 ** 90, 2.0 ** -90, -0.2)])
def test_scores_between_far_factors(hd, q_mult, k_mult, scale, form, kernel):
    """Scores of ordinary size from queries, keys and a scale that are far from it."""
    ops.check(ops.gen(hd), hd, 8, 2, 2, [0, 7, 200], 16, form, q_mult=q_mult, k_mult=k_mult, scale=scale)


@pytest.mark.parametrize("form", ops.FORMS)
@pytest.mark.parametrize("hd", ops.HD)
@pytest.mark.parametrize("T,window", [(2, 0), (40, 0), (40, 90)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -140, -(2.0 ** -126)])
def test_small_scales_over_large_products(hd, scale, T, window, form, kernel):
    """A scale of 0 gives every key the same weight, however large its product with the query is, and one below 2^-126 counts."""
    ops.check(ops.gen(hd), hd, 8, 2, T, [0, 7, 200], 16, form, q_mult=2.0 ** 58, k_mult=2.0 ** 58, scale=scale, window=window, causal=True)
