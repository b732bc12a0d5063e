"""``torch.ops.fmha_gb300.fwd``: the attention forward as a PyTorch custom op.

Registers one operator around the C ABI (``fmha_fwd``) with a fake (meta)
implementation, so that ``torch.compile`` can trace programs that call it
without running it.  The real implementation is the library's CUDA kernels;
like the binding, it accepts contiguous CUDA bf16 tensors only.

    q [b, n_h, T, hd], k, v [b, n_kv_h, s_k, hd]  ->  (O [b, n_h, T, hd] bf16, LSE [b, n_h, T] fp32)

``fwd_first`` and ``fwd_kv4`` do the same for ``fmha_fwd_first`` and ``fmha_fwd_kv4``,
``paged_append`` (which changes the cache), ``paged_gather`` and ``fwd_paged`` for
the cache in pages.

An optional ``sink`` tensor (fp32, n_h attention-sink logits) selects
``fmha_fwd_sink``.
"""
from typing import Optional, Tuple

import torch

from . import binding


@torch.library.custom_op("fmha_gb300::fwd", mutates_args=())
def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float, window: int,
        causal: bool, sink: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    return binding.fmha_fwd(q, k, v, scale=scale, window=window, causal=causal, sink=sink)


@fwd.register_fake
def _fwd_fake(q, k, v, scale, window, causal, sink=None):
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("q [b,n_h,T,hd] and k, v [b,n_kv_h,s_k,hd] expected")
    b, n_h, T, hd = q.shape
    return torch.empty_like(q), q.new_empty((b, n_h, T), dtype=torch.float32)


def attention(q, k, v, scale=None, window=0, causal=False, sink=None):
    """Convenience wrapper: ``torch.ops.fmha_gb300.fwd`` with scale defaulting to 1/sqrt(hd)."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return torch.ops.fmha_gb300.fwd(q, k, v, float(scale), int(window), bool(causal), sink)


@torch.library.custom_op("fmha_gb300::fwd_first", mutates_args=())
def fwd_first(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_first: int, scale: float, window: int, causal: bool,
              sink: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``fwd`` with the keys j < n_first attended outside the window too."""
    return binding.fmha_fwd_first(q, k, v, n_first, scale=scale, window=window, causal=causal, sink=sink)


@fwd_first.register_fake
def _fwd_first_fake(q, k, v, n_first, scale, window, causal, sink=None):
    return _fwd_fake(q, k, v, scale, window, causal, sink)


@torch.library.custom_op("fmha_gb300::fwd_kv4", mutates_args=())
def fwd_kv4(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
            seq_lens: Optional[torch.Tensor], k_global: float, v_global: float, scale: float, window: int, n_first: int,
            causal: bool, sink: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The forward over a 4-bit cache: q [b, n_h, T, hd], codes [b, n_kv_h, cap, hd/2], scales [b, n_kv_h, cap, hd/16]."""
    return binding.fmha_fwd_kv4(q, k_codes, k_scales, v_codes, v_scales, seq_lens, k_global=k_global, v_global=v_global,
                                scale=scale, window=window, n_first=n_first, causal=causal, sink=sink)


@fwd_kv4.register_fake
def _fwd_kv4_fake(q, k_codes, k_scales, v_codes, v_scales, seq_lens, k_global, v_global, scale, window, n_first, causal,
                  sink=None):
    if q.dim() != 4 or k_codes.dim() != 4 or k_codes.shape != v_codes.shape or k_scales.shape != v_scales.shape:
        raise ValueError("q [b,n_h,T,hd], codes [b,n_kv_h,cap,hd/2] and scales [b,n_kv_h,cap,hd/16] expected")
    b, n_h, T, hd = q.shape
    return torch.empty_like(q), q.new_empty((b, n_h, T), dtype=torch.float32)


@torch.library.custom_op("fmha_gb300::paged_append", mutates_args=("k_pages", "v_pages", "k_scales", "v_scales"))
def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: Optional[torch.Tensor],
                 v_scales: Optional[torch.Tensor], block_table: torch.Tensor, start: torch.Tensor, cu_q: Optional[torch.Tensor] = None) -> None:
    """New K and V rows into a cache in pages; k and v as in binding.fmha_paged_append."""
    binding.fmha_paged_append(k, v, k_pages, v_pages, k_scales, v_scales, block_table, start, cu_q=cu_q)


@paged_append.register_fake
def _paged_append_fake(k, v, k_pages, v_pages, k_scales, v_scales, block_table, start, cu_q=None):
    if k.shape != v.shape or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("k and v of one shape and pages [n_pages,n_kv_h,page,hd] expected")


@torch.library.custom_op("fmha_gb300::paged_gather", mutates_args=())
def paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: Optional[torch.Tensor], v_scales: Optional[torch.Tensor],
                 block_table: torch.Tensor, seq_lens: torch.Tensor, rows: int,
                 start: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """k and v [b, n_kv_h, rows, hd] of a cache in pages, zeros where there is no row."""
    return binding.fmha_paged_gather(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, rows, start=start)


@paged_gather.register_fake
def _paged_gather_fake(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, rows, start=None):
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or block_table.dim() != 2:
        raise ValueError("pages [n_pages,n_kv_h,page,hd] and a block table [b,n] expected")
    shape = (block_table.shape[0], k_pages.shape[1], rows, k_pages.shape[3])
    return tuple(k_pages.new_empty(shape, dtype=torch.bfloat16) for _ in range(2))


@torch.library.custom_op("fmha_gb300::fwd_paged", mutates_args=())
def fwd_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: Optional[torch.Tensor], v_scales: Optional[torch.Tensor],
              block_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: Optional[torch.Tensor], max_q: Optional[int], scale: float,
              window: int, n_first: int, causal: bool, sink: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The forward over a cache in pages: q [b, n_h, T, hd], or with cu_q [total, n_h, hd], where rows that belong to no
    sequence give rows of any value.  The lengths are bounded by what the block table holds, which the chunks divide: where it is
    much wider than the sequences, pass a copy of the columns in use."""
    return binding.fmha_fwd_paged(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q=cu_q, max_q=max_q, scale=scale,
                                  window=window, n_first=n_first, causal=causal, sink=sink)


@fwd_paged.register_fake
def _fwd_paged_fake(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, max_q, scale, window, n_first, causal, sink=None):
    if q.dim() != (4 if cu_q is None else 3) or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("q [b,n_h,T,hd], or with cu_q [total,n_h,hd], and pages [n_pages,n_kv_h,page,hd] expected")
    return q.new_empty(q.shape), q.new_empty(q.shape[:-1], dtype=torch.float32)
