"""``torch.ops.fmha_gb300.fwd``: the attention forward as a PyTorch custom op.

Registers one operator around the C ABI (``fmha_fwd``) with a fake (meta)
implementation, so that ``torch.compile`` can trace programs that call it
without running it.  The real implementation is the library's CUDA kernels;
like the binding, it accepts contiguous CUDA bf16 tensors only.

    q [b, n_h, T, hd], k, v [b, n_kv_h, s_k, hd]  ->  (O [b, n_h, T, hd] bf16, LSE [b, n_h, T] fp32)

``fwd_first`` and ``fwd_kv4`` do the same for ``fmha_fwd_first`` and ``fmha_fwd_kv4``.

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
