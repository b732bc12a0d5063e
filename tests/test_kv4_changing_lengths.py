"""Lengths of the 4-bit cache that another stream rewrites while calls of its tensor-core kernel run: what such a call gives is any value,
but it ends and the next call is right.  (One warp of a block reads the lengths for all.)"""
import pytest
import torch

import serving_ref as ref
import test_serving_ops as ops
from head_attention_forward_fmha_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("kv_chunk", [0, 256])
def test_calls_end_while_their_lengths_change(hd, kv_chunk):
    g = torch.Generator(device=ops.DEV).manual_seed(hd)
    b, n_h, n_kv, T, cap = 3, 8, 2, 40, 512
    k, v = (torch.randn(b, n_kv, cap, hd, generator=g, device=ops.DEV).to(torch.bfloat16) for _ in range(2))
    cache = binding.fmha_kv4_cache(b, n_kv, cap, hd)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(b, dtype=torch.int32, device=ops.DEV))
    q = torch.randn(b, n_h, T, hd, generator=g, device=ops.DEV).to(torch.bfloat16)
    states = [torch.tensor(x, dtype=torch.int32, device=ops.DEV) for x in ([512, 0, 77], [0, 512, 2 ** 31 - 1], [-5, 30, 0], [511, 512, 100])]
    n = states[0].clone()
    binding.fmha_set_kernel_path(2)
    try:
        binding.fmha_fwd_kv4(q, *cache, n, causal=True, kv_chunk=kv_chunk)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(60):
            with torch.cuda.stream(side):
                for x in states:
                    n.copy_(x)
            binding.fmha_fwd_kv4(q, *cache, n, causal=True, kv_chunk=kv_chunk)
        torch.cuda.synchronize()
        binding.fmha_check_device_status()
        n.copy_(states[0])
        got = binding.fmha_fwd_kv4(q, *cache, n, causal=True, kv_chunk=kv_chunk)
        want = binding.fmha_fwd_kv4(q, *cache, states[0], causal=True, kv_chunk=kv_chunk)
        torch.cuda.synchronize()
    finally:
        binding.fmha_set_kernel_path(0)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
