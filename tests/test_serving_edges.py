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
    cache = binding.fmha_kv4_cache(1, 2, cap, hd)
    out = torch.zeros_like(k), torch.zeros_like(v)
    binding.fmha_kv4_append(k, v, *cache, torch.zeros(1, dtype=torch.int32, device=DEV), k_global=g, v_global=g, k_out=out[0], v_out=out[1])
    for x, codes, scales, o in ((k, cache[0], cache[1], out[0]), (v, cache[2], cache[3], out[1])):
        c, s = binding.fmha_quantize_nvfp4(x.float(), global_scale=g)
        assert torch.equal(codes[:, :, :T], c) and torch.equal(scales[:, :, :T], s)
        values = ref.dequantise(c, s, 1.0).float() * torch.tensor(g, dtype=torch.float32, device=DEV)
        assert torch.equal(o, values.to(torch.bfloat16))
    assert (cache[0][0, 1, 0] == 0xFF).all() and (cache[0][0, 1, 1] == 0x77).all()
