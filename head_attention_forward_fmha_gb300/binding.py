"""Thin ctypes binding of ``libfmha_gb300.so`` (C ABI in ``include/fmha.h``).

Argument marshalling only: torch tensors are checked for dtype, shape,
contiguity and device, then their data pointers go to the C entry point of the
same name.  Every step of the attention forward runs in the library's CUDA
kernels; there is no CPU fallback, and a missing library raises.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# FMHA_GB300_LIB may name another build of the same library (for example the
# checked build, CHECKED_LIB_PATH) to load instead of the in-tree one.
LIB_PATH = os.environ.get("FMHA_GB300_LIB") or os.path.join(_PKG, "libfmha_gb300.so")
CHECKED_LIB_PATH = os.path.join(_PKG, "libfmha_gb300_checked.so")
FMHA_BUILD_CHECKED = 1

FMHA_OK = 0
ERRORS = {
    -1: "FMHA_ERR_NULL", -2: "FMHA_ERR_ALIGN", -3: "FMHA_ERR_HEADDIM", -4: "FMHA_ERR_HEADS",
    -5: "FMHA_ERR_SHAPE", -6: "FMHA_ERR_WORKSPACE", -7: "FMHA_ERR_LAUNCH", -8: "FMHA_ERR_DEVICE_TIMEOUT",
    -9: "FMHA_ERR_UNSUPPORTED", -10: "FMHA_ERR_DEVICE_BOUNDS",
}
# Partial formats (enum fmha_parts_format).
PARTS_F32, PARTS_F16 = 0, 1

# Every symbol include/fmha.h declares, with its ctypes signature.
_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fmha_fwd": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp], _i32),
    "fmha_fwd_plan": ([_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i32)],
                      _i32),
    "fmha_split_layout": ([_i32, _i32, _i32, _i32, ctypes.POINTER(_i32)], _i32),
    "fmha_fwd_splitkv": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp],
                         _i32),
    "fmha_merge": ([_vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "fmha_fwd_splitkv_ex": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                             _i32, _vp], _i32),
    "fmha_merge_ex": ([_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "fmha_fwd_sink": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp], _i32),
    "fmha_splitkv_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "fmha_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "fmha_check_device_status": ([_vp], _i32),
    "fmha_get_last_error": ([], ctypes.c_char_p),
    "fmha_release": ([], None),
    "fmha_version": ([], _i32),
    "fmha_set_kernel_path": ([_i32], _i32),
    "fmha_selftest_wait_timeout": ([ctypes.c_uint, _vp], _i32),
    "fmha_fwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp], _i32),
    "fmha_build_flags": ([], _i32),
    "fmha_fwd_host": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp], _i32),
    "fmha_selftest_bounds_check": ([_vp], _i32),
    "fmha_fwd_nvfp4": ([_vp, _vp, _vp, _vp, _vp, _vp, _f32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp],
                       _i32),
    "fmha_quantize_nvfp4": ([_vp, ctypes.c_longlong, _i32, _f32, _vp, _vp, _vp], _i32),
    "fmha_qk_norm_rope": ([_vp, ctypes.c_longlong, ctypes.c_longlong, _vp, _vp, _f32, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                           _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "fmha_kv4_append": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _f32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp], _i32),
    "fmha_fwd_kv4_plan": ([_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)], _i32),
    "fmha_fwd_kv4": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _f32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                      _f32, _i32, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "fmha_fwd_first_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32], _sz),
    "fmha_fwd_first": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz,
                        _vp], _i32),
    # arguments in one struct
    "fmha_qk_norm_rope_packed": ([ctypes.c_char_p], _i32),
    "fmha_kv4_append_packed": ([ctypes.c_char_p], _i32),
    "fmha_fwd_kv4_packed": ([ctypes.c_char_p], _i32),
    "fmha_fwd_first_packed": ([ctypes.c_char_p], _i32),
}
# Size of the fixed split-KV scratch fmha_fwd_noalloc uses (FMHA_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 32 << 20


_lib = None
_call = None      # _tensor_args.call (csrc/tensor_args.cpp), from the first call that needs it on
_packed = {}      # address of each *_packed entry


class FmhaError(RuntimeError):
    def __init__(self, code, fn, msg):
        super().__init__("%s returned %s (%d): %s" % (fn, ERRORS.get(code, "?"), code, msg))
        self.code = code


def load(path=None):
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError("libfmha_gb300.so not found at %s: run head_attention_forward_fmha_gb300.build" % p)
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _packed.update((n[:-7], ctypes.cast(getattr(lib, n), _vp).value) for n in SIGNATURES if n.endswith("_packed"))
        _lib = lib
    return lib


def _load_packer():
    """Load the argument packer (once), which the serving operators' calls need and no other."""
    global _call
    load()
    try:
        from . import _tensor_args
    except ImportError as e:
        raise ImportError("the argument packer _tensor_args.so is missing or was built against another torch (%s): run "
                          "head_attention_forward_fmha_gb300.build" % e) from e
    _call = _tensor_args.call


def _check(rc, fn):
    if rc != FMHA_OK:
        raise FmhaError(rc, fn, load().fmha_get_last_error().decode(errors="replace"))


def _stream(stream):
    if stream is None:
        # the current stream's handle, without the Stream object around it (0.1 us against 2.9)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream_object(stream, dev):
    """The torch stream of a call's `stream` argument, a Stream or a handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)  # ExternalStream(0) would be one of torch's own streams
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _empty(shape, dtype, dev, stream):
    """A new tensor that a call on `stream` (None: the current one) writes.

    On another stream it takes that stream's memory: what tensors of the current stream have left may still be in use by
    work queued there.  It counts as used by the current stream too, where the caller may read it and then drop it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    side, here = _stream_object(stream, dev), torch.cuda.current_stream(dev)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if side.cuda_stream != here.cuda_stream:
        t.record_stream(here)
    return t


def _bf16(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous CUDA bf16 tensor" % name)
    return t.data_ptr()


def _f32(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous CUDA float32 tensor" % name)
    return t.data_ptr()


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or tuple(k.shape) != tuple(v.shape):
        raise ValueError("q [b,n_h,T,hd] and k, v [b,n_kv_h,s_k,hd] expected")
    b, n_h, T, hd = q.shape
    bk, n_kv_h, s_k, hdk = k.shape
    if bk != b or hdk != hd:
        raise ValueError("q %s and k %s disagree" % (tuple(q.shape), tuple(k.shape)))
    return b, n_h, n_kv_h, T, s_k, hd


def _check_outputs(q, o, lse):
    """o must be shaped like q and lse [b, n_h, T], both on q's device, so that
    the kernels never write past the end of a caller's buffer."""
    b, n_h, T, _ = q.shape
    if not isinstance(o, torch.Tensor) or tuple(o.shape) != tuple(q.shape):
        raise ValueError("o must be shaped like q %s" % (tuple(q.shape),))
    if not isinstance(lse, torch.Tensor) or tuple(lse.shape) != (b, n_h, T):
        raise ValueError("lse must be [b,n_h,T] = %s" % ((b, n_h, T),))
    if o.device != q.device or lse.device != q.device:
        raise ValueError("o and lse must be on q's device (%s)" % q.device)


def _sink_ptr(sink, n_h):
    if sink is None:
        return None
    if sink.numel() != n_h:
        raise ValueError("sink must hold one logit per query head (%d), got %d" % (n_h, sink.numel()))
    return _f32(sink, "sink")


def fmha_fwd(q, k, v, o=None, lse=None, scale=None, window=0, causal=False, stream=None, sink=None):
    """O (bf16 [b,n_h,T,hd]) and LSE (fp32 [b,n_h,T]); allocates them if not given.
    sink: optional fp32 CUDA tensor of n_h attention-sink logits (fmha_fwd_sink)."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    qp, kp, vp = _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v")
    if o is None:
        o = _empty(q.shape, torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((b, n_h, T), torch.float32, q.device, stream)
    _check_outputs(q, o, lse)
    if scale is None:
        scale = hd ** -0.5
    if sink is None:
        rc = load().fmha_fwd(qp, kp, vp, _bf16(o, "o"), _f32(lse, "lse"),
                             b, n_h, n_kv_h, T, s_k, hd, float(scale), int(window), int(bool(causal)),
                             _stream(stream))
        _check(rc, "fmha_fwd")
    else:
        rc = load().fmha_fwd_sink(qp, kp, vp, _bf16(o, "o"), _f32(lse, "lse"),
                                  _sink_ptr(sink, n_h), b, n_h, n_kv_h, T, s_k, hd, float(scale), int(window),
                                  int(bool(causal)), _stream(stream))
        _check(rc, "fmha_fwd_sink")
    return o, lse


def _host(t, name, dtype):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous host (CPU) %s tensor" % (name, dtype))
    return t.data_ptr()


def fmha_fwd_host(q, k, v, o=None, lse=None, scale=None, window=0, causal=False, stream=None):
    """fmha_fwd on host tensors (fmha_fwd_host): q, k, v are contiguous CPU bf16
    tensors, preferably page-locked; O and LSE come back in CPU tensors
    (page-locked ones are allocated if not given).  Stream-ordered: the results
    are valid, and the inputs may be changed, once `stream` has passed the call."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    if o is None:
        o = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    if lse is None:
        lse = torch.empty((b, n_h, T), dtype=torch.float32).pin_memory()
    if tuple(o.shape) != tuple(q.shape) or tuple(lse.shape) != (b, n_h, T):
        raise ValueError("o must be [b,n_h,T,hd] and lse [b,n_h,T]")
    if scale is None:
        scale = hd ** -0.5
    rc = load().fmha_fwd_host(_host(q, "q", torch.bfloat16), _host(k, "k", torch.bfloat16),
                              _host(v, "v", torch.bfloat16), _host(o, "o", torch.bfloat16),
                              _host(lse, "lse", torch.float32), b, n_h, n_kv_h, T, s_k, hd, float(scale),
                              int(window), int(bool(causal)), _stream(stream))
    _check(rc, "fmha_fwd_host")
    return o, lse


KERNELS = {1: "decode_splitkv", 2: "fwd_tc", 3: "fwd_tc_wide", 4: "fwd_tc_pair"}


def fmha_fwd_plan(batch, n_h, n_kv_h, T, s_k, hd, window=0, causal=False, with_kernel=False):
    """(n_splits, kv_chunk) that fmha_fwd uses for this shape, plus the kernel
    family name if ``with_kernel``."""
    chunk, kern = ctypes.c_int(0), ctypes.c_int(0)
    n = load().fmha_fwd_plan(batch, n_h, n_kv_h, T, s_k, hd, int(window), int(bool(causal)), ctypes.byref(chunk),
                             ctypes.byref(kern))
    _check(n if n < 0 else 0, "fmha_fwd_plan")
    if with_kernel:
        return n, chunk.value, KERNELS.get(kern.value, "?")
    return n, chunk.value


def fmha_split_layout(T, s_k, window, kv_chunk):
    """(first key of chunk 0, number of chunks)."""
    first = ctypes.c_int(0)
    n = load().fmha_split_layout(int(T), int(s_k), int(window), int(kv_chunk), ctypes.byref(first))
    _check(n if n < 0 else 0, "fmha_split_layout")
    return first.value, n


def fmha_fwd_splitkv(q, k, v, kv_chunk, o_parts=None, lse_parts=None, scale=None, window=0, causal=False,
                     stream=None):
    """fp32 partials O_i [n,b,n_h,T,hd] and lse_i [n,b,n_h,T] for chunks of kv_chunk keys."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    _, n = fmha_split_layout(T, s_k, window, kv_chunk)
    qp, kp, vp = _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v")
    if o_parts is None:
        o_parts = _empty((n, b, n_h, T, hd), torch.float32, q.device, stream)
    if lse_parts is None:
        lse_parts = _empty((n, b, n_h, T), torch.float32, q.device, stream)
    if o_parts.numel() < n * b * n_h * T * hd or lse_parts.numel() < n * b * n_h * T:
        raise ValueError("partial buffers too small for %d chunks" % n)
    if scale is None:
        scale = hd ** -0.5
    rc = load().fmha_fwd_splitkv(qp, kp, vp, _f32(o_parts, "o_parts"),
                                 _f32(lse_parts, "lse_parts"), int(kv_chunk), b, n_h, n_kv_h, T, s_k, hd,
                                 float(scale), int(window), int(bool(causal)), _stream(stream))
    _check(rc, "fmha_fwd_splitkv")
    return o_parts, lse_parts


def fmha_merge(o_parts, lse_parts, o=None, lse=None, stream=None, sink=None):
    """Merge partials [n,b,n_h,T,hd] / [n,b,n_h,T] into bf16 O and fp32 LSE
    (with an optional [n_h] attention-sink tensor)."""
    if o_parts.dim() != 5 or lse_parts.dim() != 4 or tuple(o_parts.shape[:4]) != tuple(lse_parts.shape):
        raise ValueError("o_parts [n,b,n_h,T,hd] and lse_parts [n,b,n_h,T] expected")
    n, b, n_h, T, hd = o_parts.shape
    op, lp = _f32(o_parts, "o_parts"), _f32(lse_parts, "lse_parts")
    if o is None:
        o = _empty((b, n_h, T, hd), torch.bfloat16, o_parts.device, stream)
    if lse is None:
        lse = _empty((b, n_h, T), torch.float32, o_parts.device, stream)
    if sink is None:
        rc = load().fmha_merge(op, lp, n, _bf16(o, "o"), _f32(lse, "lse"), b, n_h, T, hd, _stream(stream))
        _check(rc, "fmha_merge")
    else:
        rc = load().fmha_merge_ex(op, lp, None, PARTS_F32, n,
                                  _sink_ptr(sink, n_h), _bf16(o, "o"), _f32(lse, "lse"), b, n_h, T, hd,
                                  _stream(stream))
        _check(rc, "fmha_merge_ex")
    return o, lse


def fmha_fwd_splitkv_f16(q, k, v, kv_chunk, o_parts=None, lse_parts=None, range_parts=None, scale=None, window=0,
                         causal=False, stream=None):
    """fp16 partials (FMHA_PARTS_F16): O_i * 2^-k as fp16 [n,b,n_h,T,hd], lse_i fp32 [n,b,n_h,T] and the
    factors 2^k fp32 [n,b,n_h,T,2] (one per 256-column half row).  hd-512 tensor-core kernel only."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    _, n = fmha_split_layout(T, s_k, window, kv_chunk)
    qp, kp, vp = _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v")
    if o_parts is None:
        o_parts = _empty((n, b, n_h, T, hd), torch.float16, q.device, stream)
    if lse_parts is None:
        lse_parts = _empty((n, b, n_h, T), torch.float32, q.device, stream)
    if range_parts is None:
        range_parts = _empty((n, b, n_h, T, 2), torch.float32, q.device, stream)
    if (o_parts.dtype != torch.float16 or not o_parts.is_cuda or not o_parts.is_contiguous()
            or o_parts.numel() < n * b * n_h * T * hd or lse_parts.numel() < n * b * n_h * T
            or range_parts.numel() < n * b * n_h * T * 2):
        raise ValueError("fp16 partial buffers too small or of the wrong type for %d chunks" % n)
    if scale is None:
        scale = hd ** -0.5
    rc = load().fmha_fwd_splitkv_ex(qp, kp, vp, o_parts.data_ptr(),
                                    _f32(lse_parts, "lse_parts"), _f32(range_parts, "range_parts"), PARTS_F16,
                                    int(kv_chunk), b, n_h, n_kv_h, T, s_k, hd, float(scale), int(window),
                                    int(bool(causal)), _stream(stream))
    _check(rc, "fmha_fwd_splitkv_ex")
    return o_parts, lse_parts, range_parts


def fmha_merge_f16(o_parts, lse_parts, range_parts, o=None, lse=None, stream=None, sink=None):
    """Merge FMHA_PARTS_F16 partials into bf16 O and fp32 LSE."""
    if o_parts.dim() != 5 or o_parts.dtype != torch.float16 or not o_parts.is_contiguous():
        raise ValueError("o_parts: contiguous fp16 [n,b,n_h,T,hd] expected")
    n, b, n_h, T, hd = o_parts.shape
    if tuple(lse_parts.shape) != (n, b, n_h, T) or tuple(range_parts.shape) != (n, b, n_h, T, 2):
        raise ValueError("lse_parts [n,b,n_h,T] and range_parts [n,b,n_h,T,2] expected")
    lp, rp = _f32(lse_parts, "lse_parts"), _f32(range_parts, "range_parts")
    if o is None:
        o = _empty((b, n_h, T, hd), torch.bfloat16, o_parts.device, stream)
    if lse is None:
        lse = _empty((b, n_h, T), torch.float32, o_parts.device, stream)
    rc = load().fmha_merge_ex(o_parts.data_ptr(), lp, rp,
                              PARTS_F16, n, _sink_ptr(sink, n_h), _bf16(o, "o"), _f32(lse, "lse"), b, n_h, T, hd,
                              _stream(stream))
    _check(rc, "fmha_merge_ex")
    return o, lse


def fmha_splitkv_workspace_bytes(batch, n_h, T, hd, n_splits):
    return int(load().fmha_splitkv_workspace_bytes(batch, n_h, T, hd, n_splits))


def fmha_workspace_bytes(batch, n_h, T, hd, n_splits):
    """Bytes of the caller buffers fmha_fwd_splitkv + fmha_merge need for n_splits chunks."""
    return int(load().fmha_workspace_bytes(batch, n_h, T, hd, n_splits))


def fmha_check_device_status(stream=None):
    rc = load().fmha_check_device_status(_stream(stream))
    _check(rc, "fmha_check_device_status")


def fmha_get_last_error():
    return load().fmha_get_last_error().decode(errors="replace")


def _u8(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous CUDA uint8 tensor" % name)
    return t.data_ptr()


def fmha_fwd_nvfp4(q, k, v, codes=None, scales=None, lse=None, global_scale=1.0, scale=None, window=0,
                   causal=False, stream=None):
    """fmha_fwd with O quantised to NVFP4 (see include/fmha.h): returns
    (codes uint8 [b,n_h,T,hd/2], scales uint8 [b,n_h,T,hd/16] E4M3, lse fp32 [b,n_h,T])."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    qp, kp, vp = _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v")
    if codes is None:
        codes = _empty((b, n_h, T, hd // 2), torch.uint8, q.device, stream)
    if scales is None:
        scales = _empty((b, n_h, T, hd // 16), torch.uint8, q.device, stream)
    if lse is None:
        lse = _empty((b, n_h, T), torch.float32, q.device, stream)
    if (tuple(codes.shape) != (b, n_h, T, hd // 2) or tuple(scales.shape) != (b, n_h, T, hd // 16)
            or tuple(lse.shape) != (b, n_h, T)):
        raise ValueError("codes [b,n_h,T,hd/2], scales [b,n_h,T,hd/16] and lse [b,n_h,T] expected")
    if codes.device != q.device or scales.device != q.device or lse.device != q.device:
        raise ValueError("codes, scales and lse must be on q's device (%s)" % q.device)
    if scale is None:
        scale = hd ** -0.5
    rc = load().fmha_fwd_nvfp4(qp, kp, vp, _u8(codes, "codes"), _u8(scales, "scales"), _f32(lse, "lse"),
                               float(global_scale), b, n_h, n_kv_h, T, s_k, hd, float(scale), int(window),
                               int(bool(causal)), _stream(stream))
    _check(rc, "fmha_fwd_nvfp4")
    return codes, scales, lse


def fmha_quantize_nvfp4(x, global_scale=1.0, stream=None):
    """NVFP4 codes and E4M3 scales of fp32 rows x [..., hd] (the fused epilogues' quantiser)."""
    if x.dim() < 1 or x.shape[-1] % 16 != 0:
        raise ValueError("x [..., hd] with hd a multiple of 16 expected")
    hd = x.shape[-1]
    rows, xp = x.numel() // hd, _f32(x, "x")
    codes = _empty(tuple(x.shape[:-1]) + (hd // 2,), torch.uint8, x.device, stream)
    scales = _empty(tuple(x.shape[:-1]) + (hd // 16,), torch.uint8, x.device, stream)
    rc = load().fmha_quantize_nvfp4(xp, rows, hd, float(global_scale), _u8(codes, "codes"),
                                    _u8(scales, "scales"), _stream(stream))
    _check(rc, "fmha_quantize_nvfp4")
    return codes, scales


def fmha_release():
    """Free the library's workspaces."""
    load().fmha_release()


def fmha_version():
    return int(load().fmha_version())


def fmha_build_flags():
    """FMHA_BUILD_CHECKED if the loaded library is the checked build, else 0."""
    return int(load().fmha_build_flags())


def fmha_selftest_bounds_check(stream=None):
    """One failing index check on the device (recorded only by the checked build)."""
    _check(load().fmha_selftest_bounds_check(_stream(stream)), "fmha_selftest_bounds_check")


def fmha_selftest_wait_timeout(timeout_us, stream=None):
    """Launch the bounded-wait self-test kernel (see include/fmha.h)."""
    _check(load().fmha_selftest_wait_timeout(int(timeout_us), _stream(stream)), "fmha_selftest_wait_timeout")


def fmha_set_kernel_path(path):
    """0 automatic, 1 decode kernel, 2 tensor-core kernels (two row tiles per block where that
    kernel applies), 3 tensor-core kernels, one row tile per block, with the row-tile kernel's
    P V in the SS form (P through shared memory) instead of the TS form, 4 tensor-core kernels,
    one row tile per block (TS form)."""
    _check(load().fmha_set_kernel_path(int(path)), "fmha_set_kernel_path")
    _first_plans.clear()
    _kv4_plans.clear()


def fmha_fwd_noalloc(q, k, v, o, lse, scale=None, window=0, causal=False, stream=None):
    """fmha_fwd for callers that cannot allocate device memory: O and LSE must be
    given, and split-KV partials use the library's fixed scratch array instead
    of a workspace (see include/fmha.h)."""
    b, n_h, n_kv_h, T, s_k, hd = _shapes(q, k, v)
    qp, kp, vp = _bf16(q, "q"), _bf16(k, "k"), _bf16(v, "v")
    _check_outputs(q, o, lse)
    if scale is None:
        scale = hd ** -0.5
    rc = load().fmha_fwd_noalloc(qp, kp, vp, _bf16(o, "o"), _f32(lse, "lse"),
                                 b, n_h, n_kv_h, T, s_k, hd, float(scale), int(window), int(bool(causal)),
                                 _stream(stream))
    _check(rc, "fmha_fwd_noalloc")
    return o, lse


# ---------------------------------------------------------------------------
# Serving operators around the forward: norm and rotation, 4-bit cache, window
# with first keys.  Their smallest calls take a few microseconds on the GPU, so
# the tensors are checked and packed by csrc/tensor_args.cpp.
# ---------------------------------------------------------------------------
_BF16, _FP32, _U8 = torch.bfloat16, torch.float32, torch.uint8

# The argument structs of include/fmha.h: entry, a character per field (tensor_args.cpp has their meaning), tensor names.
_NORM_ROPE = ("fmha_qk_norm_rope", b"SfffiBBBiqqqrnnnnnnnnn",
              ("qkv", "q_weight", "k_weight", "cos_sin", "positions", "q", "k", "v", "kv_start"))
_APPEND = ("fmha_kv4_append", b"BBUUUUIbbqrrnnnnnn",
           ("k", "v", "k_codes", "k_scales", "v_codes", "v_scales", "start", "k_out", "v_out"))
_KV4 = ("fmha_fwd_kv4", b"BUUUUiBFfuqqrrrnnnnnnnnnnn",
        ("q", "k_codes", "k_scales", "v_codes", "v_scales", "seq_lens", "o", "lse", "sink", "workspace"))
_FIRST = ("fmha_fwd_first", b"BBBBFfuqqrnnnnnnnnn", ("q", "k", "v", "o", "lse", "sink", "workspace"))


def _device(t, name):
    """CUDA device index of the tensor that decides where a call runs."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _run(entry, dev, *values):
    """Call an entry with the values of its struct's fields (tensors each with their shape), device `dev` current."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _run(entry, dev, *values)
    if _call is None:
        _load_packer()
    fn, layout, names = entry
    rc = _call(_packed[fn], layout, names, dev, *values)
    if rc:
        _check(rc, fn)


def _handle(stream, dev):
    """The stream's handle; None is the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


# Workspaces that outlive a call: none.  Those of split calls are allocated by csrc/tensor_args.cpp for the call alone, in
# the memory of its stream (of the graph's pool while torch.cuda.graph captures it).  Kept ones would stay behind threads
# and streams that are gone, and could lie in a pool that is not theirs.  (That allocator takes the per-thread default
# stream, handle 2, for one stream: threads that run on it give workspaces and outputs of their own.)
_workspaces = ()


def fmha_qk_norm_rope(qkv, cos_sin, positions, n_h, n_kv_h, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                      q=None, k=None, v=None, kv_start=None, stream=None):
    """Rows of a QKV projection to what fmha_fwd takes (fmha_qk_norm_rope in include/fmha.h): RMS norm of every
    query and key head (weights fp32 [hd]; None: no norm), rotation by position, head-major outputs.

    qkv: bf16 [b, T, (n_h + 2 n_kv_h) * hd], rows contiguous, tokens and sequences at any stride of a multiple of 8
    elements.  cos_sin: fp32 [max_pos, rot], the cosines and then the sines of each position; positions: int32 [b, T]
    (a token outside [0, max_pos) is padding, its outputs are left as they are); both None: no rotation.
    k and v given with more rows than T are written at rows kv_start[b] + t (int32 [b]; None: 0); fmha_fwd and
    fmha_fwd_first count every row of such a buffer as a key.
    Returns q [b, n_h, T, hd], k and v [b, n_kv_h, rows, hd]; what is not given is allocated, and undefined where
    nothing is written."""
    dev = _device(qkv, "qkv")
    shape = qkv.shape
    if len(shape) != 3 or n_h < 1 or n_kv_h < 1 or shape[2] % (n_h + 2 * n_kv_h):
        raise ValueError("qkv [b, T, (n_h + 2 n_kv_h) * hd] expected, got %s" % (tuple(shape),))
    b, T, width = shape
    hd = width // (n_h + 2 * n_kv_h)
    sb, st, se = qkv.stride()
    if se != 1 and width > 1:
        raise ValueError("the rows of qkv must be contiguous")
    if T <= 1:  # strides of dimensions of one element say nothing
        st = max(width, (st + 7) // 8 * 8)
    if b <= 1:
        sb = 0
    if (cos_sin is None) != (positions is None):
        raise ValueError("cos_sin and positions are given together or not at all")
    if (k is None) != (v is None) or (k is not None and k.dim() != 4):
        raise ValueError("k and v [b, n_kv_h, rows, hd] are given together or not at all")
    if cos_sin is None:
        max_pos = rot = 0
    elif cos_sin.dim() != 2:
        raise ValueError("cos_sin [max_pos, rot] expected, got %s" % (tuple(cos_sin.shape),))
    else:
        max_pos, rot = cos_sin.shape
    if q is None:
        q = _empty((b, n_h, T, hd), _BF16, dev, stream)
    if k is None:
        k, v = (_empty((b, n_kv_h, T, hd), _BF16, dev, stream) for _ in range(2))
    rows = k.shape[2]
    kv_shape, w_shape = (b, n_kv_h, rows, hd), (hd,)
    _run(_NORM_ROPE, dev, qkv, q_weight, w_shape, k_weight, w_shape, cos_sin, None, positions, (b, T), q, (b, n_h, T, hd),
         k, kv_shape, v, kv_shape, kv_start, (b,), _handle(stream, dev), sb, st, eps, max_pos, rot, bool(interleaved), rows, b, T,
         n_h, n_kv_h, hd)
    return q, k, v


def fmha_kv4_cache(batch, n_kv_h, cap, hd, device="cuda"):
    """An empty 4-bit KV cache of `cap` rows (a multiple of 16) per sequence and head: the uint8 tensors
    (k_codes, k_scales, v_codes, v_scales) that fmha_kv4_append writes and fmha_fwd_kv4 reads."""
    if hd not in (64, 128, 256, 512) or cap % 16:
        raise ValueError("hd must be 64, 128, 256 or 512 and cap a multiple of 16 (got hd=%d cap=%d)" % (hd, cap))
    return tuple(torch.zeros((batch, n_kv_h, cap, hd // w), dtype=_U8, device=device) for w in (2, 16, 2, 16))


def _kv4_heads_rows(k_codes):
    if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
        raise ValueError("k_codes [b, n_kv_h, cap, hd/2] expected")
    return k_codes.shape[1:3]


def fmha_kv4_append(k, v, k_codes, k_scales, v_codes, v_scales, start, k_global=1.0, v_global=1.0, k_out=None, v_out=None,
                    stream=None):
    """Quantise k, v (bf16 [b, n_kv_h, T, hd]) into a 4-bit cache (fmha_kv4_cache) at rows start[b] + t (int32 [b]; rows
    outside the cache are left out).  k_out and v_out, bf16 like k, receive the values that the written rows stand for."""
    dev = _device(k, "k")
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("k [b, n_kv_h, T, hd] expected, got %s" % (tuple(shape),))
    b, n_kv_h, T, hd = shape
    cap = _kv4_heads_rows(k_codes)[1]
    codes, scales = (b, n_kv_h, cap, hd // 2), (b, n_kv_h, cap, hd // 16)
    _run(_APPEND, dev, k, shape, v, shape, k_codes, codes, k_scales, scales, v_codes, codes, v_scales, scales, start, (b,),
         k_out, shape, v_out, shape, _handle(stream, dev), k_global, v_global, b, n_kv_h, T, cap, hd, 0)


def _planned(dev, query, *args):
    """What `query`, a plan, says on device `dev`: it depends on the number of SMs."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return query(*args)
    return query(*args)


def _remember(plans, key, value):
    """Keep a plan; lengths that grow with every call would otherwise fill the memory."""
    if len(plans) >= 4096:
        plans.clear()
    plans[key] = value
    return value


_kv4_plans = {}  # (chunk length, workspace bytes) by shape and device, for the kernel path that is set


def fmha_fwd_kv4_plan(batch, n_h, n_kv_h, T, s_k, hd, window=0, n_first=0, causal=False, kv_chunk=0, ragged=True):
    """(n_splits, kv_chunk) that fmha_fwd_kv4 uses for sequences of up to s_k keys (kv_chunk 0: its own choice; ragged:
    whether seq_lens is given)."""
    chunk = ctypes.c_int(int(kv_chunk))
    n = (_lib or load()).fmha_fwd_kv4_plan(batch, n_h, n_kv_h, T, s_k, hd, int(window), int(n_first), int(bool(causal)),
                                           int(bool(ragged)), ctypes.byref(chunk))
    _check(n if n < 0 else 0, "fmha_fwd_kv4_plan")
    return n, chunk.value


def fmha_fwd_kv4(q, k_codes, k_scales, v_codes, v_scales, seq_lens=None, o=None, lse=None, s_k=None, k_global=1.0,
                 v_global=1.0, scale=None, window=0, n_first=0, causal=False, sink=None, kv_chunk=0, workspace=None,
                 stream=None):
    """O (bf16) and LSE (fp32) of q (bf16 [b, n_h, T, hd]) over a 4-bit cache (fmha_fwd_kv4 in include/fmha.h).

    seq_lens: int32 [b], the keys of each sequence (None: s_k each); s_k: their bound, at most the cache's rows (the
    default).  With a window, the keys j < n_first stay attended.  workspace: an optional uint8 tensor for the split-KV
    partials (fmha_workspace_bytes of fmha_fwd_kv4_plan's n_splits); without one the call allocates
    its own (under capture by torch.cuda.graph in the graph's pool; give one under any other capture)."""
    dev = _device(q, "q")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q [b, n_h, T, hd] expected, got %s" % (tuple(shape),))
    b, n_h, T, hd = shape
    n_kv_h, cap = _kv4_heads_rows(k_codes)
    if s_k is None:
        s_k = cap
    if o is None:
        o = _empty(shape, _BF16, dev, stream)
    if lse is None:
        lse = _empty((b, n_h, T), _FP32, dev, stream)
    key = (b, n_h, n_kv_h, T, s_k, hd, window, n_first, causal, kv_chunk, seq_lens is not None, dev)
    plan = _kv4_plans.get(key)
    if plan is None:
        n, chunk = _planned(dev, fmha_fwd_kv4_plan, *key[:-1])
        plan = _remember(_kv4_plans, key, (chunk, fmha_workspace_bytes(b, n_h, T, hd, n) if n > 1 else 0))
    kv_chunk, need = plan
    handle = at = _handle(stream, dev)
    if workspace is not None:
        need, at = workspace.numel(), None
    elif need:  # the call's own, of its stream's memory
        workspace = need
    codes, scales = (b, n_kv_h, cap, hd // 2), (b, n_kv_h, cap, hd // 16)
    _run(_KV4, dev, q, shape, k_codes, codes, k_scales, scales, v_codes, codes, v_scales, scales, seq_lens, (b,), o, shape,
         lse, (b, n_h, T), sink, (n_h,), workspace, at, need, handle, k_global, v_global,
         hd ** -0.5 if scale is None else scale, b, n_h, n_kv_h, T, s_k, cap, hd, window, n_first, bool(causal), kv_chunk)
    return o, lse


_first_plans = {}  # workspace bytes by shape and device, for the kernel path that is set


def fmha_fwd_first_workspace_bytes(batch, n_h, n_kv_h, T, s_k, hd, window, n_first, causal=False):
    """Workspace bytes that fmha_fwd_first needs for this shape (0: none)."""
    return int((_lib or load()).fmha_fwd_first_workspace_bytes(batch, n_h, n_kv_h, T, s_k, hd, int(window), int(n_first),
                                                               int(bool(causal))))


def fmha_fwd_first(q, k, v, n_first, o=None, lse=None, scale=None, window=0, causal=False, sink=None, workspace=None,
                   stream=None):
    """fmha_fwd with the keys j < n_first attended outside the window too (fmha_fwd_first in include/fmha.h).
    workspace: an optional uint8 tensor of fmha_fwd_first_workspace_bytes; without one the call allocates
    its own (under capture by torch.cuda.graph in the graph's pool; give one under any other capture)."""
    dev = _device(q, "q")
    q_shape, kv_shape = q.shape, k.shape
    if len(q_shape) != 4 or len(kv_shape) != 4:
        raise ValueError("q [b,n_h,T,hd] and k, v [b,n_kv_h,s_k,hd] expected")
    b, n_h, T, hd = q_shape
    n_kv_h, s_k = kv_shape[1:3]
    if o is None:
        o = _empty(q_shape, _BF16, dev, stream)
    if lse is None:
        lse = _empty((b, n_h, T), _FP32, dev, stream)
    key = (b, n_h, n_kv_h, T, s_k, hd, window, n_first, causal, dev)
    need = _first_plans.get(key)
    if need is None:
        need = _remember(_first_plans, key, _planned(dev, fmha_fwd_first_workspace_bytes, *key[:-1]))
    handle = at = _handle(stream, dev)
    if workspace is not None:
        need, at = workspace.numel(), None
    elif need:  # the call's own, of its stream's memory
        workspace = need
    kv_shape = (b, n_kv_h, s_k, hd)
    _run(_FIRST, dev, q, q_shape, k, kv_shape, v, kv_shape, o, q_shape, lse, (b, n_h, T), sink, (n_h,), workspace, at, need,
         handle, hd ** -0.5 if scale is None else scale, b, n_h, n_kv_h, T, s_k, hd, window, n_first, bool(causal))
    return o, lse
