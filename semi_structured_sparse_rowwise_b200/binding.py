"""Thin Python binding of libsfp8.so (ctypes).

Argument marshalling only: tensors are passed as raw device pointers with
their sizes, on torch's current CUDA stream.  Every step of the layer runs in
the library's CUDA kernels; there is no fallback of any kind.  If the library
is missing or fails to load, every call raises.

The functions carry the C names (``sfp8_quantize_rowwise`` and so on) and
allocate their outputs with torch when none are given.
"""

import ctypes
import functools
import os

import torch

from . import build as _build

OK = 0
STATUS_NAMES = {
    0: "SFP8_OK", 1: "SFP8_ERR_INVALID_ARG", 2: "SFP8_ERR_UNSUPPORTED_SHAPE",
    3: "SFP8_ERR_MISALIGNED", 4: "SFP8_ERR_UNSUPPORTED_DTYPE", 5: "SFP8_ERR_ARCH",
    6: "SFP8_ERR_WORKSPACE", 7: "SFP8_ERR_CUDA", 8: "SFP8_ERR_TIMEOUT",
    9: "SFP8_ERR_DEVICE_CHECK",
}
DTYPE = {"bf16": 0, "f16": 1, "f32": 2, "e4m3": 3, "e5m2": 4}
TORCH_WIDE = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}
AMAX_MODE = {"reduce": 0, "atomic": 1}
ACTIVATION = {"silu": 0, "gelu": 1}
DEVICE_TIMEOUT = 0x1
DEVICE_CHECK_FAIL = 0x2

# Every symbol declared in include/sfp8.h, with its C signature.
_c_void_p, _i64, _sz, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
SIGNATURES = {
    "sfp8_quantize_rowwise": (_i32, [_c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _i32,
                                     _c_void_p, _c_void_p]),
    "sfp8_quantize_tensorwise_workspace_bytes": (_sz, [_i32]),
    "sfp8_quantize_tensorwise": (_i32, [_c_void_p, _i32, _i64, _c_void_p, _i32, _c_void_p, _i32,
                                        _c_void_p, _sz, _c_void_p]),
    "sfp8_prune_24": (_i32, [_c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _c_void_p]),
    "sfp8_padded_rows": (_i64, [_i64]),
    "sfp8_compressed_bytes": (_sz, [_i64, _i64]),
    "sfp8_compressed_values_bytes": (_sz, [_i64, _i64]),
    "sfp8_compressed_meta_bytes": (_sz, [_i64, _i64]),
    "sfp8_compress_24": (_i32, [_c_void_p, _i32, _i64, _i64, _c_void_p, _c_void_p]),
    "sfp8_decompress_24": (_i32, [_c_void_p, _i64, _i64, _c_void_p, _c_void_p]),
    "sfp8_prepare_weight_24": (_i32, [_c_void_p, _i32, _i64, _i64, _i64, _i32, _c_void_p,
                                      _c_void_p, _c_void_p]),
    "sfp8_sparse_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_workspace_clear": (_i32, [_c_void_p, _sz, _c_void_p]),
    "sfp8_sparse_linear": (_i32, [_c_void_p, _i32, _c_void_p, _i64, _c_void_p, _i32,
                                  _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _sz,
                                  _c_void_p]),
    "sfp8_sparse_linear_noalloc": (_i32, [_c_void_p, _i32, _c_void_p, _i64, _c_void_p,
                                          _i32, _c_void_p, _i64, _i64, _c_void_p,
                                          _c_void_p, _c_void_p]),
    "sfp8_sparse_linear_algo_count": (_i32, [_i64, _i64, _i64]),
    "sfp8_sparse_linear_algo_info": (_i32, [_i64, _i64, _i64, _i32,
                                            ctypes.POINTER(ctypes.c_int32)]),
    "sfp8_sparse_linear_algo_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "sfp8_sparse_linear_plan_count": (_i32, [_i64, _i64, _i64, _i32]),
    "sfp8_sparse_linear_plan_info": (_i32, [_i64, _i64, _i64, _i32, _i32,
                                            ctypes.POINTER(ctypes.c_int64)]),
    "sfp8_sparse_linear_search_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_sparse_linear_algo": (_i32, [_c_void_p, _i32, _c_void_p, _i64, _c_void_p, _i32,
                                       _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _i32,
                                       _c_void_p, _sz, _c_void_p]),
    "sfp8_sparse_linear_search": (_i32, [_c_void_p, _i32, _c_void_p, _i64, _c_void_p, _i32,
                                         _c_void_p, _i64, _i64, _c_void_p, _c_void_p,
                                         _c_void_p, _sz, _c_void_p, _sz, _i32,
                                         ctypes.POINTER(ctypes.c_int32),
                                         ctypes.POINTER(ctypes.c_float), _i32, _c_void_p]),
    "sfp8_sparse_linear_set_algo": (_i32, [_i64, _i64, _i64, _i32]),
    "sfp8_sparse_linear_get_algo": (_i32, [_i64, _i64, _i64]),
    "sfp8_sparse_linear_quant_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_sparse_linear_quant": (_i32, [_c_void_p, _i32, _i64, _i32, _c_void_p, _c_void_p,
                                        _i64, _c_void_p, _i32, _c_void_p, _i64, _i64,
                                        _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "sfp8_sparse_linear_quant_fused": (_i32, [_c_void_p, _i32, _i64, _i32, _c_void_p,
                                              _c_void_p, _i64, _c_void_p, _i32, _c_void_p,
                                              _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                              _sz, _c_void_p]),
    "sfp8_sparse_linear_quant_chained": (_i32, [_c_void_p, _i32, _i64, _i32, _c_void_p,
                                                _c_void_p, _i64, _c_void_p, _i32, _c_void_p,
                                                _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                                _sz, _c_void_p]),
    "sfp8_sparse_linear_quant_fusable": (_i32, [_i64, _i64, _i64]),
    "sfp8_prepare_gated_weight_24": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i64, _i64, _i32,
                                            _c_void_p, _c_void_p, _c_void_p]),
    "sfp8_gated_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_gated_linear": (_i32, [_c_void_p, _i32, _c_void_p, _i64, _c_void_p, _i32, _c_void_p,
                                 _i64, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _sz,
                                 _c_void_p]),
    "sfp8_gated_linear_quant_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_gated_linear_quant": (_i32, [_c_void_p, _i32, _i64, _i32, _c_void_p, _c_void_p, _i64,
                                       _c_void_p, _i32, _c_void_p, _i64, _i64, _i32, _c_void_p,
                                       _c_void_p, _c_void_p, _sz, _c_void_p]),
    "sfp8_sparse_linear_backward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_sparse_linear_backward": (_i32, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _i64,
                                           _c_void_p, _i32, _c_void_p, _i64, _i64, _c_void_p,
                                           _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "sfp8_gated_linear_backward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "sfp8_gated_linear_backward": (_i32, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _i64,
                                          _c_void_p, _i32, _c_void_p, _i64, _i64, _i32,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _sz, _c_void_p]),
    "sfp8_layernorm": (_i32, [_c_void_p, _i32, _i64, _i64, _i64, _c_void_p, _c_void_p, _i32,
                              ctypes.c_float, _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p,
                              _c_void_p, _c_void_p]),
    "sfp8_layernorm_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "sfp8_layernorm_backward": (_i32, [_c_void_p, _i64, _c_void_p, _i32, _i64, _i64, _i64,
                                       _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p,
                                       _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "sfp8_selftest_timeout": (_i32, [_c_void_p]),
    "sfp8_sparse_linear_quant_host": (_i32, [_c_void_p, _c_void_p, _i32, _i32, _c_void_p,
                                             _c_void_p, _i64, _c_void_p, _i32, _c_void_p, _i64,
                                             _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                             _sz, _c_void_p]),
    "sfp8_read_device_status": (_i32, [ctypes.POINTER(ctypes.c_uint32), _i32]),
    "sfp8_last_device_status": (_i32, []),
    "sfp8_status_string": (ctypes.c_char_p, [_i32]),
    "sfp8_layout_version": (_i32, []),
}

_LIB = None


class Sfp8Error(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, STATUS_NAMES.get(status, "?"), status))


def library_path():
    return _build.LIB_PATH


def load_library():
    """Loads libsfp8.so from the package directory (raises if absent)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                "libsfp8.so is not built (%s); run "
                "`python -m semi_structured_sparse_rowwise_b200.build`" % path)
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(status, what):
    if status != OK:
        raise Sfp8Error(status, what)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _fp8_name(d):
    if d not in ("e4m3", "e5m2"):
        raise ValueError("fp8 dtype must be 'e4m3' or 'e5m2'")
    return d


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")


def _ws_bytes(ws, device):
    """Size in bytes of a caller's workspace (any dtype), which must be a
    contiguous CUDA tensor on `device`."""
    if not ws.is_cuda or ws.device != torch.device(device) or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % (device,))
    return ws.numel() * ws.element_size()


def sfp8_quantize_rowwise(x, q_dtype="e4m3", q=None, scales=None):
    """x [rows, cols] bf16/f16/f32 (unit column stride) -> (q uint8, scales f32)."""
    lib = load_library()
    _require_cuda(x)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    rows, cols = x.shape
    xd = TORCH_WIDE.get(x.dtype)
    if xd is None:
        raise ValueError("x dtype must be bfloat16, float16 or float32")
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows,), dtype=torch.float32, device=x.device)
    ld = x.stride(0) if rows > 1 else cols
    with torch.cuda.device(x.device):
        st = lib.sfp8_quantize_rowwise(_ptr(x), DTYPE[xd], rows, cols, ld, _ptr(q),
                                       DTYPE[_fp8_name(q_dtype)], _ptr(scales), _stream(x.device))
    _check(st, "sfp8_quantize_rowwise")
    return q, scales


def sfp8_quantize_tensorwise_workspace_bytes(mode="reduce", device=None):
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib.sfp8_quantize_tensorwise_workspace_bytes(AMAX_MODE[mode]))


def new_tensorwise_workspace(mode, device):
    """A zeroed workspace for sfp8_quantize_tensorwise on `device`."""
    nbytes = sfp8_quantize_tensorwise_workspace_bytes(mode, device)
    return torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=device)


def sfp8_quantize_tensorwise(x, q_dtype="e4m3", mode="reduce", q=None, scale=None,
                             workspace=None):
    """x (any shape, contiguous) bf16/f16/f32 -> (q uint8 of x's shape, scale f32 [1]):
    one scale for the whole tensor, the global amax found by `mode`
    ('reduce': per-block partials, 'atomic': one word with atomic max)."""
    lib = load_library()
    _require_cuda(x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    xd = TORCH_WIDE.get(x.dtype)
    if xd is None:
        raise ValueError("x dtype must be bfloat16, float16 or float32")
    if mode not in AMAX_MODE:
        raise ValueError("mode must be 'reduce' or 'atomic'")
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty((1,), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = new_tensorwise_workspace(mode, x.device)
    with torch.cuda.device(x.device):
        st = lib.sfp8_quantize_tensorwise(_ptr(x), DTYPE[xd], x.numel(), _ptr(q),
                                          DTYPE[_fp8_name(q_dtype)], _ptr(scale),
                                          AMAX_MODE[mode], _ptr(workspace),
                                          _ws_bytes(workspace, x.device),
                                          _stream(x.device))
    _check(st, "sfp8_quantize_tensorwise")
    return q, scale


def sfp8_prune_24(w, out=None):
    """2:4 magnitude prune along rows; w [rows, cols] bf16/f16/f32."""
    lib = load_library()
    _require_cuda(w)
    if w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be 2-D with unit column stride")
    wd = TORCH_WIDE.get(w.dtype)
    if wd is None:
        raise ValueError("w dtype must be bfloat16, float16 or float32")
    rows, cols = w.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=w.dtype, device=w.device)
    ld = w.stride(0) if rows > 1 else cols
    with torch.cuda.device(w.device):
        st = lib.sfp8_prune_24(_ptr(w), DTYPE[wd], rows, cols, ld, _ptr(out), _stream(w.device))
    _check(st, "sfp8_prune_24")
    return out


def sfp8_padded_rows(n):
    return int(load_library().sfp8_padded_rows(n))


def sfp8_compressed_bytes(n, k):
    return int(load_library().sfp8_compressed_bytes(n, k))


def sfp8_compress_24(w_q, w_dtype="e4m3", packed=None):
    """w_q [n, k] uint8 FP8 codes -> packed compressed weight (layout v3)."""
    lib = load_library()
    _require_cuda(w_q)
    if w_q.dim() != 2 or not w_q.is_contiguous() or w_q.dtype != torch.uint8:
        raise ValueError("w_q must be a contiguous 2-D uint8 tensor")
    n, k = w_q.shape
    if packed is None:
        packed = torch.empty((lib.sfp8_compressed_bytes(n, k),), dtype=torch.uint8,
                             device=w_q.device)
    with torch.cuda.device(w_q.device):
        st = lib.sfp8_compress_24(_ptr(w_q), DTYPE[_fp8_name(w_dtype)], n, k, _ptr(packed),
                                  _stream(w_q.device))
    _check(st, "sfp8_compress_24")
    return packed


def sfp8_prepare_weight_24(w, q_dtype="e4m3", packed=None, scales=None):
    """w [n, k] bf16/f16/f32 (unit column stride) -> (packed, s_w): prune 2:4,
    quantise row-wise and compress in one pass (the same bytes as
    sfp8_prune_24 -> sfp8_quantize_rowwise -> sfp8_compress_24)."""
    lib = load_library()
    _require_cuda(w)
    if w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be 2-D with unit column stride")
    wd = TORCH_WIDE.get(w.dtype)
    if wd is None:
        raise ValueError("w dtype must be bfloat16, float16 or float32")
    n, k = w.shape
    if packed is None:
        packed = torch.empty((lib.sfp8_compressed_bytes(n, k),), dtype=torch.uint8,
                             device=w.device)
    if scales is None:
        scales = torch.empty((n,), dtype=torch.float32, device=w.device)
    ld = w.stride(0) if n > 1 else k
    with torch.cuda.device(w.device):
        st = lib.sfp8_prepare_weight_24(_ptr(w), DTYPE[wd], n, k, ld, DTYPE[_fp8_name(q_dtype)],
                                        _ptr(packed), _ptr(scales), _stream(w.device))
    _check(st, "sfp8_prepare_weight_24")
    return packed, scales


def sfp8_decompress_24(packed, n, k, out=None):
    lib = load_library()
    _require_cuda(packed)
    if out is None:
        out = torch.empty((n, k), dtype=torch.uint8, device=packed.device)
    with torch.cuda.device(packed.device):
        st = lib.sfp8_decompress_24(_ptr(packed), n, k, _ptr(out), _stream(packed.device))
    _check(st, "sfp8_decompress_24")
    return out


def sfp8_sparse_linear_workspace_bytes(m, n, k, device=None):
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib.sfp8_sparse_linear_workspace_bytes(m, n, k))


def new_workspace(m, n, k, device):
    """A zeroed workspace for sfp8_sparse_linear(m, n, k) on `device`."""
    nbytes = sfp8_sparse_linear_workspace_bytes(m, n, k, device)
    return torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=device)


def sfp8_workspace_clear(workspace):
    lib = load_library()
    with torch.cuda.device(workspace.device):
        st = lib.sfp8_workspace_clear(_ptr(workspace), _ws_bytes(workspace, workspace.device),
                                      _stream(workspace.device))
    _check(st, "sfp8_workspace_clear")


def _linear_args(a_q, n, k, bias, out):
    """Shape, dtype and layout checks shared by the sparse linear wrappers,
    made before anything reaches the library; returns m."""
    if a_q.dim() != 2 or not a_q.is_contiguous() or a_q.dtype != torch.uint8:
        raise ValueError("a_q must be a contiguous 2-D uint8 tensor")
    m = a_q.shape[0]
    if a_q.shape[1] != k:
        raise ValueError("a_q has %d columns, expected k=%d" % (a_q.shape[1], k))
    if bias is not None and (bias.dtype != torch.bfloat16 or bias.dim() != 1
                             or bias.shape[0] != n or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous bfloat16 vector of n=%d elements" % n)
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != (m, n)
                            or not out.is_contiguous() or out.device != a_q.device):
        raise ValueError("out must be a contiguous (m, n) = (%d, %d) bfloat16 tensor on "
                         "a_q's device" % (m, n))
    return m


def sfp8_sparse_linear(a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, bias=None,
                       out=None, workspace=None):
    """y [m, n] bf16 = (s_a s_w^T) * (A_q . W_q^T) + bias."""
    lib = load_library()
    m = _linear_args(a_q, n, k, bias, out)
    _require_cuda(a_q, s_a, packed, s_w, bias)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a_q.device)
    if workspace is None:
        workspace = new_workspace(m, n, k, a_q.device)
    with torch.cuda.device(a_q.device):
        st = lib.sfp8_sparse_linear(_ptr(a_q), DTYPE[_fp8_name(a_dtype)], _ptr(s_a), m,
                                    _ptr(packed), DTYPE[_fp8_name(w_dtype)],
                                    _ptr(s_w), n, k, _ptr(bias), _ptr(out), _ptr(workspace),
                                    _ws_bytes(workspace, a_q.device), _stream(a_q.device))
    _check(st, "sfp8_sparse_linear")
    return out


def sfp8_sparse_linear_noalloc(a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k,
                               bias=None, out=None):
    """sfp8_sparse_linear without a workspace, for callers that cannot
    allocate device memory at call time (see include/sfp8.h): the library's
    built-in scratch buffer is used instead.  `out` must be given by such a
    caller; only when it is None does this wrapper allocate it with torch."""
    lib = load_library()
    m = _linear_args(a_q, n, k, bias, out)
    _require_cuda(a_q, s_a, packed, s_w, bias)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a_q.device)
    with torch.cuda.device(a_q.device):
        st = lib.sfp8_sparse_linear_noalloc(_ptr(a_q), DTYPE[_fp8_name(a_dtype)], _ptr(s_a), m,
                                            _ptr(packed), DTYPE[_fp8_name(w_dtype)],
                                            _ptr(s_w), n, k, _ptr(bias), _ptr(out),
                                            _stream(a_q.device))
    _check(st, "sfp8_sparse_linear_noalloc")
    return out


ALGO_FIELDS = ("pair", "bn", "ks", "wt", "whole_tiles", "ra", "stages", "grid")


def _dev_ctx(device):
    return torch.cuda.device(device if device is not None else torch.cuda.current_device())


def sfp8_sparse_linear_algo_count(m, n, k, device=None):
    with _dev_ctx(device):
        return int(load_library().sfp8_sparse_linear_algo_count(m, n, k))


def sfp8_sparse_linear_algo_info(m, n, k, algo, device=None):
    """dict of the algorithm's work split (keys ALGO_FIELDS)."""
    info = (ctypes.c_int32 * 8)()
    with _dev_ctx(device):
        st = load_library().sfp8_sparse_linear_algo_info(m, n, k, algo, info)
    _check(st, "sfp8_sparse_linear_algo_info")
    return dict(zip(ALGO_FIELDS, [int(v) for v in info]))


PLAN_FIELDS = ("pair", "bn", "ks", "wt", "whole_tiles", "ra", "stages", "grid", "producers",
               "smem_bytes", "workspace_bytes", "m_tiles")


def sfp8_sparse_linear_plan(m, n, k, num_sms, algo=0):
    """Host-only: the plan of an algorithm for a device of num_sms SMs (dict
    of PLAN_FIELDS), no device involved."""
    info = (ctypes.c_int64 * len(PLAN_FIELDS))()
    st = load_library().sfp8_sparse_linear_plan_info(m, n, k, num_sms, algo, info)
    _check(st, "sfp8_sparse_linear_plan_info")
    return dict(zip(PLAN_FIELDS, [int(v) for v in info]))


def sfp8_sparse_linear_plan_count(m, n, k, num_sms):
    return int(load_library().sfp8_sparse_linear_plan_count(m, n, k, num_sms))


def sfp8_sparse_linear_algo_workspace_bytes(m, n, k, algo, device=None):
    with _dev_ctx(device):
        return int(load_library().sfp8_sparse_linear_algo_workspace_bytes(m, n, k, algo))


def sfp8_sparse_linear_search_workspace_bytes(m, n, k, device=None):
    with _dev_ctx(device):
        return int(load_library().sfp8_sparse_linear_search_workspace_bytes(m, n, k))


def sfp8_sparse_linear_algo(a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, algo, bias=None,
                            out=None, workspace=None):
    """sfp8_sparse_linear with an explicit work split (algorithm index)."""
    lib = load_library()
    m = _linear_args(a_q, n, k, bias, out)
    _require_cuda(a_q, s_a, packed, s_w, bias)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a_q.device)
    if workspace is None:
        nbytes = sfp8_sparse_linear_algo_workspace_bytes(m, n, k, algo, a_q.device)
        workspace = torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=a_q.device)
    with torch.cuda.device(a_q.device):
        st = lib.sfp8_sparse_linear_algo(_ptr(a_q), DTYPE[_fp8_name(a_dtype)], _ptr(s_a), m,
                                         _ptr(packed), DTYPE[_fp8_name(w_dtype)], _ptr(s_w), n,
                                         k, _ptr(bias), _ptr(out), algo, _ptr(workspace),
                                         _ws_bytes(workspace, a_q.device), _stream(a_q.device))
    _check(st, "sfp8_sparse_linear_algo")
    return out


def sfp8_sparse_linear_search(a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, bias=None,
                              reps=10, flush=None, out=None):
    """Times every work split of the shape (see include/sfp8.h); returns
    (best algorithm, [median microseconds per algorithm])."""
    lib = load_library()
    m = _linear_args(a_q, n, k, bias, out)
    _require_cuda(a_q, s_a, packed, s_w, bias, flush)
    dev = a_q.device
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    count = sfp8_sparse_linear_algo_count(m, n, k, dev)
    nbytes = sfp8_sparse_linear_search_workspace_bytes(m, n, k, dev)
    ws = torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=dev)
    best = ctypes.c_int32(-1)
    times = (ctypes.c_float * max(count, 1))()
    with torch.cuda.device(dev):
        st = lib.sfp8_sparse_linear_search(_ptr(a_q), DTYPE[_fp8_name(a_dtype)], _ptr(s_a), m,
                                           _ptr(packed), DTYPE[_fp8_name(w_dtype)], _ptr(s_w),
                                           n, k, _ptr(bias), _ptr(out), _ptr(ws), ws.numel(),
                                           _ptr(flush),
                                           0 if flush is None else _ws_bytes(flush, dev),
                                           reps, ctypes.byref(best), times, count, _stream(dev))
    _check(st, "sfp8_sparse_linear_search")
    return int(best.value), [float(t) for t in times[:count]]


# Bumped by every change of the shape-keyed algorithm table made through this
# binding: workspaces cached for a shape are re-sized when it moves.
_ALGO_EPOCH = [0]


def algo_epoch():
    return _ALGO_EPOCH[0]


def sfp8_sparse_linear_set_algo(m, n, k, algo, device=None):
    with _dev_ctx(device):
        st = load_library().sfp8_sparse_linear_set_algo(m, n, k, algo)
    _check(st, "sfp8_sparse_linear_set_algo")
    _ALGO_EPOCH[0] += 1


def sfp8_sparse_linear_get_algo(m, n, k, device=None):
    with _dev_ctx(device):
        return int(load_library().sfp8_sparse_linear_get_algo(m, n, k))


def sfp8_sparse_linear_quant_workspace_bytes(m, n, k, device=None):
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib.sfp8_sparse_linear_quant_workspace_bytes(m, n, k))


def new_quant_workspace(m, n, k, device):
    """A zeroed workspace for sfp8_sparse_linear_quant(m, n, k) on `device`."""
    nbytes = sfp8_sparse_linear_quant_workspace_bytes(m, n, k, device)
    return torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=device)


def sfp8_sparse_linear_quant(x, a_dtype, packed, w_dtype, s_w, n, k, bias=None, out=None,
                             workspace=None, a_q=None, s_a=None):
    """Quantise x [m, k] (bf16/f16/f32, unit column stride) row-wise and apply
    the sparse linear, one library call: returns (y [m, n] bf16,
    a_q [m, k] uint8, s_a [m] f32), by the chained form (quantiser, then
    the GEMM as its programmatic dependent)."""
    return _quant_linear("sfp8_sparse_linear_quant", x, a_dtype, packed, w_dtype, s_w, n, k,
                         bias, out, workspace, a_q, s_a)


def sfp8_sparse_linear_quant_fused(x, a_dtype, packed, w_dtype, s_w, n, k, bias=None, out=None,
                                   workspace=None, a_q=None, s_a=None):
    """sfp8_sparse_linear_quant in its fused form: one kernel in which every
    CTA quantises the (at most 16) rows itself.  Raises Sfp8Error
    (SFP8_ERR_UNSUPPORTED_SHAPE) where the form does not apply."""
    return _quant_linear("sfp8_sparse_linear_quant_fused", x, a_dtype, packed, w_dtype, s_w, n,
                         k, bias, out, workspace, a_q, s_a)


def sfp8_sparse_linear_quant_chained(x, a_dtype, packed, w_dtype, s_w, n, k, bias=None,
                                     out=None, workspace=None, a_q=None, s_a=None):
    """sfp8_sparse_linear_quant in its chained form: the row-wise quantiser,
    then the GEMM as its programmatic dependent."""
    return _quant_linear("sfp8_sparse_linear_quant_chained", x, a_dtype, packed, w_dtype, s_w,
                         n, k, bias, out, workspace, a_q, s_a)


def sfp8_sparse_linear_quant_fusable(m, n, k, device=None):
    """Whether sfp8_sparse_linear_quant_fused accepts (m, n, k) on `device`
    (host-only query)."""
    lib = load_library()
    with _dev_ctx(device):
        return bool(lib.sfp8_sparse_linear_quant_fusable(m, n, k))


def _quant_linear(name, x, a_dtype, packed, w_dtype, s_w, n, k, bias, out, workspace, a_q, s_a):
    lib = load_library()
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x has %d columns, expected k=%d" % (x.shape[1], k))
    xd = TORCH_WIDE.get(x.dtype)
    if xd is None:
        raise ValueError("x dtype must be bfloat16, float16 or float32")
    if bias is not None and bias.dtype != torch.bfloat16:
        raise ValueError("bias must be bfloat16")
    dev = x.device
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
    if a_q is None:
        a_q = torch.empty((m, k), dtype=torch.uint8, device=dev)
    if s_a is None:
        s_a = torch.empty((m,), dtype=torch.float32, device=dev)
    for t, shape, dtype, what in ((out, (m, n), torch.bfloat16, "out"),
                                  (a_q, (m, k), torch.uint8, "a_q"),
                                  (s_a, (m,), torch.float32, "s_a")):
        if (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()
                or t.device != dev):
            raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                             % (what, dtype, shape, dev))
    _require_cuda(x, packed, s_w, bias)
    if workspace is None:
        workspace = new_quant_workspace(m, n, k, dev)
    ld = x.stride(0) if m > 1 else k
    with torch.cuda.device(dev):
        st = getattr(lib, name)(_ptr(x), DTYPE[xd], ld, DTYPE[_fp8_name(a_dtype)], _ptr(a_q),
                                _ptr(s_a), m, _ptr(packed), DTYPE[_fp8_name(w_dtype)],
                                _ptr(s_w), n, k, _ptr(bias), _ptr(out), _ptr(workspace),
                                _ws_bytes(workspace, dev), _stream(dev))
    _check(st, name)
    return out, a_q, s_a


# ---------------------------------------------------------------- feed-forward sublayer
# The wrappers below are called once a layer and token in serving, where the
# host's share of a call is as long as its kernels (on a B200 host: 4 us in the
# library, 1.3 to 2.3 us for each result that torch allocates, and what
# Python adds).  So they check their arguments in few, flat expressions that only a
# refusal takes apart again, pass plain integers for pointers and read the
# device and the raw stream directly; torch's device context manager, stream
# object and ctypes pointer objects alone would take 10 us more.

# absent from a torch without CUDA, which still imports this module
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_U8, _F32, _BF16 = torch.uint8, torch.float32, torch.bfloat16
_WIDE_CODE = {t: DTYPE[name] for t, name in TORCH_WIDE.items()}
_FP8_CODE = {"e4m3": DTYPE["e4m3"], "e5m2": DTYPE["e5m2"]}
_FN = {}


def _run(name, device, *args):
    """Calls the library on `device`'s current stream (the last argument) and
    raises on a status other than OK."""
    fn = _FN.get(name)
    if fn is None:
        fn = _FN[name] = getattr(load_library(), name)
    index = device.index
    if _get_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status != OK:
        raise Sfp8Error(status, name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _fp8(dtype):
    code = _FP8_CODE.get(dtype)
    if code is None:
        raise ValueError("fp8 dtype must be 'e4m3' or 'e5m2'")
    return code


def _activation(act):
    code = ACTIVATION.get(act)
    if code is None:
        raise ValueError("act must be 'silu' or 'gelu'")
    return code


def _tensor(t, what, shape, dtype, device):
    """Refuses anything but a contiguous CUDA tensor of this shape (a tuple),
    dtype and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (what, dtype, tuple(shape), device))


def _like(x, t, what, dtype):
    """A contiguous output of x's shape: given (checked) or new (empty_like is
    the cheaper call where it gives that)."""
    if t is not None:
        _tensor(t, what, x.shape, dtype, x.device)
        return t
    return torch.empty_like(x, dtype=dtype) if x.is_contiguous() else x.new_empty(x.shape,
                                                                                 dtype=dtype)


def _rows_in(x, what, cols=None):
    """A 2-D CUDA input with unit column stride (and `cols` columns): the code
    of its type, its rows, columns and row stride."""
    code = _WIDE_CODE.get(x.dtype)
    shape = x.shape
    if code is None or not x.is_cuda or len(shape) != 2:
        raise ValueError("%s must be a 2-D CUDA tensor of bfloat16, float16 or float32" % what)
    rows, width = shape
    ld, unit = x.stride()
    if (unit != 1 and width > 1) or (cols is not None and width != cols):
        raise ValueError("%s must have unit column stride%s"
                         % (what, "" if cols is None else " and %d columns" % cols))
    return code, rows, width, ld if rows > 1 else width


def _weight(packed, s_w, rows, k, device):
    """The compressed weight of `rows` rows and its scales, on `device`."""
    need = (rows + 127) // 128 * 128 * k * 5 // 8
    if (rows < 0 or k < 0 or packed.dtype != _U8 or packed.device != device
            or not packed.is_contiguous() or packed.numel() < need):
        raise ValueError("packed must be a contiguous uint8 tensor of at least %d bytes on %s "
                         "(n and k not negative)" % (need, device))
    if (s_w.shape != (rows,) or s_w.dtype != _F32 or s_w.device != device
            or not s_w.is_contiguous()):
        _tensor(s_w, "s_w", (rows,), _F32, device)


def _codes(a_q, s_a, k):
    """A quantised activation [m, k] and its scales: its rows and device."""
    shape = a_q.shape
    if (len(shape) != 2 or shape[1] != k or a_q.dtype != _U8 or not a_q.is_cuda
            or not a_q.is_contiguous()):
        raise ValueError("a_q must be a contiguous uint8 CUDA tensor [m, k=%d]" % k)
    m, dev = shape[0], a_q.device
    if s_a.shape != (m,) or s_a.dtype != _F32 or s_a.device != dev or not s_a.is_contiguous():
        _tensor(s_a, "s_a", (m,), _F32, dev)
    return m, dev


def _workspace(ws, device):
    """Address and size of a caller's workspace (any dtype), which must be a
    contiguous CUDA tensor on `device`."""
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % (device,))
    return ws.data_ptr(), ws.nbytes


def _new_workspace(query, sizes, device):
    with torch.cuda.device(device):
        nbytes = int(query(*sizes))
    return torch.zeros((max(nbytes, 16),), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=4096)
def _scratch_bytes(query, sizes, index):
    with torch.cuda.device(index):
        return max(int(getattr(load_library(), query)(*sizes)), 16)


def _new_scratch(query, sizes, device):
    """A workspace that needs no clearing; its size is a matter of the call's
    sizes and the device only, and is asked for once."""
    index = torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    return torch.empty((_scratch_bytes(query, sizes, index),), dtype=torch.uint8, device=device)


# ---- gated block


def sfp8_prepare_gated_weight_24(w_gate, w_up, q_dtype="e4m3", packed=None, scales=None):
    """w_gate, w_up [n, k] bf16/f16/f32 (unit column stride, the same type and
    strides) -> (packed, s_w): the compressed weight of a gated block, 2n rows
    that alternate gate and up, each prepared as by sfp8_prepare_weight_24."""
    wd, n, k, ld = _rows_in(w_gate, "w_gate")
    dev = w_gate.device
    if w_up.device != dev or _rows_in(w_up, "w_up") != (wd, n, k, ld):
        raise ValueError("w_up must have w_gate's shape, dtype, device and strides")
    if packed is None:
        packed = torch.empty((load_library().sfp8_compressed_bytes(2 * n, k),),
                             dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((2 * n,), dtype=torch.float32, device=dev)
    _weight(packed, scales, 2 * n, k, dev)
    _run("sfp8_prepare_gated_weight_24", dev, w_gate.data_ptr(), w_up.data_ptr(), wd, n, k, ld,
         _fp8(q_dtype), packed.data_ptr(), scales.data_ptr())
    return packed, scales


def new_gated_workspace(m, n, k, device):
    """A zeroed workspace for sfp8_gated_linear(m, n, k) on `device`."""
    return _new_workspace(load_library().sfp8_gated_linear_workspace_bytes, (m, n, k), device)


def new_gated_quant_workspace(m, n, k, device):
    """A zeroed workspace for sfp8_gated_linear_quant(m, n, k) on `device`."""
    return _new_workspace(load_library().sfp8_gated_linear_quant_workspace_bytes, (m, n, k),
                          device)


def sfp8_gated_linear(a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, act="silu", bias=None,
                      out=None, workspace=None):
    """h [m, n] bf16 = act(gate) * up of a quantised activation a_q [m, k],
    s_a [m]; packed, s_w from sfp8_prepare_gated_weight_24, bias [2n] bf16
    (gate's n values, then up's)."""
    m, dev = _codes(a_q, s_a, k)
    _weight(packed, s_w, 2 * n, k, dev)
    if bias is not None:
        _tensor(bias, "bias", (2 * n,), _BF16, dev)
    if out is None:
        out = a_q.new_empty((m, n), dtype=_BF16)
    else:
        _tensor(out, "out", (m, n), _BF16, dev)
    if workspace is None:
        workspace = new_gated_workspace(m, n, k, dev)
    _run("sfp8_gated_linear", dev, a_q.data_ptr(), _fp8(a_dtype), s_a.data_ptr(), m,
         packed.data_ptr(), _fp8(w_dtype), s_w.data_ptr(), n, k, _activation(act), _addr(bias),
         out.data_ptr(), *_workspace(workspace, dev))
    return out


def sfp8_gated_linear_quant(x, a_dtype, packed, w_dtype, s_w, n, k, act="silu", bias=None,
                            out=None, workspace=None, a_q=None, s_a=None):
    """Quantise x [m, k] (bf16/f16/f32, unit column stride) row-wise and apply
    the gated block, one library call: returns (h [m, n] bf16, a_q [m, k]
    uint8, s_a [m] f32); a_q and s_a are what the backward pass needs."""
    xd, m, _, ld = _rows_in(x, "x", k)
    dev = x.device
    _weight(packed, s_w, 2 * n, k, dev)
    if bias is not None:
        _tensor(bias, "bias", (2 * n,), _BF16, dev)
    if out is None:
        out = x.new_empty((m, n), dtype=_BF16)
    else:
        _tensor(out, "out", (m, n), _BF16, dev)
    a_q = _like(x, a_q, "a_q", _U8)
    if s_a is None:
        s_a = s_w.new_empty(m)
    else:
        _tensor(s_a, "s_a", (m,), _F32, dev)
    if workspace is None:
        workspace = new_gated_quant_workspace(m, n, k, dev)
    _run("sfp8_gated_linear_quant", dev, x.data_ptr(), xd, ld, _fp8(a_dtype), a_q.data_ptr(),
         s_a.data_ptr(), m, packed.data_ptr(), _fp8(w_dtype), s_w.data_ptr(), n, k,
         _activation(act), _addr(bias), out.data_ptr(), *_workspace(workspace, dev))
    return out, a_q, s_a


# ---- backward passes


def new_linear_backward_workspace(m, n, k, device):
    """A workspace for sfp8_sparse_linear_backward(m, n, k) on `device`."""
    return _new_scratch("sfp8_sparse_linear_backward_workspace_bytes", (m, n, k), device)


def new_gated_backward_workspace(m, n, k, device):
    """A workspace for sfp8_gated_linear_backward(m, n, k) on `device`."""
    return _new_scratch("sfp8_gated_linear_backward_workspace_bytes", (m, n, k), device)


def _gradient(t, wanted, what, shape, like):
    """A bf16 gradient asked for: given (checked) or new; None where it is not."""
    if t is not None:
        _tensor(t, what, shape, _BF16, like.device)
        return t
    return like.new_empty(shape) if wanted else None


def _grad_in(dy, what, m, n, device):
    """Row stride of the output's gradient [m, n] bf16, unit column stride."""
    if dy.dtype != _BF16 or dy.shape != (m, n) or dy.device != device:
        raise ValueError("%s must be a bfloat16 tensor of shape %s on %s" % (what, (m, n), device))
    return _rows_in(dy, what)[3]


def sfp8_sparse_linear_backward(dy, a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, need_dx=True,
                                need_dw=True, need_dbias=False, dx=None, dw=None, dbias=None,
                                workspace=None):
    """Gradients of the sparse linear from dy [m, n] bf16 and the forward's
    8-bit checkpoint a_q [m, k], s_a [m]: returns (dx [m, k], dw [n, k],
    dbias [n]), bf16, None where not asked for.  A given dx, dw or dbias is
    written (and counts as asked for)."""
    m, dev = _codes(a_q, s_a, k)
    _weight(packed, s_w, n, k, dev)
    ld = _grad_in(dy, "dy", m, n, dev)
    dx = _gradient(dx, need_dx, "dx", (m, k), dy)
    dw = _gradient(dw, need_dw, "dw", (n, k), dy)
    dbias = _gradient(dbias, need_dbias, "dbias", (n,), dy)
    if workspace is None:
        workspace = a_q.new_empty(
            _scratch_bytes("sfp8_sparse_linear_backward_workspace_bytes", (m, n, k), dev.index))
    _run("sfp8_sparse_linear_backward", dev, dy.data_ptr(), ld, a_q.data_ptr(), _fp8(a_dtype),
         s_a.data_ptr(), m, packed.data_ptr(), _fp8(w_dtype), s_w.data_ptr(), n, k, _addr(dx),
         _addr(dw), _addr(dbias), *_workspace(workspace, dev))
    return dx, dw, dbias


def sfp8_gated_linear_backward(dh, a_q, a_dtype, s_a, packed, w_dtype, s_w, n, k, act="silu",
                               bias=None, need_dx=True, need_dw=True, need_dbias=False, dx=None,
                               dw=None, dbias=None, workspace=None):
    """Gradients of the gated block from dh [m, n] bf16 and the forward's
    8-bit checkpoint a_q [m, k], s_a [m]: returns (dx [m, k], dw [2n, k],
    dbias [2n]), bf16, None where not asked for; dw's and dbias's first n rows
    are gate's, the others up's."""
    m, dev = _codes(a_q, s_a, k)
    _weight(packed, s_w, 2 * n, k, dev)
    if bias is not None:
        _tensor(bias, "bias", (2 * n,), _BF16, dev)
    ld = _grad_in(dh, "dh", m, n, dev)
    dx = _gradient(dx, need_dx, "dx", (m, k), dh)
    dw = _gradient(dw, need_dw, "dw", (2 * n, k), dh)
    dbias = _gradient(dbias, need_dbias, "dbias", (2 * n,), dh)
    if workspace is None:
        workspace = a_q.new_empty(
            _scratch_bytes("sfp8_gated_linear_backward_workspace_bytes", (m, n, k), dev.index))
    _run("sfp8_gated_linear_backward", dev, dh.data_ptr(), ld, a_q.data_ptr(), _fp8(a_dtype),
         s_a.data_ptr(), m, packed.data_ptr(), _fp8(w_dtype), s_w.data_ptr(), n, k,
         _activation(act), _addr(bias), _addr(dx), _addr(dw), _addr(dbias),
         *_workspace(workspace, dev))
    return dx, dw, dbias


# ---- layer norm


def _norm_in(x, weight, bias):
    """Checks layer norm's inputs: the codes of x's and the parameters' types, x's
    rows, columns and row stride, its device."""
    xd, rows, cols, ld = _rows_in(x, "x")
    dtype, dev = x.dtype, x.device
    pd = None
    for t in (weight, bias):
        if t is None:
            continue
        td = t.dtype
        if ((td != dtype and td != _F32) or (pd is not None and td != pd) or t.shape != (cols,)
                or t.device != dev or not t.is_contiguous()):
            raise ValueError("weight and bias must be contiguous tensors of shape %s on %s, both "
                             "of x's dtype or both float32" % ((cols,), dev))
        pd = td
    return xd, rows, cols, ld, xd if pd is None else _WIDE_CODE[pd], dev


def _row_vector(t, what, rows, dev, like=None):
    """A float32 [rows] output: given (checked) or new."""
    if t is not None:
        _tensor(t, what, (rows,), _F32, dev)
        return t
    if like is None:
        return torch.empty((rows,), dtype=_F32, device=dev)
    return torch.empty_like(like)  # the cheaper call


def sfp8_layernorm(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None):
    """Layer norm of x [rows, cols] bf16/f16/f32 (unit column stride), weight
    and bias [cols] of x's dtype or float32: returns (y of x's dtype, mean
    [rows], rstd [rows] float32)."""
    xd, rows, cols, ld, pd, dev = _norm_in(x, weight, bias)
    out = _like(x, out, "out", x.dtype)
    mean = _row_vector(mean, "mean", rows, dev)
    rstd = _row_vector(rstd, "rstd", rows, dev, mean)
    _run("sfp8_layernorm", dev, x.data_ptr(), xd, rows, cols, ld, _addr(weight), _addr(bias), pd,
         eps, out.data_ptr(), None, _FP8_CODE["e4m3"], None, mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def sfp8_layernorm_quant(x, weight=None, bias=None, eps=1e-5, q_dtype="e4m3", q=None, scales=None,
                         mean=None, rstd=None, out=None):
    """Layer norm of x straight to row-wise FP8 codes, the input of the linear
    and the gated block: returns (q [rows, cols] uint8, scales, mean, rstd
    [rows] float32).  A given `out` also receives y in x's dtype."""
    xd, rows, cols, ld, pd, dev = _norm_in(x, weight, bias)
    q = _like(x, q, "q", _U8)
    if out is not None:
        _tensor(out, "out", x.shape, x.dtype, dev)
    scales = _row_vector(scales, "scales", rows, dev)
    mean = _row_vector(mean, "mean", rows, dev, scales)
    rstd = _row_vector(rstd, "rstd", rows, dev, scales)
    _run("sfp8_layernorm", dev, x.data_ptr(), xd, rows, cols, ld, _addr(weight), _addr(bias), pd,
         eps, _addr(out), q.data_ptr(), _fp8(q_dtype), scales.data_ptr(), mean.data_ptr(),
         rstd.data_ptr())
    return q, scales, mean, rstd


def new_layernorm_backward_workspace(rows, cols, device):
    """A workspace for sfp8_layernorm_backward on `device`."""
    return _new_scratch("sfp8_layernorm_backward_workspace_bytes", (rows, cols), device)


def sfp8_layernorm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None,
                            workspace=None):
    """Gradients of layer norm from dy [rows, cols] (x's dtype) and the
    forward's x, weight (or None), mean and rstd: returns (dx of x's dtype,
    dweight, dbias [cols] float32)."""
    xd, rows, cols, ld_x, pd, dev = _norm_in(x, weight, None)
    dyd, dy_rows, dy_cols, ld_dy = _rows_in(dy, "dy")
    if dyd != xd or dy_rows != rows or dy_cols != cols or dy.device != dev:
        raise ValueError("dy must have x's shape, dtype and device")
    for t, what in ((mean, "mean"), (rstd, "rstd")):
        if t.shape != (rows,) or t.dtype != _F32 or t.device != dev or not t.is_contiguous():
            _tensor(t, what, (rows,), _F32, dev)
    dx = _like(x, dx, "dx", x.dtype)
    if dweight is None:
        dweight = mean.new_empty(cols)
    else:
        _tensor(dweight, "dweight", (cols,), _F32, dev)
    dbias = _row_vector(dbias, "dbias", cols, dev, dweight)
    if workspace is None:
        workspace = new_layernorm_backward_workspace(rows, cols, dev)
    _run("sfp8_layernorm_backward", dev, dy.data_ptr(), ld_dy, x.data_ptr(), xd, rows, cols, ld_x,
         _addr(weight), pd, mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
         dbias.data_ptr(), *_workspace(workspace, dev))
    return dx, dweight, dbias


def sfp8_selftest_timeout(device=None):
    """Runs the library's failure-path self-test on `device` (a bounded wait
    that runs out, about a second); read the status word afterwards."""
    lib = load_library()
    with _dev_ctx(device):
        dev = torch.cuda.current_device()
        st = lib.sfp8_selftest_timeout(_stream(dev))
    _check(st, "sfp8_selftest_timeout")


def sfp8_sparse_linear_quant_host(x_host, a_dtype, packed, w_dtype, s_w, n, k, x_dev, a_q, s_a,
                                  y_dev, y_host, workspace, bias=None):
    """Host x [m, k] -> host y [m, n] in one library call: copy in, quantise,
    sparse linear, copy out, all on the current stream (page-locked host
    tensors keep it asynchronous).  Every buffer is given by the caller."""
    lib = load_library()
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("x_host and y_host must be host tensors")
    if not (x_host.is_contiguous() and y_host.is_contiguous() and x_dev.is_contiguous()
            and y_dev.is_contiguous()):
        raise ValueError("x_host, x_dev, y_dev and y_host must be contiguous")
    m = x_host.shape[0]
    if (x_host.shape != (m, k) or x_dev.shape != (m, k) or y_host.shape != (m, n)
            or y_dev.shape != (m, n) or y_dev.dtype != torch.bfloat16):
        raise ValueError("shapes: x_host/x_dev [m, k], y_host/y_dev [m, n] (y bfloat16)")
    xd = TORCH_WIDE.get(x_host.dtype)
    if xd is None or x_dev.dtype != x_host.dtype or y_host.dtype != torch.bfloat16:
        raise ValueError("x dtype bfloat16/float16/float32 (same on host and device), y bfloat16")
    _require_cuda(x_dev, a_q, s_a, packed, s_w, bias, y_dev, workspace)
    dev = x_dev.device
    with torch.cuda.device(dev):
        st = lib.sfp8_sparse_linear_quant_host(
            _ptr(x_host), _ptr(x_dev), DTYPE[xd], DTYPE[_fp8_name(a_dtype)], _ptr(a_q), _ptr(s_a),
            m, _ptr(packed), DTYPE[_fp8_name(w_dtype)], _ptr(s_w), n, k, _ptr(bias), _ptr(y_dev),
            _ptr(y_host), _ptr(workspace), _ws_bytes(workspace, dev), _stream(dev))
    _check(st, "sfp8_sparse_linear_quant_host")
    return y_host


def sfp8_read_device_status(clear=True):
    """(status, flags) of the current device's status word; synchronises."""
    lib = load_library()
    flags = ctypes.c_uint32(0)
    st = lib.sfp8_read_device_status(ctypes.byref(flags), 1 if clear else 0)
    return st, flags.value


def sfp8_last_device_status():
    """Status of the current device's status word (not cleared); synchronises."""
    return int(load_library().sfp8_last_device_status())


def sfp8_compressed_values_bytes(n, k):
    return int(load_library().sfp8_compressed_values_bytes(n, k))


def sfp8_compressed_meta_bytes(n, k):
    return int(load_library().sfp8_compressed_meta_bytes(n, k))


def sfp8_status_string(status):
    return load_library().sfp8_status_string(status).decode()


def sfp8_layout_version():
    return int(load_library().sfp8_layout_version())
