"""Thin ctypes binding of the EXL3 B200 C ABI (include/exl3.h): layers of trellis
weights, 4-bit microscaled matrices (exl3_mx4_*) and expert routing (exl3_moe_*).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libexl3_b200.so.  PyTorch supplies device memory and streams.
There is no CPU fallback: if the library cannot be built or loaded, or no
CUDA device is present, these functions raise.
"""
import ctypes
import os
import threading

import torch

from . import build as _build

EXL3_OK = 0
EXL3_ERR_INVALID_ARG = 1
EXL3_ERR_UNSUPPORTED = 2
EXL3_ERR_WORKSPACE = 3
EXL3_ERR_CUDA = 4
EXL3_ERR_TIMEOUT = 5

# Every symbol the public headers declare.
EXPORTED = ["exl3_status_string", "exl3_version", "exl3_hadamard", "exl3_decode_tiles",
            "exl3_gemv_workspace_size", "exl3_gemv", "exl3_gemv_multi_workspace_size", "exl3_gemv_multi",
            "exl3_gemv_noalloc_max_scratch",
            "exl3_gemv_noalloc", "exl3_gemm_workspace_size", "exl3_gemm",
            "exl3_matmul_workspace_size", "exl3_matmul",
            "exl3_gemm_multi_workspace_size", "exl3_gemm_multi",
            "exl3_matmul_multi_workspace_size", "exl3_matmul_multi",
            "exl3_encode_workspace_size", "exl3_encode", "exl3_udu_workspace_size", "exl3_udu",
            "exl3_ldlq_workspace_size", "exl3_ldlq",
            "exl3_workspace_status", "exl3_set_launch_flags", "exl3_launch_flags",
            "exl3_debug_set_wait_limit_ns", "exl3_debug_wait_limit_ns"]

EXPORTED += ["exl3_mx4_scale_stride", "exl3_mx4_quantize", "exl3_mx4_dequantize",
             "exl3_mx4_matmul_workspace_size", "exl3_mx4_matmul", "exl3_mx4_linear_workspace_size",
             "exl3_mx4_linear", "exl3_mx4_matmul_experts_workspace_size", "exl3_mx4_matmul_experts",
             "exl3_moe_sort_workspace_size", "exl3_moe_sort", "exl3_moe_gather", "exl3_moe_combine",
             "exl3_moe_combine_grad"]

EXL3_LAUNCH_PDL = 1

# exl3_dtype
DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

_lib = None
_lock = threading.Lock()


class Exl3Linear(ctypes.Structure):
    """The C struct exl3_linear: one layer of an exl3_gemv_multi call."""
    _fields_ = [("x", ctypes.c_void_p), ("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p),
                ("svh", ctypes.c_void_p), ("y", ctypes.c_void_p), ("k", ctypes.c_int64),
                ("n", ctypes.c_int64), ("K", ctypes.c_int)]


class Exl3Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def library_path():
    return _build.LIB


def load(build_if_needed=True):
    """Load (building first if the sources are newer) the shared library."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build() if build_if_needed else _build.LIB
        if not os.path.exists(path):
            raise RuntimeError("EXL3 CUDA library not found at %s" % path)
        lib = ctypes.CDLL(path)
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        ci = ctypes.c_int
        lib.exl3_status_string.argtypes = [ci]
        lib.exl3_status_string.restype = ctypes.c_char_p
        lib.exl3_version.argtypes = []
        lib.exl3_version.restype = ctypes.c_char_p
        lib.exl3_hadamard.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        lib.exl3_hadamard.restype = ci
        lib.exl3_decode_tiles.argtypes = [vp, vp, i64, i64, ci, vp]
        lib.exl3_decode_tiles.restype = ci
        for name in ("exl3_gemv_workspace_size", "exl3_gemm_workspace_size", "exl3_matmul_workspace_size"):
            getattr(lib, name).argtypes = [i64, i64, i64, ci]
            getattr(lib, name).restype = sz
        for name in ("exl3_gemv", "exl3_gemm", "exl3_matmul"):
            getattr(lib, name).argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp, sz, vp]
            getattr(lib, name).restype = ci
        for kind in ("gemv", "gemm", "matmul"):
            getattr(lib, "exl3_%s_multi_workspace_size" % kind).argtypes = [ctypes.POINTER(Exl3Linear), ci, i64]
            getattr(lib, "exl3_%s_multi_workspace_size" % kind).restype = sz
            getattr(lib, "exl3_%s_multi" % kind).argtypes = [ctypes.POINTER(Exl3Linear), ci, i64, vp, sz, vp]
            getattr(lib, "exl3_%s_multi" % kind).restype = ci
        lib.exl3_gemv_noalloc_max_scratch.argtypes = []
        lib.exl3_gemv_noalloc_max_scratch.restype = sz
        lib.exl3_gemv_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, vp]
        lib.exl3_gemv_noalloc.restype = ci
        lib.exl3_encode_workspace_size.argtypes = [i64, i64, ci]
        lib.exl3_encode_workspace_size.restype = sz
        lib.exl3_encode.argtypes = [vp, vp, vp, i64, i64, ci, vp, sz, vp]
        lib.exl3_encode.restype = ci
        lib.exl3_udu_workspace_size.argtypes = [i64]
        lib.exl3_udu_workspace_size.restype = sz
        lib.exl3_udu.argtypes = [vp, vp, i64, vp, sz, vp]
        lib.exl3_udu.restype = ci
        lib.exl3_ldlq_workspace_size.argtypes = [i64, i64, ci]
        lib.exl3_ldlq_workspace_size.restype = sz
        lib.exl3_ldlq.argtypes = [vp, vp, vp, vp, i64, i64, ci, vp, sz, vp]
        lib.exl3_ldlq.restype = ci
        lib.exl3_mx4_scale_stride.argtypes = [i64]
        lib.exl3_mx4_scale_stride.restype = i64
        lib.exl3_mx4_quantize.argtypes = [vp, ci, vp, ci, vp, i64, i64, vp, vp, i64, i64, vp]
        lib.exl3_mx4_dequantize.argtypes = [vp, vp, vp, ci, i64, i64, vp]
        lib.exl3_mx4_matmul_workspace_size.argtypes = [i64, i64, i64]
        lib.exl3_mx4_matmul.argtypes = [vp, vp, vp, vp, vp, ci, i64, i64, i64, vp, sz, vp]
        lib.exl3_mx4_linear_workspace_size.argtypes = [i64, i64, i64]
        lib.exl3_mx4_linear.argtypes = [vp, ci, vp, ci, vp, vp, vp, i64, i64, i64, vp, sz, vp]
        lib.exl3_mx4_matmul_experts_workspace_size.argtypes = [i64, i64, i64, i64]
        lib.exl3_mx4_matmul_experts.argtypes = [vp, vp, vp, vp, vp, vp, ci, i64, i64, i64, i64, vp, sz, vp]
        lib.exl3_moe_sort_workspace_size.argtypes = [i64, i64, i64]
        lib.exl3_moe_sort.argtypes = [vp, i64, i64, i64, vp, vp, vp, sz, vp]
        lib.exl3_moe_gather.argtypes = [vp, ci, vp, i64, i64, i64, i64, vp, vp]
        lib.exl3_moe_combine.argtypes = [vp, ci, vp, vp, i64, i64, i64, i64, vp, ci, vp]
        lib.exl3_moe_combine_grad.argtypes = [vp, vp, ci, vp, vp, i64, i64, i64, i64, vp, vp, vp]
        for name in ("mx4_matmul", "mx4_linear", "mx4_matmul_experts", "moe_sort"):
            getattr(lib, "exl3_%s_workspace_size" % name).restype = sz
        for name in ("mx4_quantize", "mx4_dequantize", "mx4_matmul", "mx4_linear", "mx4_matmul_experts",
                     "moe_sort", "moe_gather", "moe_combine", "moe_combine_grad"):
            getattr(lib, "exl3_" + name).restype = ci
        lib.exl3_workspace_status.argtypes = [vp, sz, ci, vp]
        lib.exl3_workspace_status.restype = ci
        lib.exl3_set_launch_flags.argtypes = [ctypes.c_uint]
        lib.exl3_set_launch_flags.restype = None
        lib.exl3_launch_flags.argtypes = []
        lib.exl3_launch_flags.restype = ctypes.c_uint
        lib.exl3_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        lib.exl3_debug_set_wait_limit_ns.restype = None
        lib.exl3_debug_wait_limit_ns.argtypes = []
        lib.exl3_debug_wait_limit_ns.restype = ctypes.c_uint64
        _lib = lib
        return lib


def status_string(status):
    return load().exl3_status_string(int(status)).decode()


def version():
    return load().exl3_version().decode()


def _check(status, where):
    if status != EXL3_OK:
        raise Exl3Error(status, where)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _ptr_or_none(t, dtype, name):
    return None if t is None else _dev(t, dtype, name)


def _check_layer_shapes(x, trellis, suh, svh, K, y):
    """Sizes of a layer's tensors against (m, k, n, K), checked before the C
    call so that an undersized tensor never reaches a kernel."""
    if x.dim() != 2:
        raise ValueError("x must be m x k")
    m, k = x.shape
    n = svh.numel()
    if suh.numel() != k:
        raise ValueError("suh must have k = %d elements, has %d" % (k, suh.numel()))
    if k % 16 or n % 16 or trellis.numel() != (k // 16) * (n // 16) * 16 * int(K):
        raise ValueError("trellis must have (k/16)(n/16)16K = %d words for k=%d, n=%d, K=%d, has %d"
                         % ((k // 16) * (n // 16) * 16 * int(K), k, n, int(K), trellis.numel()))
    if y is not None and tuple(y.shape) != (m, n):
        raise ValueError("y must be m x n = %d x %d, is %s" % (m, n, tuple(y.shape)))
    return m, k, n


# ----------------------------------------------------------------- calls ---

def exl3_hadamard(x, y=None, pre=None, post=None, stream=None):
    """y = H128(x .* pre)/sqrt(128) .* post, blockwise over the last dimension."""
    rows, cols = x.shape
    if y is None:
        y = torch.empty_like(x)
    _check(load().exl3_hadamard(_dev(x, torch.float16, "x"), _dev(y, torch.float16, "y"), rows, cols,
                                _ptr_or_none(pre, torch.float16, "pre"),
                                _ptr_or_none(post, torch.float16, "post"), _stream(stream)),
           "exl3_hadamard")
    return y


def exl3_decode_tiles(trellis, k, n, K, w=None, stream=None):
    """Dense k x n fp16 weights decoded from a [k/16, n/16, 16K] uint16 trellis."""
    if w is None:
        w = torch.empty((k, n), dtype=torch.float16, device=trellis.device)
    _check(load().exl3_decode_tiles(_dev(trellis, torch.uint16, "trellis"), _dev(w, torch.float16, "w"),
                                    k, n, K, _stream(stream)), "exl3_decode_tiles")
    return w


def exl3_gemv_workspace_size(m, k, n, K):
    return int(load().exl3_gemv_workspace_size(m, k, n, K))


def exl3_gemm_workspace_size(m, k, n, K):
    return int(load().exl3_gemm_workspace_size(m, k, n, K))


def exl3_matmul_workspace_size(m, k, n, K):
    return int(load().exl3_matmul_workspace_size(m, k, n, K))


def new_workspace(nbytes, device=None):
    """Zero-filled workspace buffer (uint8) of at least nbytes, 256-byte aligned."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _linear(fn, name, x, trellis, suh, svh, K, y, workspace, stream):
    m, k, n = _check_layer_shapes(x, trellis, suh, svh, K, y)
    if y is None:
        y = torch.empty((m, n), dtype=torch.float16, device=x.device)
    if workspace is None:
        raise ValueError("%s needs a workspace (see new_workspace / *_workspace_size)" % name)
    _check(fn(_dev(x, torch.float16, "x"), _dev(trellis, torch.uint16, "trellis"),
              _dev(suh, torch.float16, "suh"), _dev(svh, torch.float16, "svh"),
              _dev(y, torch.float16, "y"), m, k, n, int(K), _dev(workspace, torch.uint8, "workspace"),
              workspace.numel(), _stream(stream)), name)
    return y


def exl3_gemv(x, trellis, suh, svh, K, y=None, workspace=None, stream=None):
    """y = svh .* H(H(x .* suh) W_hat) for 1 <= m <= 16 (memory-bound path)."""
    return _linear(load().exl3_gemv, "exl3_gemv", x, trellis, suh, svh, K, y, workspace, stream)


def _linear_array(layers, m):
    """layers: sequence of (x, trellis, suh, svh, K, y) CUDA tensors (y may be None)."""
    arr = (Exl3Linear * len(layers))()
    ys = []
    for i, (x, trellis, suh, svh, K, y) in enumerate(layers):
        if x.shape[0] != m:
            raise ValueError("every layer of a multi call has the same batch size m")
        _, k, n = _check_layer_shapes(x, trellis, suh, svh, K, y)
        if y is None:
            y = torch.empty((m, n), dtype=torch.float16, device=x.device)
        arr[i] = Exl3Linear(_dev(x, torch.float16, "x"), _dev(trellis, torch.uint16, "trellis"),
                            _dev(suh, torch.float16, "suh"), _dev(svh, torch.float16, "svh"),
                            _dev(y, torch.float16, "y"), k, n, int(K))
        ys.append(y)
    return arr, ys


def _multi_workspace_size(kind, layers, m):
    arr, _ = _linear_array(layers, m)
    return int(getattr(load(), "exl3_%s_multi_workspace_size" % kind)(arr, len(layers), m))


def _multi(kind, layers, workspace, stream):
    m = layers[0][0].shape[0]
    arr, ys = _linear_array(layers, m)
    name = "exl3_%s_multi" % kind
    if workspace is None:
        raise ValueError("%s needs a workspace (%s_workspace_size)" % (name, name))
    _check(getattr(load(), name)(arr, len(layers), m, _dev(workspace, torch.uint8, "workspace"),
                                 workspace.numel(), _stream(stream)), name)
    return ys


def exl3_gemv_multi_workspace_size(layers, m):
    """Workspace bytes for exl3_gemv_multi over `layers` (see exl3_gemv_multi)."""
    return _multi_workspace_size("gemv", layers, m)


def exl3_gemv_multi(layers, workspace=None, stream=None):
    """Several independent layers (same m <= 16) in one call: each entry is
    (x, trellis, suh, svh, K, y-or-None); returns the list of y."""
    return _multi("gemv", layers, workspace, stream)


def exl3_gemm_multi_workspace_size(layers, m):
    """Workspace bytes for exl3_gemm_multi over `layers` (see exl3_gemm_multi)."""
    return _multi_workspace_size("gemm", layers, m)


def exl3_gemm_multi(layers, workspace=None, stream=None):
    """Several layers with the same m, k and K through the GEMM in one call
    (entries as for exl3_gemv_multi); returns the list of y."""
    return _multi("gemm", layers, workspace, stream)


def exl3_matmul_multi_workspace_size(layers, m):
    """Workspace bytes for exl3_matmul_multi over `layers`."""
    return _multi_workspace_size("matmul", layers, m)


def exl3_matmul_multi(layers, workspace=None, stream=None):
    """Several layers with the same m, the kernel chosen by m (GEMV multi for
    m <= 16, GEMM multi above); returns the list of y."""
    return _multi("matmul", layers, workspace, stream)


class MultiCall:
    """A prepared multi-layer call (`kind` "gemv", "gemm" or "matmul"): the
    descriptor array is built once, so repeated calls (a decode loop) cost
    only the C call.  `layers` as for exl3_gemv_multi; the tensors must stay
    alive and in place."""

    kind = "matmul"

    def __init__(self, layers, kind=None):
        if kind is not None:
            self.kind = kind
        self.m = layers[0][0].shape[0]
        self.count = len(layers)
        self._arr, self.ys = _linear_array(layers, self.m)
        self._name = "exl3_%s_multi" % self.kind
        self.workspace_size = int(getattr(load(), self._name + "_workspace_size")(self._arr, self.count, self.m))

    def __call__(self, workspace, stream=None):
        _check(getattr(load(), self._name)(self._arr, self.count, self.m, _dev(workspace, torch.uint8, "workspace"),
                                           workspace.numel(), _stream(stream)), self._name)
        return self.ys


class GemvMulti(MultiCall):
    """A prepared exl3_gemv_multi call (see MultiCall)."""

    kind = "gemv"


def exl3_gemv_noalloc_max_scratch():
    return int(load().exl3_gemv_noalloc_max_scratch())


def exl3_gemv_noalloc(x, trellis, suh, svh, K, y, stream=None):
    """exl3_gemv without a workspace: the library's own fixed scratch array is
    used, for callers that cannot allocate device memory (y must be given)."""
    m, k, n = _check_layer_shapes(x, trellis, suh, svh, K, y)
    _check(load().exl3_gemv_noalloc(_dev(x, torch.float16, "x"), _dev(trellis, torch.uint16, "trellis"),
                                    _dev(suh, torch.float16, "suh"), _dev(svh, torch.float16, "svh"),
                                    _dev(y, torch.float16, "y"), m, k, n, int(K), _stream(stream)),
           "exl3_gemv_noalloc")
    return y


def exl3_gemm(x, trellis, suh, svh, K, y=None, workspace=None, stream=None):
    """The same layer on the tensor cores, any m (tuned for m >= 64)."""
    return _linear(load().exl3_gemm, "exl3_gemm", x, trellis, suh, svh, K, y, workspace, stream)


def exl3_matmul(x, trellis, suh, svh, K, y=None, workspace=None, stream=None):
    """The layer for any m, the kernel chosen by the library (GEMV for m <= 16,
    tensor-core GEMM above)."""
    return _linear(load().exl3_matmul, "exl3_matmul", x, trellis, suh, svh, K, y, workspace, stream)


def exl3_encode_workspace_size(k, n, K):
    return int(load().exl3_encode_workspace_size(k, n, K))


def exl3_encode(w, K, trellis=None, cost=None, workspace=None, stream=None):
    """Tail-biting trellis encoding of a k x n fp32 matrix into a [k/16, n/16, 16K]
    uint16 trellis.  Returns (trellis, cost): cost[tk, tn] is the tile's fp32
    squared-error sum."""
    k, n = w.shape
    if trellis is None:
        trellis = torch.empty((k // 16, n // 16, 16 * K), dtype=torch.uint16, device=w.device)
    if cost is None:
        cost = torch.empty((k // 16, n // 16), dtype=torch.float32, device=w.device)
    if workspace is None:
        raise ValueError("exl3_encode needs a workspace (see new_workspace / exl3_encode_workspace_size)")
    _check(load().exl3_encode(_dev(w, torch.float32, "w"), _dev(trellis, torch.uint16, "trellis"),
                              _dev(cost, torch.float32, "cost"), k, n, int(K),
                              _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
           "exl3_encode")
    return trellis, cost


def exl3_udu(h, ud=None, stream=None):
    """Block factorisation H = U D U^T (fp64, 16 x 16 blocks) of a k x k CUDA
    tensor: returns ud with D in the diagonal blocks, U above them, zeros below."""
    k = h.shape[0]
    if ud is None:
        ud = torch.empty_like(h)
    ws = new_workspace(load().exl3_udu_workspace_size(k), device=h.device)
    _check(load().exl3_udu(_dev(h, torch.float64, "h"), _dev(ud, torch.float64, "ud"), k,
                           _dev(ws, torch.uint8, "workspace"), ws.numel(), _stream(stream)), "exl3_udu")
    return ud


def exl3_ldlq_workspace_size(k, n, K):
    return int(load().exl3_ldlq_workspace_size(k, n, K))


def exl3_ldlq(w, h, K, trellis=None, w_hat=None, workspace=None, stream=None):
    """LDLQ of a k x n fp32 layer against the k x k fp64 Hessian h with the
    K-bit trellis encoder.  Returns (trellis, w_hat)."""
    k, n = w.shape
    if trellis is None:
        trellis = torch.empty((k // 16, n // 16, 16 * K), dtype=torch.uint16, device=w.device)
    if w_hat is None:
        w_hat = torch.empty((k, n), dtype=torch.float32, device=w.device)
    if workspace is None:
        raise ValueError("exl3_ldlq needs a workspace (see new_workspace / exl3_ldlq_workspace_size)")
    _check(load().exl3_ldlq(_dev(w, torch.float32, "w"), _dev(h, torch.float64, "h"),
                            _dev(trellis, torch.uint16, "trellis"), _dev(w_hat, torch.float32, "w_hat"), k, n,
                            int(K), _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
           "exl3_ldlq")
    return trellis, w_hat


# ------------------------------------------- 4-bit matrices and experts ---
#
# A decoding step makes these calls by the dozen, each of a few microseconds on
# the GPU, so their checks are written to cost little: one pass over a call's
# tensors, no context manager and no stream object unless one is needed.

_HALF_TYPES = (torch.float16, torch.bfloat16)


def _arg(t, dtype, name, device):
    """Address of a contiguous CUDA tensor of `dtype` on device number `device`."""
    try:
        # a device number belongs to a CUDA tensor: others have -1
        if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, name, device)


def _refuse(t, dtype, name, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.get_device() != device:
        raise ValueError("tensors of one call must be on one device: %s is on %s, not cuda:%d"
                         % (name, t.device, device))


def _device(t, name, types):
    """Device number and exl3_dtype of a call's first tensor."""
    try:
        if t.is_cuda and t.dtype in types:
            return t.get_device(), DTYPES.get(t.dtype)
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype not in types:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in types), t.dtype))
    raise TypeError("%s is no tensor that this call can take" % name)


def _shape(t, shape, name):
    if t.shape != shape:
        raise ValueError("%s must be %s, is %s" % (name, " x ".join(str(s) for s in shape), tuple(t.shape)))


def _new(like, shape, dtype, stream):
    """An output on like's device whose memory belongs to the stream that writes
    it: on another one it could be memory that work queued there still uses, now
    or when the caller has dropped it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _call(name, device, stream, *args):
    """Calls the library on `stream`, or on the current stream of `device`,
    with that device current."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == device:
        s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            s = torch.cuda.current_stream() if stream is None else stream
            status = fn(*args, s.cuda_stream)
    if status != EXL3_OK:
        raise Exl3Error(status, name)


def _workspace(t, name, device):
    if t is None:
        raise ValueError("%s needs a workspace (see new_workspace / %s_workspace_size)" % (name, name))
    return _arg(t, torch.uint8, "workspace", device)


def exl3_mx4_scale_stride(k):
    """Bytes of a row of scales of a 4-bit matrix with k columns (0: no valid k)."""
    return 0 if k <= 0 or k % 32 or k > 1 << 22 else (k + 511) // 512 * 16


def _mx4_stride(k):
    stride = exl3_mx4_scale_stride(k)
    if stride == 0:
        raise ValueError("k = %d must be a multiple of 32 from 32 to 2^22" % k)
    return stride


def _mx4_operand(codes, scales, dims, what):
    """Checks a 4-bit operand's shapes; returns its leading dimensions and k."""
    shape = codes.shape
    if len(shape) != dims + 1:
        raise ValueError("%s codes must have %d dimensions" % (what, dims + 1))
    k = shape[-1] * 2
    _shape(scales, shape[:-1] + (_mx4_stride(k),), what + " scales")
    return shape[:-1], k


def exl3_mx4_quantize(x, signs=None, rotate=False, positions=None, out_rows=None, codes=None, scales=None,
                      stream=None):
    """Rows x k (fp16, bf16, fp32) to 4-bit codes [rows, k/2] and scales
    [rows, exl3_mx4_scale_stride(k)] (uint8), optionally behind the signs and
    the 128-point rotation.  With `positions` (int32 [rows, topk], from
    exl3_moe_sort) row r goes to each of the rows positions[r] of `out_rows`."""
    if x.dim() != 2:
        raise ValueError("x must be rows x k")
    rows, k = x.shape
    stride = _mx4_stride(k)
    topk, to = 1, rows
    if positions is not None:
        if positions.dim() != 2 or positions.shape[0] != rows:
            raise ValueError("positions must be rows x topk")
        topk = positions.shape[1]
        if out_rows is None:
            raise ValueError("positions need out_rows")
        to = int(out_rows)
    device, dtype = _device(x, "x", DTYPES)
    if signs is not None:
        _shape(signs, (k,), "signs")
    if codes is None:
        codes = _new(x, (to, k // 2), torch.uint8, stream)
    else:
        _shape(codes, (to, k // 2), "codes")
    if scales is None:
        scales = _new(x, (to, stride), torch.uint8, stream)
    else:
        _shape(scales, (to, stride), "scales")
    _call("exl3_mx4_quantize", device, stream, _arg(x, x.dtype, "x", device), dtype,
          None if signs is None else _arg(signs, torch.float16, "signs", device), 1 if rotate else 0,
          None if positions is None else _arg(positions, torch.int32, "positions", device), topk, to,
          _arg(codes, torch.uint8, "codes", device), _arg(scales, torch.uint8, "scales", device), rows, k)
    return codes, scales


def exl3_mx4_dequantize(codes, scales, dtype=torch.float16, out=None, stream=None):
    """The values of a 4-bit matrix, rows x k, as fp16, bf16 or fp32."""
    (rows,), k = _mx4_operand(codes, scales, 1, "matrix")
    if out is None:
        out = _new(codes, (rows, k), dtype, stream)
    else:
        _shape(out, (rows, k), "out")
    device, dt = _device(out, "out", DTYPES)
    _call("exl3_mx4_dequantize", device, stream, _arg(codes, torch.uint8, "codes", device),
          _arg(scales, torch.uint8, "scales", device), _arg(out, out.dtype, "out", device), dt, rows, k)
    return out


def exl3_mx4_matmul_workspace_size(m, k, n):
    return int(load().exl3_mx4_matmul_workspace_size(m, k, n))


def exl3_mx4_matmul(xc, xs, wc, ws, dtype=torch.float16, y=None, workspace=None, stream=None):
    """y = x . w^T of two 4-bit matrices (m rows and n rows of k), fp16, bf16 or fp32."""
    (m,), k = _mx4_operand(xc, xs, 1, "x")
    (n,), kw = _mx4_operand(wc, ws, 1, "w")
    if kw != k:
        raise ValueError("x has k = %d, w has %d" % (k, kw))
    if y is None:
        y = _new(xc, (m, n), dtype, stream)
    else:
        _shape(y, (m, n), "y")
    device, dt = _device(y, "y", DTYPES)
    _call("exl3_mx4_matmul", device, stream, _arg(xc, torch.uint8, "x codes", device),
          _arg(xs, torch.uint8, "x scales", device), _arg(wc, torch.uint8, "w codes", device),
          _arg(ws, torch.uint8, "w scales", device), _arg(y, y.dtype, "y", device), dt, m, k, n,
          _workspace(workspace, "exl3_mx4_matmul", device), workspace.numel())
    return y


def exl3_mx4_linear_workspace_size(m, k, n):
    return int(load().exl3_mx4_linear_workspace_size(m, k, n))


def exl3_mx4_linear(x, wc, ws, signs=None, rotate=False, y=None, workspace=None, stream=None):
    """A layer with 4-bit weights (n rows of k): x (m x k, fp16 or bf16) is
    quantised as by exl3_mx4_quantize, then multiplied; y has x's type."""
    if x.dim() != 2:
        raise ValueError("x must be m x k")
    m, k = x.shape
    (n,), kw = _mx4_operand(wc, ws, 1, "w")
    if kw != k:
        raise ValueError("x has k = %d, w has %d" % (k, kw))
    device, dt = _device(x, "x", _HALF_TYPES)
    if signs is not None:
        _shape(signs, (k,), "signs")
    if y is None:
        y = _new(x, (m, n), x.dtype, stream)
    else:
        _shape(y, (m, n), "y")
    _call("exl3_mx4_linear", device, stream, _arg(x, x.dtype, "x", device), dt,
          None if signs is None else _arg(signs, torch.float16, "signs", device), 1 if rotate else 0,
          _arg(wc, torch.uint8, "w codes", device), _arg(ws, torch.uint8, "w scales", device),
          _arg(y, x.dtype, "y", device), m, k, n, _workspace(workspace, "exl3_mx4_linear", device), workspace.numel())
    return y


def exl3_mx4_matmul_experts_workspace_size(rows, k, n, experts):
    return int(load().exl3_mx4_matmul_experts_workspace_size(rows, k, n, experts))


def exl3_mx4_matmul_experts(xc, xs, offsets, wc, ws, dtype=torch.float16, y=None, workspace=None, stream=None):
    """Rows [offsets[e], offsets[e + 1]) of x times expert e's weights, for
    wc [experts, n, k/2]: y rows x n (rows behind offsets[experts] are not written)."""
    (rows,), k = _mx4_operand(xc, xs, 1, "x")
    (experts, n), kw = _mx4_operand(wc, ws, 2, "w")
    if kw != k:
        raise ValueError("x has k = %d, w has %d" % (k, kw))
    _shape(offsets, (experts + 1,), "offsets")
    if y is None:
        y = _new(xc, (rows, n), dtype, stream)
    else:
        _shape(y, (rows, n), "y")
    device, dt = _device(y, "y", DTYPES)
    _call("exl3_mx4_matmul_experts", device, stream, _arg(xc, torch.uint8, "x codes", device),
          _arg(xs, torch.uint8, "x scales", device), _arg(offsets, torch.int32, "offsets", device),
          _arg(wc, torch.uint8, "w codes", device), _arg(ws, torch.uint8, "w scales", device),
          _arg(y, y.dtype, "y", device), dt, rows, k, n, experts,
          _workspace(workspace, "exl3_mx4_matmul_experts", device), workspace.numel())
    return y


def exl3_moe_sort_workspace_size(tokens, topk, experts):
    return int(load().exl3_moe_sort_workspace_size(tokens, topk, experts))


def exl3_moe_sort(ids, experts, offsets=None, positions=None, workspace=None, stream=None):
    """Order of tokens by expert for ids int32 [tokens, topk]: returns offsets
    int32 [experts + 1] and positions int32 [tokens, topk] (-1: no row)."""
    if ids.dim() != 2:
        raise ValueError("ids must be tokens x topk")
    tokens, topk = ids.shape
    device, _ = _device(ids, "ids", (torch.int32,))
    if offsets is None:
        offsets = _new(ids, (experts + 1,), torch.int32, stream)
    else:
        _shape(offsets, (experts + 1,), "offsets")
    if positions is None:
        positions = _new(ids, (tokens, topk), torch.int32, stream)
    else:
        _shape(positions, (tokens, topk), "positions")
    _call("exl3_moe_sort", device, stream, _arg(ids, torch.int32, "ids", device), tokens, topk, experts,
          _arg(offsets, torch.int32, "offsets", device), _arg(positions, torch.int32, "positions", device),
          _workspace(workspace, "exl3_moe_sort", device), workspace.numel())
    return offsets, positions


def _topk(positions, tokens):
    if positions.dim() != 2 or (tokens is not None and positions.shape[0] != tokens):
        raise ValueError("positions must be tokens x topk")
    return positions.shape[1]


def exl3_moe_gather(x, positions, out=None, out_rows=None, stream=None):
    """out[positions[t, j]] = x[t]; `out` (or `out_rows`, default one row per
    choice, for a new one whose other rows are not written)."""
    if x.dim() != 2:
        raise ValueError("x must be tokens x h")
    tokens, h = x.shape
    topk = _topk(positions, tokens)
    device, dt = _device(x, "x", DTYPES)
    if out is None:
        out = _new(x, (tokens * topk if out_rows is None else int(out_rows), h), x.dtype, stream)
    elif out.dim() != 2 or out.shape[1] != h:
        raise ValueError("out must be rows x h")
    _call("exl3_moe_gather", device, stream, _arg(x, x.dtype, "x", device), dt,
          _arg(positions, torch.int32, "positions", device), tokens, topk, h, out.shape[0],
          _arg(out, x.dtype, "out", device))
    return out


def exl3_moe_combine(ys, positions, weights=None, dtype=None, y=None, stream=None):
    """y[t] = sum over j of weights[t, j] ys[positions[t, j]] (weights fp32,
    None: ones); y has ys's type, or with fp32 ys the one of `dtype`."""
    if ys.dim() != 2:
        raise ValueError("ys must be rows x h")
    rows, h = ys.shape
    topk = _topk(positions, None)
    tokens = positions.shape[0]
    device, dt = _device(ys, "ys", DTYPES)
    if weights is not None:
        _shape(weights, (tokens, topk), "weights")
    if y is None:
        y = _new(ys, (tokens, h), ys.dtype if dtype is None else dtype, stream)
    else:
        _shape(y, (tokens, h), "y")
    if y.dtype not in DTYPES or (y.dtype != ys.dtype and ys.dtype != torch.float32):
        raise TypeError("y must be %s, got %s" % (ys.dtype, y.dtype))
    _call("exl3_moe_combine", device, stream, _arg(ys, ys.dtype, "ys", device), dt,
          _arg(positions, torch.int32, "positions", device),
          None if weights is None else _arg(weights, torch.float32, "weights", device), tokens, topk, h, rows,
          _arg(y, y.dtype, "y", device), DTYPES[y.dtype])
    return y


def exl3_moe_combine_grad(dy, ys, positions, weights=None, dys=None, dweights=None, stream=None):
    """Gradients of exl3_moe_combine: (dys, dweights).  Rows of dys that no
    position names are not written."""
    if dy.dim() != 2 or ys.dim() != 2 or dy.shape[1] != ys.shape[1]:
        raise ValueError("dy must be tokens x h and ys rows x h")
    tokens, h = dy.shape
    rows = ys.shape[0]
    topk = _topk(positions, tokens)
    device, dt = _device(dy, "dy", DTYPES)
    if weights is not None:
        _shape(weights, (tokens, topk), "weights")
    if dys is None:
        dys = _new(dy, (rows, h), dy.dtype, stream)
    else:
        _shape(dys, (rows, h), "dys")
    if dweights is None:
        dweights = _new(dy, (tokens, topk), torch.float32, stream)
    else:
        _shape(dweights, (tokens, topk), "dweights")
    _call("exl3_moe_combine_grad", device, stream, _arg(dy, dy.dtype, "dy", device),
          _arg(ys, dy.dtype, "ys", device), dt, _arg(positions, torch.int32, "positions", device),
          None if weights is None else _arg(weights, torch.float32, "weights", device), tokens, topk, h, rows,
          _arg(dys, dy.dtype, "dys", device), _arg(dweights, torch.float32, "dweights", device))
    return dys, dweights


def exl3_workspace_status(workspace, clear=False, stream=None):
    """Status word of a gemv/gemm workspace (synchronises the stream)."""
    return int(load().exl3_workspace_status(_dev(workspace, torch.uint8, "workspace"), workspace.numel(),
                                            1 if clear else 0, _stream(stream)))


def exl3_set_launch_flags(flags):
    """EXL3_LAUNCH_PDL: programmatic dependent launch (weights must be immutable)."""
    load().exl3_set_launch_flags(int(flags))


def exl3_launch_flags():
    return int(load().exl3_launch_flags())


def exl3_debug_set_wait_limit_ns(ns):
    load().exl3_debug_set_wait_limit_ns(int(ns))


def exl3_debug_wait_limit_ns():
    return int(load().exl3_debug_wait_limit_ns())
