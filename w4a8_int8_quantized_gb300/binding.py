"""Thin Python binding of libw8a8 (ctypes): argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch
tensors that already live on the current CUDA device, checks their dtype and
contiguity, passes raw pointers, sizes and the current stream to the library,
and raises ``W8A8Error`` on a nonzero status.  All arithmetic runs in the
library's kernels; there is no fallback of any kind: if the library is not
built, or the device is not a compute-capability 10.3 GPU, the call fails.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libw8a8.so")

_lock = threading.Lock()
_lib = None

STATUS = {0: "ok", 1: "invalid argument", 2: "misaligned pointer or K",
          3: "unsupported device", 4: "CUDA error", 5: "device-side wait timed out",
          6: "workspace too small or misaligned",
          7: "slot, page, length or query offset out of range"}

# every symbol that include/w8a8.h declares
EXPORTS = ("w8a8_is_available", "w8a8_status_string", "w8a8_check_status",
           "quantize_weight_int8", "pack_weight_int4", "quantize_act_per_token",
           "w8a8_gemm", "w8a8_mv", "w4a8_gemm", "quantize_act_per_token_h", "w8a8_gemm_h",
           "w8a8_linear_workspace_bytes", "linear", "linear_noalloc", "w8a8_gemm_i32",
           "w8a8_test_set_fault", "weight_only_gemm", "kv_cache_write", "kv_cache_read",
           "kv_cache_attention_workspace_bytes", "kv_cache_attention")


class W8A8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


def load(path: str | None = None):
    """Load libw8a8.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libw8a8 is not built ({p} missing): run "
                               "w4a8_int8_quantized_gb300.build.build() first")
        lib = ctypes.CDLL(p)
        P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
        sig = {
            "w8a8_is_available": ([], I),
            "w8a8_status_string": ([I], ctypes.c_char_p),
            "w8a8_check_status": ([P], I),
            "quantize_weight_int8": ([P, I, I, I, P, P, P], I),
            "pack_weight_int4": ([P, I, I, P, P, P], I),
            "quantize_act_per_token": ([P, I, I, I, P, P, P], I),
            "w8a8_gemm": ([P, P, P, P, I, I, I, I, P, P], I),
            "w8a8_mv": ([P, P, P, P, I, I, I, I, P, P], I),
            "w4a8_gemm": ([P, P, P, P, I, I, I, P, P], I),
            "quantize_act_per_token_h": ([P, I, I, I, P, P, P], I),
            "w8a8_gemm_h": ([P, P, P, P, I, I, I, I, I, P, P], I),
            "w8a8_linear_workspace_bytes": ([I, I, I], Z),
            "linear": ([P, P, P, I, I, I, I, I, P, Z, P, P], I),
            "linear_noalloc": ([P, P, P, I, I, I, I, I, P, P], I),
            "w8a8_gemm_i32": ([P, P, I, I, I, I, I, P, P], I),
            "w8a8_test_set_fault": ([ctypes.c_longlong, I], I),
            "weight_only_gemm": ([P, P, P, I, I, I, I, I, P, P], I),
            "kv_cache_write": ([P, L, L, P, L, L, P, I, P, P], I),
            "kv_cache_read": ([P, I, P, P, P, P], I),
            "kv_cache_attention_workspace_bytes": ([I, I, I, I, I, P], Z),
            "kv_cache_attention": ([P, L, L, I, I, P, I, I, P, I, P, P, ctypes.c_float, I, I, P,
                                    Z, P, P, P], I),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check(status: int, what: str):
    if status != 0:
        raise W8A8Error(status, what)


def _groups(K: int, group_size: int) -> int:
    return 1 if group_size == 0 else K // group_size


def w8a8_is_available() -> bool:
    return bool(load().w8a8_is_available())


def w8a8_status_string(status: int) -> str:
    return load().w8a8_status_string(int(status)).decode()


def w8a8_check_status() -> int:
    return load().w8a8_check_status(_stream())


def quantize_weight_int8(W: torch.Tensor, group_size: int = 0, Wq=None, scale_w=None):
    """fp16 W [N, K] -> (int8 Wq [N, K], fp32 scale_w [N, G])."""
    _need(W, torch.float16, "W")
    N, K = W.shape
    G = _groups(K, group_size)
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device) if Wq is None else Wq
    scale_w = (torch.empty((N, G), dtype=torch.float32, device=W.device)
               if scale_w is None else scale_w)
    _need(Wq, torch.int8, "Wq", (N, K))
    _need(scale_w, torch.float32, "scale_w", (N, G))
    _check(load().quantize_weight_int8(_ptr(W), N, K, group_size, _ptr(Wq), _ptr(scale_w),
                                       _stream()), "quantize_weight_int8")
    return Wq, scale_w


def pack_weight_int4(W: torch.Tensor, Wp=None, scale_w=None):
    """fp16 W [N, K] -> (uint8 Wp [N, K/2], fp32 scale_w [N, 1])."""
    _need(W, torch.float16, "W")
    N, K = W.shape
    Wp = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device) if Wp is None else Wp
    scale_w = (torch.empty((N, 1), dtype=torch.float32, device=W.device)
               if scale_w is None else scale_w)
    _need(Wp, torch.uint8, "Wp", (N, K // 2))
    _need(scale_w, torch.float32, "scale_w", (N, 1))
    _check(load().pack_weight_int4(_ptr(W), N, K, _ptr(Wp), _ptr(scale_w), _stream()),
           "pack_weight_int4")
    return Wp, scale_w


def quantize_act_per_token(x: torch.Tensor, group_size: int = 0, xq=None, scale_a=None):
    """fp16 x [M, K] -> (int8 xq [M, K], fp32 scale_a [M, G])."""
    _need(x, torch.float16, "x")
    M, K = x.shape
    G = _groups(K, group_size)
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device) if xq is None else xq
    scale_a = (torch.empty((M, G), dtype=torch.float32, device=x.device)
               if scale_a is None else scale_a)
    _need(xq, torch.int8, "xq", (M, K))
    _need(scale_a, torch.float32, "scale_a", (M, G))
    _check(load().quantize_act_per_token(_ptr(x), M, K, group_size, _ptr(xq), _ptr(scale_a),
                                         _stream()), "quantize_act_per_token")
    return xq, scale_a


def _gemm_args(xq, scale_a, Wq, scale_w, group_size, wdtype, kdiv):
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    G = _groups(K, group_size)
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] * kdiv != K:
        raise ValueError("Wq inner dimension does not match K")
    _need(scale_a, torch.float32, "scale_a", (M, G))
    _need(scale_w, torch.float32, "scale_w", (N, G))
    return M, N, K


def w8a8_gemm(xq, scale_a, Wq, scale_w, group_size: int = 0, y=None):
    """int8 xq [M, K] x int8 Wq [N, K]^T with fused dequant -> fp16 y [M, N]."""
    M, N, K = _gemm_args(xq, scale_a, Wq, scale_w, group_size, torch.int8, 1)
    y = torch.empty((M, N), dtype=torch.float16, device=xq.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().w8a8_gemm(_ptr(xq), _ptr(scale_a), _ptr(Wq), _ptr(scale_w), M, N, K,
                            group_size, _ptr(y), _stream()), "w8a8_gemm")
    return y


def w8a8_mv(xq, scale_a, Wq, scale_w, group_size: int = 0, y=None):
    """Decode matrix-vector product; xq must have one row."""
    M, N, K = _gemm_args(xq, scale_a, Wq, scale_w, group_size, torch.int8, 1)
    y = torch.empty((M, N), dtype=torch.float16, device=xq.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().w8a8_mv(_ptr(xq), _ptr(scale_a), _ptr(Wq), _ptr(scale_w), M, N, K,
                          group_size, _ptr(y), _stream()), "w8a8_mv")
    return y


def w4a8_gemm(xq, scale_a, Wp, scale_w, y=None):
    """int8 xq [M, K] x packed int4 Wp [N, K/2]^T with fused dequant."""
    M, N, K = _gemm_args(xq, scale_a, Wp, scale_w, 0, torch.uint8, 2)
    y = torch.empty((M, N), dtype=torch.float16, device=xq.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().w4a8_gemm(_ptr(xq), _ptr(scale_a), _ptr(Wp), _ptr(scale_w), M, N, K,
                            _ptr(y), _stream()), "w4a8_gemm")
    return y


def quantize_act_per_token_h(x: torch.Tensor, group_size: int = 0, xq_h=None, scale_a=None):
    """fp16 x [M, K] -> (INT8 codes as fp16 xq_h [M, K], fp32 scale_a [M, G])."""
    _need(x, torch.float16, "x")
    M, K = x.shape
    G = _groups(K, group_size)
    xq_h = torch.empty((M, K), dtype=torch.float16, device=x.device) if xq_h is None else xq_h
    scale_a = (torch.empty((M, G), dtype=torch.float32, device=x.device)
               if scale_a is None else scale_a)
    _need(xq_h, torch.float16, "xq_h", (M, K))
    _need(scale_a, torch.float32, "scale_a", (M, G))
    _check(load().quantize_act_per_token_h(_ptr(x), M, K, group_size, _ptr(xq_h),
                                           _ptr(scale_a), _stream()), "quantize_act_per_token_h")
    return xq_h, scale_a


def w8a8_gemm_h(xq_h, scale_a, Wq, scale_w, group_size: int = 0, wbits: int = 8, y=None):
    """GEMM with the activation codes given as fp16 values (wbits 8: int8 Wq
    [N, K]; wbits 4: packed Wq [N, K/2])."""
    _need(xq_h, torch.float16, "xq_h")
    M, K = xq_h.shape
    G = _groups(K, group_size)
    wdtype = torch.int8 if wbits == 8 else torch.uint8
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] * (1 if wbits == 8 else 2) != K:
        raise ValueError("Wq inner dimension does not match K")
    _need(scale_a, torch.float32, "scale_a", (M, G))
    _need(scale_w, torch.float32, "scale_w", (N, G))
    y = torch.empty((M, N), dtype=torch.float16, device=xq_h.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().w8a8_gemm_h(_ptr(xq_h), _ptr(scale_a), _ptr(Wq), _ptr(scale_w), M, N, K,
                              group_size, wbits, _ptr(y), _stream()), "w8a8_gemm_h")
    return y


def w8a8_linear_workspace_bytes(M: int, K: int, group_size: int = 0) -> int:
    return int(load().w8a8_linear_workspace_bytes(M, K, group_size))


def linear(x, Wq, scale_w, group_size: int = 0, wbits: int = 8, workspace=None, y=None):
    """The whole layer: per-token quantization of x, then GEMM (M > 1) or
    matrix-vector (M == 1) with the fused dequant.  Wq is int8 [N, K]
    (wbits 8) or packed uint8 [N, K/2] (wbits 4)."""
    _need(x, torch.float16, "x")
    M, K = x.shape
    wdtype = torch.int8 if wbits == 8 else torch.uint8
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    _need(scale_w, torch.float32, "scale_w", (N, _groups(K, group_size)))
    need = w8a8_linear_workspace_bytes(M, K, group_size)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _need(workspace, torch.uint8, "workspace")
    y = torch.empty((M, N), dtype=torch.float16, device=x.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().linear(_ptr(x), _ptr(Wq), _ptr(scale_w), M, N, K, group_size, wbits,
                         _ptr(workspace), workspace.numel(), _ptr(y), _stream()), "linear")
    return y


def linear_noalloc(x, Wq, scale_w, group_size: int = 0, wbits: int = 8, y=None):
    """linear() without a workspace: the library's fixed 8 MiB device array
    serves as the workspace, so the C call allocates nothing (the output is
    allocated here if not given).  Problems that do not fit raise W8A8Error
    (status 6).  Calls on streams that overlap on the GPU race on the array."""
    _need(x, torch.float16, "x")
    M, K = x.shape
    wdtype = torch.int8 if wbits == 8 else torch.uint8
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    _need(scale_w, torch.float32, "scale_w", (N, _groups(K, group_size)))
    y = torch.empty((M, N), dtype=torch.float16, device=x.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().linear_noalloc(_ptr(x), _ptr(Wq), _ptr(scale_w), M, N, K, group_size, wbits,
                                 _ptr(y), _stream()), "linear_noalloc")
    return y


def weight_only_gemm(x, Wq, scale_w, group_size: int = 0, wbits: int = 8, y=None):
    """Weight-only product (W8A16 / W4A16): fp16 x [M, K] times the dequantized
    weights (int8 Wq [N, K], or packed uint8 [N, K/2] with wbits 4)."""
    _need(x, torch.float16, "x")
    M, K = x.shape
    wdtype = torch.int8 if wbits == 8 else torch.uint8
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    if Wq.shape[1] * (1 if wbits == 8 else 2) != K:
        raise ValueError("Wq inner dimension does not match K")
    _need(scale_w, torch.float32, "scale_w", (N, _groups(K, group_size)))
    y = torch.empty((M, N), dtype=torch.float16, device=x.device) if y is None else y
    _need(y, torch.float16, "y", (M, N))
    _check(load().weight_only_gemm(_ptr(x), _ptr(Wq), _ptr(scale_w), M, N, K, group_size, wbits,
                                   _ptr(y), _stream()), "weight_only_gemm")
    return y


def w8a8_gemm_i32(xq, Wq, group_size: int = 0, wbits: int = 8, acc=None):
    """Exact INT32 (per-group) sums acc [M, N, G] of the tensor-core contraction."""
    _need(xq, torch.int8, "xq")
    M, K = xq.shape
    wdtype = torch.int8 if wbits == 8 else torch.uint8
    _need(Wq, wdtype, "Wq")
    N = Wq.shape[0]
    G = _groups(K, group_size)
    acc = torch.empty((M, N, G), dtype=torch.int32, device=xq.device) if acc is None else acc
    _need(acc, torch.int32, "acc", (M, N, G))
    _check(load().w8a8_gemm_i32(_ptr(xq), _ptr(Wq), M, N, K, group_size, wbits, _ptr(acc),
                                _stream()), "w8a8_gemm_i32")
    return acc


def w8a8_test_set_fault(wait_limit_cycles: int = 0, skip_first_copy: bool = False) -> None:
    """Test hook: the bounded-wait limit (cycles, 0 = default) of the GEMM and of
    the cache attention, and whether each CTA's first copy is left unissued, for
    the launches that follow."""
    _check(load().w8a8_test_set_fault(int(wait_limit_cycles), int(bool(skip_first_copy))),
           "w8a8_test_set_fault")


# ---- quantized key/value cache ---------------------------------------------

class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_longlong), ("kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("bits", ctypes.c_int)]


class KVCache:
    """Handle of one layer's paged cache (w8a8_kv_cache) over the caller's tensors.

    ``k_codes``, ``v_codes``: int8 [num_pages, kv_heads, page_size, D] (8 bits)
    or packed uint8 [num_pages, kv_heads, page_size, D / 2] (4 bits);
    ``k_scale``, ``v_scale``: fp32 [num_pages, kv_heads, page_size].  All
    contiguous, on one CUDA device.  The checks are made here, once; the calls
    take the handle."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype not in (torch.int8, torch.uint8):
                raise TypeError(f"{name} must be torch.int8 (8 bits) or torch.uint8 (4 bits), "
                                f"got {t.dtype}")
            if t.dim() != 4:
                raise ValueError(f"{name} must have 4 dimensions")
            _need(t, k_codes.dtype, name, k_codes.shape)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t, torch.float32, name, k_codes.shape[:3])
        if len({t.device for t in (k_codes, v_codes, k_scale, v_scale)}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.bits = 8 if k_codes.dtype == torch.int8 else 4
        self.num_pages, self.kv_heads, self.page_size, d = k_codes.shape
        self.head_dim = d * 8 // self.bits
        if self.head_dim not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {self.head_dim}")
        if not 16 <= self.page_size <= 1024 or self.page_size & (self.page_size - 1):
            raise ValueError(f"page_size must be a power of two from 16 to 1024, got {self.page_size}")
        self.device = k_codes.device
        self.index = self.device.index
        self._struct = _CacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                    v_scale.data_ptr(), self.num_pages, self.kv_heads,
                                    self.page_size, self.head_dim, self.bits)
        self._at = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, bits: int = 4,
              device="cuda"):
        """A cache over new, uninitialised tensors."""
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8, got {bits}")
        shape = (num_pages, kv_heads, page_size)
        codes = [torch.empty((*shape, head_dim * bits // 8), device=device,
                             dtype=torch.int8 if bits == 8 else torch.uint8) for _ in range(2)]
        return cls(*codes, *(torch.empty(shape, dtype=torch.float32, device=device)
                             for _ in range(2)))


# A decoding step's kernels take a few microseconds, so these calls keep their
# checks short: plain comparisons first, the words only when one fails.

_HALF, _INT, _LONG, _FLOAT = torch.float16, torch.int32, torch.int64, torch.float32
# the current stream's handle and the current device, without building objects
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(cache: KVCache, t, dtype, name: str, shape):
    """Says what is wrong with a tensor that failed its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's device {cache.device}, got {t.device}")
    if len(t.shape) != len(shape) or any(a is not None and a != b for a, b in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)} (None: any), got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _vector(cache: KVCache, t: torch.Tensor, dtype, name: str, shape):
    """t is a contiguous tensor of this type and shape on the cache's device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == cache.device and t.is_contiguous()):
        _refuse(cache, t, dtype, name, shape)


def _rows(cache: KVCache, t: torch.Tensor, name: str, heads: int | None, T: int | None):
    """Token and head strides of t, an fp16 [tokens, heads, D] with contiguous rows
    (heads, T: None for any)."""
    D = cache.head_dim
    if not (isinstance(t, torch.Tensor) and t.dtype is _HALF and t.device == cache.device
            and t.dim() == 3):
        _refuse(cache, t, _HALF, name, (T, heads, D))
    n, h, d = t.shape
    if d != D or (heads is not None and h != heads) or (T is not None and n != T):
        _refuse(cache, t, _HALF, name, (T, heads, D))
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name} must be contiguous along the head dimension")
    # the stride of a dimension of one element says nothing
    return (ts if n > 1 else 0), (hs if h > 1 else 0), n, h


def _stream_of(cache: KVCache) -> int:
    """The current stream of the cache's device, which has to be the current device."""
    index = cache.index
    if _current_device() != index:
        raise ValueError(f"the cache is on {cache.device}, which is not the current device")
    return _raw_stream(index)


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: KVCache) -> None:
    """Quantizes fp16 k, v [T, kv_heads, D] (any token and head strides that are
    multiples of 8) into the cache's slots, int64 [T] (page * page_size +
    offset; negative: not stored)."""
    kts, khs, T, heads = _rows(cache, k, "k", cache.kv_heads, None)
    vts, vhs, _, _ = _rows(cache, v, "v", heads, T)
    _vector(cache, slots, _LONG, "slots", (T,))
    status = (_lib or load()).kv_cache_write(k.data_ptr(), kts, khs, v.data_ptr(), vts, vhs,
                                             slots.data_ptr(), T, cache._at, _stream_of(cache))
    if status:
        _check(status, "kv_cache_write")


def kv_cache_read(slots: torch.Tensor, cache: KVCache, k=None, v=None):
    """The dequantized fp16 (k, v) [T, kv_heads, D] of the slots, int64 [T]
    (negative: zeros)."""
    T = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else None
    _vector(cache, slots, _LONG, "slots", (T,))
    shape = (T, cache.kv_heads, cache.head_dim)
    device = cache.device
    if k is None:
        k = torch.empty(shape, dtype=_HALF, device=device)
    else:
        _vector(cache, k, _HALF, "k", shape)
    if v is None:
        v = torch.empty(shape, dtype=_HALF, device=device)
    else:
        _vector(cache, v, _HALF, "v", shape)
    status = (_lib or load()).kv_cache_read(slots.data_ptr(), T, cache._at, k.data_ptr(),
                                            v.data_ptr(), _stream_of(cache))
    if status:
        _check(status, "kv_cache_read")
    return k, v


def kv_cache_attention_workspace_bytes(T: int, q_heads: int, cache: KVCache,
                                       block_table: torch.Tensor, max_q: int | None = None) -> int:
    """Workspace of kv_cache_attention() for T queries of q_heads heads."""
    B, width = block_table.shape
    return int(load().kv_cache_attention_workspace_bytes(
        T, q_heads, B, max(T, 1) if max_q is None else max_q, width, cache._at))


def kv_cache_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, q_offsets=None, max_q: int | None = None,
                       softmax_scale: float | None = None, causal: bool = True, window: int = 0,
                       return_lse: bool = False, workspace=None, out=None, lse=None):
    """Attention of fp16 q [T, q_heads, D] over the cached tokens.

    block_table int32 [B, pages], seq_lens int32 [B]; q_offsets int32 [B + 1]
    (None: one query per sequence); max_q: upper bound of one sequence's
    queries (default T).  causal, window: which keys a query sees.  Returns out
    fp16 [T, q_heads, D], or (out, lse fp32 [T, q_heads]) with return_lse.  Rows
    that see no key, and rows of no sequence, hold 0 (lse -inf)."""
    ts, hs, T, heads = _rows(cache, q, "q", None, None)
    device = cache.device
    if not (isinstance(block_table, torch.Tensor) and block_table.dtype is _INT
            and block_table.dim() == 2 and block_table.device == device
            and block_table.is_contiguous()):
        _refuse(cache, block_table, _INT, "block_table", (None, None))
    B, width = block_table.shape
    _vector(cache, seq_lens, _INT, "seq_lens", (B,))
    if q_offsets is None:
        offsets_at, max_q = 0, 1
    else:
        _vector(cache, q_offsets, _INT, "q_offsets", (B + 1,))
        offsets_at = q_offsets.data_ptr()
        if max_q is None:
            max_q = T or 1
    lib = _lib or load()
    if workspace is None:
        need = lib.kv_cache_attention_workspace_bytes(T, heads, B, max_q, width, cache._at)
        workspace = torch.empty(need or 1, dtype=torch.uint8, device=device)
    elif not (workspace.dtype is torch.uint8 and workspace.device == device
              and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous torch.uint8 tensor on the cache's device")
    D = cache.head_dim
    if out is None:
        out = torch.empty((T, heads, D), dtype=_HALF, device=device)
    else:
        _vector(cache, out, _HALF, "out", (T, heads, D))
    lse_at = 0
    if return_lse:
        if lse is None:
            lse = torch.empty((T, heads), dtype=_FLOAT, device=device)
        else:
            _vector(cache, lse, _FLOAT, "lse", (T, heads))
        lse_at = lse.data_ptr()
    status = lib.kv_cache_attention(
        q.data_ptr(), ts, hs, T, heads, offsets_at, B, max_q, block_table.data_ptr(), width,
        seq_lens.data_ptr(), cache._at, D ** -0.5 if softmax_scale is None else softmax_scale,
        1 if causal else 0, window, workspace.data_ptr(), workspace.numel(), out.data_ptr(),
        lse_at, _stream_of(cache))
    if status:
        _check(status, "kv_cache_attention")
    return (out, lse) if return_lse else out
