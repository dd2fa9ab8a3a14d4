"""Python binding of libkq (argument marshalling only).

Every computation runs in the CUDA kernels of ``libkq.so``; this module only
passes device pointers, sizes and the current torch stream through the C
ABI declared in ``include/kq.h``.  There is no CPU fallback: if the library
is missing or fails to load, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import numpy as np

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkq.so")

Q4_K = 1
Q6_K = 2
Q5_K = 3
Q2_K = 4
Q3_K = 5
Q8_0 = 6
FORMATS = {"q4_k": Q4_K, "q6_k": Q6_K, "q5_k": Q5_K, "q2_k": Q2_K, "q3_k": Q3_K, "q8_0": Q8_0}
BLOCK_BYTES = {Q4_K: 144, Q6_K: 210, Q5_K: 176, Q2_K: 84, Q3_K: 110, Q8_0: 272}  # per 256 weights

OK = 0
STATUS = {0: "KQ_OK", 1: "KQ_ERR_INVALID_ARG", 2: "KQ_ERR_UNSUPPORTED", 3: "KQ_ERR_NOT_PINNED",
          4: "KQ_ERR_OOM", 5: "KQ_ERR_CUDA", 6: "KQ_ERR_TIMEOUT", 7: "KQ_ERR_DEVICE_CHECK",
          8: "KQ_ERR_INJECTED"}

_lib = None


class KQError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({detail})")
        self.status = status


class Prologue(ctypes.Structure):
    """kq_prologue: the activation prologue of kq_gemv_fused."""
    _fields_ = [("kind", ctypes.c_int), ("gamma", ctypes.c_void_p), ("eps", ctypes.c_float)]


PROLOGUE = {"none": 0, "rmsnorm": 1, "swiglu": 2}


class Step(ctypes.Structure):
    """kq_step: one GEMV of kq_gemv_steps."""
    _fields_ = [("W", ctypes.c_void_p), ("fmt", ctypes.c_int), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("pro", Prologue), ("after", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """Load libkq.so (built in-tree by ``dequant_quant_gemv_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkq.so not built at {LIB_PATH}; run python -m dequant_quant_gemv_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.kq_version.restype = i32
        L.kq_status_str.restype = ctypes.c_char_p
        L.kq_status_str.argtypes = [i32]
        L.kq_last_error.restype = ctypes.c_char_p
        L.kq_device_fault.restype = i32
        L.kq_device_fault.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.kq_block_bytes.restype = sz
        L.kq_block_bytes.argtypes = [i32]
        L.kq_row_bytes.restype = sz
        L.kq_row_bytes.argtypes = [i32, i64]
        L.kq_gemv.restype = i32
        L.kq_gemv.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        L.kq_gemv_multi.restype = i32
        L.kq_gemv_multi.argtypes = [vp, i32, i64, i64, vp, i64, i32, vp, i64, vp]
        L.kq_moe_gemv.restype = i32
        L.kq_moe_gemv.argtypes = [vp, i32, i32, i64, i64, sz, vp, i32, vp, i64, vp, vp, vp]
        L.kq_unpack.restype = i32
        L.kq_unpack.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, vp]
        L.kq_unpack_fields.restype = i32
        L.kq_unpack_fields.argtypes = [vp, i32, i64, vp, vp, vp, vp]
        L.kq_gemv_fused.restype = i32
        L.kq_gemv_fused.argtypes = [vp, i32, i64, i64, vp, i64, i32, ctypes.POINTER(Prologue), vp, i64, vp]
        L.kq_gemv_steps.restype = i32
        L.kq_gemv_steps.argtypes = [ctypes.POINTER(Step), i32, vp]
        _lib = L
    return _lib


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _check(status: int, what: str) -> None:
    if status != OK:
        raise KQError(status, what, lib().kq_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def row_bytes(fmt, K: int) -> int:
    return int(lib().kq_row_bytes(_fmt(fmt), K))


def gemv(W: torch.Tensor, fmt, N: int, K: int, x: torch.Tensor, y: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """y = W x.  W: uint8 device tensor of N*row_bytes; x: K float32."""
    if y is None:
        y = torch.empty(N, dtype=torch.float32, device=x.device)
    _check(lib().kq_gemv(_dev(W, "W"), _fmt(fmt), N, K, _dev(x, "x", torch.float32),
                         _dev(y, "y", torch.float32), _stream(stream)), "kq_gemv")
    return y


def gemv_multi(W: torch.Tensor, fmt, N: int, K: int, X: torch.Tensor, Y: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Y[c] = W X[c] for the k rows of X (shape (k, K), rows may be strided)."""
    k = X.shape[0]
    if Y is None:
        Y = torch.empty((k, N), dtype=torch.float32, device=X.device)
    _check(lib().kq_gemv_multi(_dev(W, "W"), _fmt(fmt), N, K, _dev(X, "X", torch.float32), X.stride(0), k,
                               _dev(Y, "Y", torch.float32), Y.stride(0), _stream(stream)), "kq_gemv_multi")
    return Y


def gemv_fused(W: torch.Tensor, fmt, N: int, K: int, X: torch.Tensor, kind: str = "none",
               gamma: torch.Tensor | None = None, eps: float = 1e-5, Y: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Y[c] = W P(X[c]) for the k rows of X: P = "none", "rmsnorm" (with gamma,
    eps; rows of K) or "swiglu" (rows of 2K: [gate; up])."""
    if X.dim() == 1:
        X = X[None, :]
    k = X.shape[0]
    if Y is None:
        Y = torch.empty((k, N), dtype=torch.float32, device=X.device)
    pro = Prologue(PROLOGUE[kind], _dev(gamma, "gamma", torch.float32) if gamma is not None else None, eps)
    _check(lib().kq_gemv_fused(_dev(W, "W"), _fmt(fmt), N, K, _dev(X, "X", torch.float32), X.stride(0), k,
                               ctypes.byref(pro), _dev(Y, "Y", torch.float32), Y.stride(0), _stream(stream)),
           "kq_gemv_fused")
    return Y


def make_step(W: torch.Tensor, fmt, N: int, K: int, x: torch.Tensor, y: torch.Tensor, kind: str = "none",
              gamma: torch.Tensor | None = None, eps: float = 1e-5, after: bool = False) -> Step:
    """A kq_step for gemv_steps: y = W P(x), one column (x of K floats, 2K for
    "swiglu"); `after`: x is written by an earlier step of the same call."""
    pro = Prologue(PROLOGUE[kind], _dev(gamma, "gamma", torch.float32) if gamma is not None else None, eps)
    return Step(_dev(W, "W"), _fmt(fmt), N, K, _dev(x, "x", torch.float32), _dev(y, "y", torch.float32), pro,
                1 if after else 0)


def gemv_steps(steps, stream=None) -> None:
    """kq_gemv_steps over a list of Step (see make_step), in order."""
    arr = (Step * max(1, len(steps)))(*steps)
    _check(lib().kq_gemv_steps(arr, len(steps), _stream(stream)), "kq_gemv_steps")


def _splitk_sigs(L):
    if not getattr(L, "_splitk_ready", False):
        L.kq_splitk_workspace_bytes.restype = ctypes.c_size_t
        L.kq_splitk_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
        L.kq_gemv_splitk.restype = ctypes.c_int
        L.kq_gemv_splitk.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_void_p]
        L._splitk_ready = True
    return L


def splitk_workspace_bytes(fmt, N: int, K: int, k: int = 1) -> int:
    return int(_splitk_sigs(lib()).kq_splitk_workspace_bytes(_fmt(fmt), N, K, k))


def gemv_splitk(W: torch.Tensor, fmt, N: int, K: int, X: torch.Tensor, Y: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kq_gemv_splitk: X is (K,) or (k, K); the workspace is allocated here
    (torch) when not given."""
    L = _splitk_sigs(lib())
    X2 = X.view(1, -1) if X.dim() == 1 else X
    k = X2.shape[0]
    if Y is None:
        Y = torch.empty((k, N), dtype=torch.float32, device=X.device)
    Y2 = Y.view(1, -1) if Y.dim() == 1 else Y
    need = splitk_workspace_bytes(fmt, N, K, k)
    if workspace is None:
        workspace = torch.empty(max(1, (need + 3) // 4), dtype=torch.float32, device=X.device)
    _check(L.kq_gemv_splitk(_dev(W, "W"), _fmt(fmt), N, K, _dev(X2, "X", torch.float32), X2.stride(0), k,
                            _dev(Y2, "Y", torch.float32), Y2.stride(0), _dev(workspace, "workspace"),
                            workspace.numel() * workspace.element_size(), _stream(stream)), "kq_gemv_splitk")
    return Y


def gemv_splitk_noalloc(W: torch.Tensor, fmt, N: int, K: int, X: torch.Tensor, Y: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """kq_gemv_splitk_noalloc: split-K GEMV with its partial sums in the
    library's built-in scratch, for callers that cannot allocate device
    memory.  X is (K,) or (k, K); Y must be given (this call allocates
    nothing)."""
    L = lib()
    if not getattr(L, "_noalloc_ready", False):
        L.kq_gemv_splitk_noalloc.restype = ctypes.c_int
        L.kq_gemv_splitk_noalloc.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_void_p]
        L._noalloc_ready = True
    X2 = X.view(1, -1) if X.dim() == 1 else X
    Y2 = Y.view(1, -1) if Y.dim() == 1 else Y
    _check(L.kq_gemv_splitk_noalloc(_dev(W, "W"), _fmt(fmt), N, K, _dev(X2, "X", torch.float32), X2.stride(0),
                                    X2.shape[0], _dev(Y2, "Y", torch.float32), Y2.stride(0), _stream(stream)),
           "kq_gemv_splitk_noalloc")
    return Y


def moe_gemv(W_experts: torch.Tensor, fmt, E: int, N: int, K: int, ids: torch.Tensor, x: torch.Tensor,
             y: torch.Tensor | None = None, status: torch.Tensor | None = None, expert_stride: int | None = None,
             stream=None) -> torch.Tensor:
    """y[i] = W_{ids[i]} x_i; x is (K,) shared or (n_ids, K) per id."""
    n = ids.numel()
    if expert_stride is None:
        expert_stride = N * row_bytes(fmt, K)
    if y is None:
        y = torch.empty((n, N), dtype=torch.float32, device=x.device)
    x_stride = 0 if x.dim() == 1 else x.stride(0)
    _check(lib().kq_moe_gemv(_dev(W_experts, "W_experts"), _fmt(fmt), E, N, K, expert_stride,
                             _dev(ids, "ids", torch.int32), n, _dev(x, "x", torch.float32), x_stride,
                             _dev(y, "y", torch.float32), None if status is None else _dev(status, "status"),
                             _stream(stream)), "kq_moe_gemv")
    return y


def unpack(W: torch.Tensor, fmt, n_blocks: int, stream=None):
    """(q, sc, d) integer fields as decoded on the GPU, packed form
    (kq_unpack_fields in kq.h)."""
    q = torch.empty(n_blocks * 256, dtype=torch.uint8, device=W.device)
    sc = torch.empty(n_blocks * 16, dtype=torch.uint8, device=W.device)
    d = torch.empty(n_blocks * 2, dtype=torch.float32, device=W.device)
    _check(lib().kq_unpack_fields(_dev(W, "W"), _fmt(fmt), n_blocks, q.data_ptr(), sc.data_ptr(), d.data_ptr(),
                                  _stream(stream)), "kq_unpack_fields")
    return q, sc, d


def unpack_split(W: torch.Tensor, fmt, n_blocks: int, stream=None):
    """(q, sc_or_s, m, d, dmin) as decoded on the GPU (kq_unpack in kq.h):
    q int8 (n_blocks*256), sc_or_s and m uint8 (n_blocks*16 each), d and
    dmin float32 (n_blocks each)."""
    q = torch.empty(n_blocks * 256, dtype=torch.int8, device=W.device)
    sc = torch.empty(n_blocks * 16, dtype=torch.uint8, device=W.device)
    m = torch.empty(n_blocks * 16, dtype=torch.uint8, device=W.device)
    d = torch.empty(n_blocks, dtype=torch.float32, device=W.device)
    dmin = torch.empty(n_blocks, dtype=torch.float32, device=W.device)
    _check(lib().kq_unpack(_dev(W, "W"), _fmt(fmt), n_blocks, q.data_ptr(), sc.data_ptr(), m.data_ptr(),
                           d.data_ptr(), dmin.data_ptr(), _stream(stream)), "kq_unpack")
    return q, sc, m, d, dmin


def read_probe(buf: torch.Tensor, mode: int, out: torch.Tensor, stream=None) -> None:
    """kq_read_probe: read `buf` once (mode 0 loads, mode 1 the bulk-copy
    ring of the GEMV kernels); XOR of the data into out (int32, 1 element)."""
    L = lib()
    L.kq_read_probe.restype = ctypes.c_int
    L.kq_read_probe.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    _check(L.kq_read_probe(_dev(buf, "buf"), buf.numel() * buf.element_size(), mode, _dev(out, "out"),
                           _stream(stream)), "kq_read_probe")


def inject(spec: str | None) -> None:
    """kq_inject: test hook ("hold@S" withholds one weight stage of the next
    single-column launch, "hold_attn@N" one chunk of keys of the next attention
    call of many rows, so that a bounded wait runs out)."""
    L = lib()
    L.kq_inject.restype = ctypes.c_int
    L.kq_inject.argtypes = [ctypes.c_char_p]
    _check(L.kq_inject(spec.encode() if spec else None), "kq_inject")


def device_fault() -> int:
    out = ctypes.c_int(0)
    _check(lib().kq_device_fault(ctypes.byref(out)), "kq_device_fault")
    return out.value


# ------------------------------------- between a layer's products
class KVCacheDesc(ctypes.Structure):
    """kq_kv_cache: a paged key-value cache of one layer."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int), ("n_kv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64)]


class Rotary(ctypes.Structure):
    """kq_rotary: how kq_kv_append rotates and normalises heads."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("adjacent", ctypes.c_int),
                ("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p), ("eps", ctypes.c_float)]


class Residual(ctypes.Structure):
    """kq_residual: one kq_residual_norm step."""
    _fields_ = [("n_terms", ctypes.c_int), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("ld_term", ctypes.c_int64), ("weights", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("post_gamma", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64),
                ("scale", ctypes.c_float), ("res", ctypes.c_void_p), ("ldres", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ldout", ctypes.c_int64), ("pre_gamma", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("eps", ctypes.c_float)]


_layer = None
_fast = None   # the compiled fast path (csrc/kq_calls.cpp)


class _NoFastPath:
    """Takes no call, so that each goes through ctypes to the same C ABI."""
    kv_plan = kv_append = kv_attn = residual_norm = staticmethod(lambda *a: None)


def _fast_path(L: ctypes.CDLL):
    from .build import calls_key
    try:
        from . import _calls
        if getattr(_calls, "key", None) != calls_key():
            raise ImportError("built against another torch or Python")
    except ImportError as e:
        warnings.warn(f"_calls.so cannot be used ({e}): the layer operators' calls take about 5 us longer on the host; "
                      "run python -m dequant_quant_gemv_b200.build", RuntimeWarning, stacklevel=4)
        return _NoFastPath
    _calls.use(*[ctypes.cast(f, ctypes.c_void_p).value
                 for f in (L.kq_kv_plan, L.kq_kv_append, L.kq_kv_attn, L.kq_residual_norm)])
    return _calls


def _layer_lib() -> ctypes.CDLL:
    global _layer, _fast
    if _layer is None:
        L = lib()
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.kq_kv_plan.restype = i32
        L.kq_kv_plan.argtypes = [i32, vp, vp, i32, vp, i64, i32, vp, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp]
        L.kq_kv_append.restype = i32
        L.kq_kv_append.argtypes = [i64, vp, i64, i32, vp, vp, vp, vp, vp, i64, vp, vp]
        L.kq_kv_attn_workspace_bytes.restype = sz
        L.kq_kv_attn_workspace_bytes.argtypes = [i32, i32, i32, vp]
        L.kq_kv_attn.restype = i32
        L.kq_kv_attn.argtypes = [i32, i64, i32, i32, vp, i64, vp, vp, vp, vp, i64, i32, ctypes.c_float, i32, vp, i64,
                                 vp, sz, vp, vp]
        L.kq_residual_norm.restype = i32
        L.kq_residual_norm.argtypes = [vp, i64, i64, vp]
        _fast = _fast_path(L)
        _layer = L
    return _layer


def _load():
    _layer_lib()
    return _fast


def _bad(dev: int, t: torch.Tensor, name: str, dtype, shape) -> None:
    """Raises for a tensor that a layer call cannot take."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous along its last dimension")


# The layer calls go through the compiled fast path where everything is plain
# (current stream and device, outputs given); what it does not take comes here,
# to be checked, refused with a message, or called.
def _vec(dev: int, t: torch.Tensor, name: str, dtype, n: int) -> int:
    """Address of a contiguous tensor of n elements of `dtype` on device `dev`."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _bad(dev, t, name, dtype, torch.Size((n,)))
    return t.data_ptr()


def _opt(dev: int, t: torch.Tensor | None, name: str, dtype, n: int) -> int | None:
    return None if t is None else _vec(dev, t, name, dtype, n)


def _mat(dev: int, t: torch.Tensor, name: str, dtype, rows: int, cols: int) -> tuple[int, int]:
    """(address, stride between rows) of a rows x cols tensor with contiguous rows."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, cols):
        _bad(dev, t, name, dtype, torch.Size((rows, cols)))
    if t.is_contiguous():
        return t.data_ptr(), cols
    if cols > 1 and t.stride(1) != 1:
        _bad(dev, t, name, dtype, t.shape)
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def _int(v: int, name: str) -> int:
    """A whole number that fits the C ABI's int (ctypes would cut it)."""
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name}={v} does not fit in 32 bits")
    return v


def _index(t: torch.Tensor, what: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} needs CUDA tensors")
    return dev


def _layer_call(fn, what: str, dev: int, stream, *args) -> None:
    """Runs fn(*args, stream) with device `dev` current, on `stream` or that device's current stream."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st:
        _check(st, what)


def _empty(shape, dtype, dev: int, stream, fill=torch.empty) -> torch.Tensor:
    """An output or scratch tensor on device `dev`, allocated on the stream that
    the call will run on (the allocator orders its blocks by stream)."""
    if stream is None:
        return fill(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=dev)
    with torch.cuda.stream(stream):
        return fill(shape, dtype=dtype, device=dev)


class KVCache:
    """A paged key-value cache of one layer over the caller's pools k and v:
    shape (n_pages, n_kv, page_size, head_dim), float16 or bfloat16, pages
    contiguous (their stride is free)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D tensors alike in shape, strides and type")
        kind = {torch.float16: 1, torch.bfloat16: 2}.get(k.dtype)
        if kind is None:
            raise TypeError(f"the cache must be float16 or bfloat16, got {k.dtype}")
        if not k.is_cuda or k.device != v.device:
            raise ValueError("k and v must be CUDA tensors of one device")
        n, h, ps, d = k.shape
        if k.numel() and not k[0].is_contiguous():
            raise ValueError("the pages of k and v must be contiguous")
        self.k, self.v = k, v
        self.n_kv, self.page_size, self.head_dim, self.device = h, ps, d, k.device
        self._dev = k.get_device()
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), kind, h, d, ps, n, k.stride(0) if n > 1 else h * ps * d)
        self._ref = ctypes.addressof(self.desc)


class KVPlan:
    """The arrays that kq_kv_plan writes, for R requests and T columns."""

    def __init__(self, R: int, T: int, device="cuda"):
        def e(n, dt=torch.int32):
            return torch.empty(n, dtype=dt, device=device)
        self.lens, self.q_start, self.n_left = e(R), e(R + 1), e(1)
        self.slots, self.pos = e(T, torch.int64), e(T)
        self._ptr = [t.data_ptr() for t in (self.lens, self.q_start, self.slots, self.pos, self.n_left)]
        self._dev, self._R, self._T = _index(self.n_left, "KVPlan"), R, T


def kv_plan(lens: torch.Tensor, add: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
            n_free: torch.Tensor, page_size: int, plan: KVPlan, status: torch.Tensor | None = None,
            stream=None) -> KVPlan:
    """kq_kv_plan: pages, slots and positions of the step that adds add[r]
    tokens to request r (int32 tensors); fills in table (R, max_pages) and
    plan."""
    if stream is None:
        st = (_fast or _load()).kv_plan(lens, add, table, free_pages, n_free, page_size, plan.lens, plan.q_start, plan.slots,
                                        plan.pos, plan.n_left, status)
        if st is not None:
            if st:
                _check(st, "kq_kv_plan")
            return plan
    i32 = torch.int32
    dev, R = _index(lens, "kv_plan"), lens.numel()
    if plan._dev != dev or plan._R != R:
        raise ValueError("the plan is for other requests or another device")
    width, n_stack, p = table.shape[-1], free_pages.numel(), plan._ptr
    tab, ld = _mat(dev, table, "table", i32, R, width)
    _layer_call(_layer_lib().kq_kv_plan, "kq_kv_plan", dev, stream, R, _vec(dev, lens, "lens", i32, R),
                _vec(dev, add, "add", i32, R), _int(page_size, "page_size"), tab, ld, width,
                _vec(dev, free_pages, "free_pages", i32, n_stack), n_stack, _vec(dev, n_free, "n_free", i32, 1), plan._T,
                p[0], p[1], p[2], p[3], p[4],
                _opt(dev, status, "status", i32, 1))
    return plan


_PAIRING = {"half": 0, "adjacent": 1}


def kv_append(qkv: torch.Tensor, n_q: int, cache: KVCache, slots: torch.Tensor, pos: torch.Tensor,
              inv_freq: torch.Tensor | None, pairing: str = "half", q_gamma: torch.Tensor | None = None,
              k_gamma: torch.Tensor | None = None, eps: float = 1e-5, q_out: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kq_kv_append: the columns qkv (T, (n_q + 2 n_kv) head_dim) to rotated
    queries (T, n_q head_dim), returned, and keys and values in the cache at
    `slots`.  inv_freq: rot_dim/2 angles per position (None: no rotation);
    pairing "half" or "adjacent"."""
    if stream is None and q_out is not None and pairing in _PAIRING:
        st = (_fast or _load()).kv_append(qkv, n_q, cache._ref, slots, pos, inv_freq, _PAIRING[pairing], q_gamma, k_gamma, eps,
                                          q_out, status, cache._dev)
        if st is not None:
            if st:
                _check(st, "kq_kv_append")
            return q_out
    dev, f32, D = cache._dev, torch.float32, cache.head_dim
    if qkv.dim() == 1:
        qkv = qkv[None, :]
    T, nq = qkv.shape[0], n_q * D
    x, ld = _mat(dev, qkv, "qkv", f32, T, nq + 2 * cache.n_kv * D)
    if pairing not in _PAIRING:
        raise ValueError(f"unknown pairing {pairing!r}")
    if q_out is None:
        q_out = _empty((T, nq), f32, dev, stream)
    q, ldq = _mat(dev, q_out, "q_out", f32, T, nq)
    n = 0 if inv_freq is None else inv_freq.numel()
    rot = Rotary(_opt(dev, inv_freq, "inv_freq", f32, n), 2 * n, _PAIRING[pairing],
                 _opt(dev, q_gamma, "q_gamma", f32, D), _opt(dev, k_gamma, "k_gamma", f32, D), eps)
    _layer_call(_layer_lib().kq_kv_append, "kq_kv_append", dev, stream, T, x, ld, n_q, cache._ref,
                _vec(dev, slots, "slots", torch.int64, T), _vec(dev, pos, "pos", torch.int32, T), ctypes.addressof(rot),
                q, ldq, _opt(dev, status, "status", torch.int32, 1))
    return q_out


def kv_attn_workspace_bytes(R: int, max_q: int, n_q: int, cache: KVCache) -> int:
    """Bytes of kv_attn's workspace (kq_kv_attn_workspace_bytes), on the cache's device."""
    with torch.cuda.device(cache._dev):
        return int(_layer_lib().kq_kv_attn_workspace_bytes(_int(R, "R"), _int(max_q, "max_q"), _int(n_q, "n_q"),
                                                            cache._ref))


def kv_attn(q: torch.Tensor, cache: KVCache, lens: torch.Tensor, table: torch.Tensor,
            q_start: torch.Tensor | None = None, max_q: int = 1, scale: float | None = None, window: int = 0,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kq_kv_attn: attention of the query columns q (T, n_q head_dim) over the
    cache.  lens: tokens of each request in the cache, its query columns
    included; table (R, max_pages); q_start (R + 1): the requests' columns
    (None: one each); scale defaults to head_dim ** -0.5.  The workspace is
    allocated here (torch) when not given."""
    if stream is None and out is not None and workspace is not None:
        st = (_fast or _load()).kv_attn(q, cache._ref, lens, table, q_start, max_q,
                                        cache.head_dim ** -0.5 if scale is None else scale, window, out, workspace, status,
                                        cache._dev)
        if st is not None:
            if st:
                _check(st, "kq_kv_attn")
            return out
    dev, f32, i32, D = cache._dev, torch.float32, torch.int32, cache.head_dim
    T, cols = q.shape
    n_q, R, width, max_q, window = cols // D, lens.numel(), table.shape[-1], _int(max_q, "max_q"), _int(window, "window")
    if n_q * D != cols:
        raise ValueError(f"q must have head_dim = {D} columns per head, got {cols}")
    x, ldq = _mat(dev, q, "q", f32, T, cols)
    if out is None:
        out = _empty((T, cols), f32, dev, stream, torch.empty if q_start is None else torch.zeros)
    o, ldo = _mat(dev, out, "out", f32, T, cols)
    if workspace is None:
        n = max(16, kv_attn_workspace_bytes(R, max_q, n_q, cache))
        workspace = _empty(n, torch.uint8, dev, stream)
    else:
        n = workspace.nbytes
    tab, ld = _mat(dev, table, "table", i32, R, width)
    _layer_call(_layer_lib().kq_kv_attn, "kq_kv_attn", dev, stream, R, T, max_q, n_q, x, ldq, cache._ref,
                _vec(dev, lens, "lens", i32, R), _opt(dev, q_start, "q_start", i32, R + 1), tab, ld, width,
                D ** -0.5 if scale is None else scale, window, o, ldo,
                _vec(dev, workspace, "workspace", workspace.dtype, workspace.numel()), n,
                _opt(dev, status, "status", i32, 1))
    return out


def residual_norm(res: torch.Tensor | None, y: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                  post_gamma: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  pre_gamma: torch.Tensor | None = None, eps: float = 1e-5, out: torch.Tensor | None = None,
                  h: torch.Tensor | None = None, stream=None):
    """kq_residual_norm: (out, h) of the step after a block.  res (T, N); y
    (T, N) or (T, n_terms, N), with weights (T, n_terms); gate (N,) or
    (T, N).  out may be res; h is computed where pre_gamma is given (else
    None)."""
    if stream is None and out is not None and (h is None) == (pre_gamma is None):
        st = (_fast or _load()).residual_norm(out, res, y, weights, post_gamma, gate, scale, pre_gamma, eps, h)
        if st is not None:
            if st:
                _check(st, "kq_residual_norm")
            return out, h
    like = res if res is not None else y
    if like is None:
        raise ValueError("neither res nor y")
    dev, f32 = _index(like, "residual_norm"), torch.float32
    T, N = like.shape[0], like.shape[-1]
    a = Residual(scale=scale, eps=eps)
    if y is not None:
        if y.dim() == 2:
            a.n_terms = E = 1
            a.y, a.ldy = _mat(dev, y, "y", f32, T, N)
            a.ld_term = N
        else:
            a.n_terms = E = y.shape[1]
            if y.dtype is not f32 or y.get_device() != dev or y.shape != (T, E, N):
                _bad(dev, y, "y", f32, torch.Size((T, E, N)))
            if not y.is_contiguous() and N > 1 and y.stride(2) != 1:
                _bad(dev, y, "y", f32, y.shape)
            a.y, a.ldy, a.ld_term = y.data_ptr(), y.stride(0) if T > 1 else E * N, y.stride(1) if E > 1 else N
        if weights is not None:
            a.weights, a.ldw = _mat(dev, weights, "weights", f32, T, E)
    elif weights is not None:
        raise ValueError("weights without y")
    if post_gamma is not None:
        a.post_gamma = _vec(dev, post_gamma, "post_gamma", f32, N)
    if gate is not None:
        if gate.dim() == 1:
            a.gate = _vec(dev, gate, "gate", f32, N)
        else:
            a.gate, a.ldg = _mat(dev, gate, "gate", f32, T, N)
    if res is not None:
        a.res, a.ldres = _mat(dev, res, "res", f32, T, N)
    if out is None:
        out = _empty((T, N), f32, dev, stream)
    a.out, a.ldout = _mat(dev, out, "out", f32, T, N)
    if pre_gamma is not None:
        if h is None:
            h = _empty((T, N), f32, dev, stream)
        a.pre_gamma = _vec(dev, pre_gamma, "pre_gamma", f32, N)
        a.h, a.ldh = _mat(dev, h, "h", f32, T, N)
    elif h is not None:
        raise ValueError("h without pre_gamma")
    _layer_call(_layer_lib().kq_residual_norm, "kq_residual_norm", dev, stream, ctypes.addressof(a), T, N)
    return out, h


# --------------------------------------------------------------- chain
class MatrixDesc(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("fmt", ctypes.c_int), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


def _chain_sigs(L):
    if getattr(L, "_chain_ready", False):
        return
    vp = ctypes.c_void_p
    L.kq_chain_create.restype = ctypes.c_int
    L.kq_chain_create.argtypes = [ctypes.POINTER(MatrixDesc), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                  ctypes.POINTER(vp)]
    L.kq_chain_create_resident.restype = ctypes.c_int
    L.kq_chain_create_resident.argtypes = [ctypes.POINTER(MatrixDesc), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_int, ctypes.POINTER(vp)]
    L.kq_chain_plan.restype = ctypes.c_int
    L.kq_chain_plan.argtypes = [ctypes.POINTER(MatrixDesc), ctypes.c_int, ctypes.c_int, ctypes.c_size_t,
                                ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    L.kq_chain_resident_layers.restype = ctypes.c_int
    L.kq_chain_resident_layers.argtypes = [vp]
    L.kq_chain_slot_bytes.restype = ctypes.c_size_t
    L.kq_chain_slot_bytes.argtypes = [vp]
    L.kq_chain_run.restype = ctypes.c_int
    L.kq_chain_run.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
    L.kq_chain_wait.restype = ctypes.c_int
    L.kq_chain_wait.argtypes = [vp, ctypes.c_int64]
    L.kq_chain_last_error.restype = ctypes.c_char_p
    L.kq_chain_destroy.restype = None
    L.kq_chain_destroy.argtypes = [vp]
    L._chain_ready = True


def chain_plan(layers, budget_bytes: int, max_slots: int = 4):
    """kq_chain_plan: (n_resident, n_slots) for a device-memory budget.
    layers: list over layers of lists of (W, fmt, N, K) (W unused here)."""
    L = lib()
    _chain_sigs(L)
    flat = [m for layer in layers for m in layer]
    arr = (MatrixDesc * len(flat))()
    for i, (W, fmt, N, K) in enumerate(flat):
        arr[i] = MatrixDesc(None if W is None else W.data_ptr(), _fmt(fmt), N, K)
    r, s = ctypes.c_int(), ctypes.c_int()
    st = L.kq_chain_plan(arr, len(layers), len(layers[0]), budget_bytes, max_slots, ctypes.byref(r), ctypes.byref(s))
    if st != OK:
        raise KQError(st, "kq_chain_plan", L.kq_chain_last_error().decode())
    return int(r.value), int(s.value)


def _moe_stream_sigs(L):
    if getattr(L, "_moe_stream_sigs", False):
        return
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    L.kq_moe_stream_create.restype = i32
    L.kq_moe_stream_create.argtypes = [vp, i32, i32, i64, i64, sz, i32, i32, ctypes.POINTER(vp)]
    L.kq_moe_stream_run.restype = i32
    L.kq_moe_stream_run.argtypes = [vp, vp, i32, vp, i64, vp, vp]
    L.kq_moe_stream_wait.restype = i32
    L.kq_moe_stream_wait.argtypes = [vp, i64]
    L.kq_moe_stream_destroy.restype = None
    L.kq_moe_stream_destroy.argtypes = [vp]
    L.kq_moe_stream_last_error.restype = ctypes.c_char_p
    L._moe_stream_sigs = True


class MoEStream:
    """Routed experts kept in pinned host memory and copied to the device on
    demand (kq_moe_stream_* in kq.h).

    W_host: pinned uint8 tensor holding E expert matrices (N x K in fmt),
    expert e at byte e * stride (default N * row_bytes)."""

    def __init__(self, W_host, fmt, E: int, N: int, K: int, max_ids: int, n_sets: int = 2,
                 stride: int | None = None):
        L = lib()
        _moe_stream_sigs(L)
        self._L = L
        if W_host.is_cuda:
            raise ValueError("streamed experts must be host memory")
        self._keep = W_host
        self.N, self.K, self.max_ids = N, K, max_ids
        stride = stride if stride is not None else N * row_bytes(fmt, K)
        h = ctypes.c_void_p()
        st = L.kq_moe_stream_create(W_host.data_ptr(), _fmt(fmt), E, N, K, stride, max_ids, n_sets,
                                    ctypes.byref(h))
        if st != OK:
            raise KQError(st, "kq_moe_stream_create", L.kq_moe_stream_last_error().decode())
        self._h = h

    def run(self, ids_host, x, x_stride: int = 0, y=None, stream=None):
        """ids_host: int32 numpy array or CPU tensor; x, y: device tensors."""
        ids = np.ascontiguousarray(np.asarray(ids_host, dtype=np.int32))
        n = int(ids.size)
        if y is None:
            y = torch.empty((n, self.N), dtype=torch.float32, device=x.device)
        st = self._L.kq_moe_stream_run(self._h, ids.ctypes.data, n, _dev(x, "x", torch.float32), x_stride,
                                       _dev(y, "y", torch.float32), _stream(stream))
        if st != OK:
            raise KQError(st, "kq_moe_stream_run", self._L.kq_moe_stream_last_error().decode())
        return y

    def wait(self, timeout_ms: int = -1) -> None:
        st = self._L.kq_moe_stream_wait(self._h, timeout_ms)
        if st != OK:
            raise KQError(st, "kq_moe_stream_wait", self._L.kq_moe_stream_last_error().decode())

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._L.kq_moe_stream_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gguf_format(ggml_type: int) -> int:
    """libkq format id of a ggml type id (0 if none): kq_gguf_kq_format."""
    L = lib()
    L.kq_gguf_kq_format.restype = ctypes.c_int
    L.kq_gguf_kq_format.argtypes = [ctypes.c_int]
    return int(L.kq_gguf_kq_format(int(ggml_type)))


class GGUF:
    """Tensor table and tensor bytes of a GGUF file (kq_gguf_* in kq.h)."""

    def __init__(self, path: str):
        L = lib()
        if not getattr(L, "_gguf_sigs", False):
            i32, vp, u64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_uint64
            L.kq_gguf_open.restype = i32
            L.kq_gguf_open.argtypes = [ctypes.c_char_p, ctypes.POINTER(vp)]
            L.kq_gguf_tensor_count.restype = i32
            L.kq_gguf_tensor_count.argtypes = [vp]
            L.kq_gguf_tensor_info.restype = i32
            L.kq_gguf_tensor_info.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i32),
                                              ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_int64),
                                              ctypes.POINTER(u64), ctypes.POINTER(u64)]
            L.kq_gguf_find.restype = i32
            L.kq_gguf_find.argtypes = [vp, ctypes.c_char_p]
            L.kq_gguf_kq_format.restype = i32
            L.kq_gguf_kq_format.argtypes = [i32]
            L.kq_gguf_read.restype = i32
            L.kq_gguf_read.argtypes = [vp, i32, vp, u64]
            L.kq_gguf_close.restype = None
            L.kq_gguf_close.argtypes = [vp]
            L.kq_gguf_last_error.restype = ctypes.c_char_p
            L._gguf_sigs = True
        self._L = L
        h = ctypes.c_void_p()
        st = L.kq_gguf_open(os.fsencode(path), ctypes.byref(h))
        if st != OK:
            raise KQError(st, "kq_gguf_open", L.kq_gguf_last_error().decode())
        self._h = h

    def __len__(self) -> int:
        return int(self._L.kq_gguf_tensor_count(self._h))

    def info(self, i: int) -> dict:
        name, t, nd = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_int()
        dims = (ctypes.c_int64 * 4)()
        off, nb = ctypes.c_uint64(), ctypes.c_uint64()
        st = self._L.kq_gguf_tensor_info(self._h, i, ctypes.byref(name), ctypes.byref(t), ctypes.byref(nd), dims,
                                         ctypes.byref(off), ctypes.byref(nb))
        if st != OK:
            raise KQError(st, "kq_gguf_tensor_info", self._L.kq_gguf_last_error().decode())
        return dict(name=name.value.decode(), type=t.value, dims=list(dims)[:nd.value], offset=off.value,
                    nbytes=nb.value, fmt=int(self._L.kq_gguf_kq_format(t.value)))

    def find(self, name: str) -> int:
        return int(self._L.kq_gguf_find(self._h, name.encode()))

    def read(self, name_or_index) -> np.ndarray:
        i = name_or_index if isinstance(name_or_index, int) else self.find(name_or_index)
        nb = self.info(i)["nbytes"]
        out = np.empty(nb, np.uint8)
        st = self._L.kq_gguf_read(self._h, i, out.ctypes.data, nb)
        if st != OK:
            raise KQError(st, "kq_gguf_read", self._L.kq_gguf_last_error().decode())
        return out

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._L.kq_gguf_close(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Chain:
    """Layer chain whose weights stay in pinned host memory and stream
    through ``n_slots`` device slots (kq_chain_* in kq.h).

    mats: list over layers of lists of (W_host_pinned_uint8_tensor, fmt, N, K).
    n_resident: leading layers copied once into device memory of their own
    (kq_chain_create_resident); the rest stream.
    """

    def __init__(self, mats, n_slots: int = 4, n_resident: int = 0):
        L = lib()
        _chain_sigs(L)
        self._L = L
        self.n_layers = len(mats)
        self.per_layer = len(mats[0])
        flat = [m for layer in mats for m in layer]
        self._keep = [m[0] for m in flat]  # keep the host tensors alive
        arr = (MatrixDesc * len(flat))()
        for i, (W, fmt, N, K) in enumerate(flat):
            if W.is_cuda:
                raise ValueError("chain weights must be host memory")
            arr[i] = MatrixDesc(W.data_ptr(), _fmt(fmt), N, K)
        h = ctypes.c_void_p()
        st = L.kq_chain_create_resident(arr, self.n_layers, self.per_layer, n_resident, n_slots, ctypes.byref(h))
        if st != OK:
            raise KQError(st, "kq_chain_create_resident", L.kq_chain_last_error().decode())
        self._h = h

    @property
    def slot_bytes(self) -> int:
        return int(self._L.kq_chain_slot_bytes(self._h))

    @property
    def resident_layers(self) -> int:
        return int(self._L.kq_chain_resident_layers(self._h))

    def run(self, xs, ys, stream=None) -> None:
        n = self.n_layers * self.per_layer
        assert len(xs) == n and len(ys) == n
        xa = (ctypes.c_void_p * n)(*[_dev(x, "x", torch.float32) for x in xs])
        ya = (ctypes.c_void_p * n)(*[_dev(y, "y", torch.float32) for y in ys])
        st = self._L.kq_chain_run(self._h, xa, ya, _stream(stream))
        if st != OK:
            raise KQError(st, "kq_chain_run", self._L.kq_chain_last_error().decode())

    def wait(self, timeout_ms: int = -1) -> None:
        st = self._L.kq_chain_wait(self._h, timeout_ms)
        if st != OK:
            raise KQError(st, "kq_chain_wait", self._L.kq_chain_last_error().decode())

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._L.kq_chain_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LayerDesc(ctypes.Structure):
    """kq_layer_desc: one layer's matrices for kq_stream_chain_create."""
    _fields_ = [("mats", ctypes.POINTER(MatrixDesc)), ("n_mats", ctypes.c_int)]


class StreamChain(Chain):
    """The streamed chain through the per-layer entry points
    kq_stream_chain_create / kq_stream_chain / kq_stream_chain_destroy."""

    def __init__(self, mats, n_slots: int = 4):
        L = lib()
        _chain_sigs(L)
        if not getattr(L, "_stream_chain_ready", False):
            vp = ctypes.c_void_p
            L.kq_stream_chain_create.restype = ctypes.c_int
            L.kq_stream_chain_create.argtypes = [ctypes.POINTER(LayerDesc), ctypes.c_int, ctypes.c_int,
                                                 ctypes.POINTER(vp)]
            L.kq_stream_chain.restype = ctypes.c_int
            L.kq_stream_chain.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, ctypes.c_int64]
            L.kq_stream_chain_destroy.restype = None
            L.kq_stream_chain_destroy.argtypes = [vp]
            L._stream_chain_ready = True
        self._L = L
        self.n_layers = len(mats)
        self.per_layer = len(mats[0])
        self._keep = [m[0] for layer in mats for m in layer]
        self._arrays = []
        layers = (LayerDesc * self.n_layers)()
        for l, layer in enumerate(mats):
            arr = (MatrixDesc * len(layer))()
            for i, (W, fmt, N, K) in enumerate(layer):
                if W.is_cuda:
                    raise ValueError("chain weights must be host memory")
                arr[i] = MatrixDesc(W.data_ptr(), _fmt(fmt), N, K)
            self._arrays.append(arr)
            layers[l] = LayerDesc(arr, len(layer))
        h = ctypes.c_void_p()
        st = L.kq_stream_chain_create(layers, self.n_layers, n_slots, ctypes.byref(h))
        if st != OK:
            raise KQError(st, "kq_stream_chain_create", L.kq_chain_last_error().decode())
        self._h = h

    def run_wait(self, xs, ys, timeout_ms: int = -1, stream=None) -> None:
        """kq_stream_chain: one pass, waited for on the host (bounded)."""
        n = self.n_layers * self.per_layer
        assert len(xs) == n and len(ys) == n
        xa = (ctypes.c_void_p * n)(*[_dev(x, "x", torch.float32) for x in xs])
        ya = (ctypes.c_void_p * n)(*[_dev(y, "y", torch.float32) for y in ys])
        st = self._L.kq_stream_chain(self._h, xa, ya, _stream(stream), timeout_ms)
        if st != OK:
            raise KQError(st, "kq_stream_chain", self._L.kq_chain_last_error().decode())

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._L.kq_stream_chain_destroy(self._h)
            self._h = None
