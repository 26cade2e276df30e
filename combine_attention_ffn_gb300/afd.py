"""Thin Python binding of libafd (include/afd.h) over ctypes.

Argument marshalling only: tensors become pointers and sizes (CUDA tensors,
or page-locked CPU tensors, which the library reads and writes in place over
the host link; it refuses pageable ones), the current PyTorch stream becomes
the call's stream, and the library's device memory comes back as zero-copy
tensors. Every step of the exchange runs in
the library's CUDA kernels; there is no fallback. If ``libafd.so`` has not
been built, :func:`load_library` raises.

The names follow the afdEP-comm "API contract": ``source_dispatch``,
``worker_receive``, ``worker_reply``, ``source_collect``. On one GPU the
source and worker ranks are index arguments of one :class:`Buffer`.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libafd.so")

OK, ERR_ARG, ERR_STATE, ERR_BUCKET, ERR_RECEIPT = 0, 1, 2, 3, 4
ERR_ROUTE_RANGE, ERR_ROUTE_DUP, ERR_CUDA, ERR_OOM, ERR_CAPTURING, ERR_UNSUPPORTED = 5, 6, 7, 8, 9, 10
ERR_TIMEOUT = 11
BF16, FP8_E4M3, FP32 = 0, 1, 2
SCORINGS = {"softmax": 0, "sigmoid": 1}
COMBINE_FUSED, COMBINE_TWO_STAGE, COMBINE_TWO_STAGE_FP8 = 0, 1, 2
PRODUCT_WAIT_CYCLES = 4_000_000_000  # afd_set_product_wait_limit's default

EXPORTS = ("afd_create", "afd_destroy", "afd_source_dispatch", "afd_source_dispatch_cached",
           "afd_worker_receive",
           "afd_worker_reply", "afd_source_collect", "afd_source_collect_all", "afd_get_error",
           "afd_clear_error",
           "afd_reset_exchange", "afd_status_string", "afd_error_detail", "afd_arena_rows",
           "afd_recv_rows_for_bucket", "afd_version", "afd_route_layout_noalloc",
           "afd_set_wait_limit", "afd_phase_stamps", "afd_l2_flush", "afd_route_topk",
           "afd_grouped_linear", "afd_gated_rows", "afd_adapter_add", "afd_adapter_workspace_bytes",
           "afd_set_product_wait_limit")


class AfdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_sources", "num_workers", "num_experts", "top_k", "hidden", "capacity",
        "expert_alignment", "dtype", "num_sms", "combine_mode")]


class Recv(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("row_scales", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("row_src", ctypes.c_void_p),
                ("ends", ctypes.c_void_p), ("host_counts", ctypes.c_void_p),
                ("num_rows", ctypes.c_int64), ("receipt", ctypes.c_uint64)]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("num_tokens", ctypes.c_int32), ("is_view", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads libafd.so (once). Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise AfdError(ERR_UNSUPPORTED, f"{p} is missing; build it with "
                       "`python -m combine_attention_ffn_gb300.build`")
    lib = ctypes.CDLL(p)
    v, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    P = ctypes.POINTER
    sigs = {
        "afd_create": (i32, [P(Config), i32, P(v)]),
        "afd_destroy": (i32, [v]),
        "afd_source_dispatch": (i32, [v, i32, v, v, v, v, i64, i64, i32, i32, i32, v]),
        "afd_source_dispatch_cached": (i32, [v, i32, v, v, v, i64, i64, i32, i32, i32, v]),
        "afd_worker_receive": (i32, [v, i32, i32, i32, v, P(Recv)]),
        "afd_worker_reply": (i32, [v, i32, v, i64, u64, v]),
        "afd_source_collect": (i32, [v, i32, v, i32, v, P(View)]),
        "afd_source_collect_all": (i32, [v, v, i32, v, v]),
        "afd_get_error": (i32, [v, P(i32), P(i32), P(i32), P(i32)]),
        "afd_clear_error": (i32, [v, v]),
        "afd_reset_exchange": (i32, [v]),
        "afd_status_string": (ctypes.c_char_p, [i32]),
        "afd_error_detail": (ctypes.c_char_p, [v]),
        "afd_arena_rows": (i64, [v]),
        "afd_recv_rows_for_bucket": (i64, [v, i32]),
        "afd_version": (i32, []),
        "afd_route_layout_noalloc": (i32, [v, i32, i32, i32, i32, i32, v, v, v, v]),
        "afd_set_wait_limit": (i32, [v, i32]),
        "afd_phase_stamps": (i32, [v, P(u64), i64, i32]),
        "afd_l2_flush": (i32, [v, i64, v]),
        "afd_route_topk": (i32, [v, i32, i64, v, v, i32, i32, i32, i32, i32, ctypes.c_float, v, v, v]),
        "afd_grouped_linear": (i32, [v, i64, v, v, v, v, i32, i32, i64, i32, i32, i32, i32, v, i64, v, v]),
        "afd_set_product_wait_limit": (i32, [i64]),
        "afd_gated_rows": (i32, [v, i64, v, i32, i32, i64, i32, v, i64, v]),
        "afd_adapter_add": (i32, [v, i64, v, i64, v, v, v, v, v, v, v, i32, i32, i64, i32, i32, i32, i32,
                                  i32, v, i64, v, i64, v]),
        "afd_adapter_workspace_bytes": (i64, [i64, i32, i32, i32, i32, i32, i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        _lib = lib
    return lib


def use_library(path: str) -> ctypes.CDLL:
    """Makes the library at `path` (e.g. the phase-timer build) the one every
    Buffer created afterwards calls."""
    global _lib
    _lib = load_library(path)
    return _lib


# afd_phase_stamps: [kind][block][point] (afd.h)
STAMP_KINDS = ("dispatch", "scatter", "combine", "combine-early")
STAMP_SHAPE = (4, 4096, 8)


class _Context:
    """Owns one afd_ctx. It is destroyed when the Buffer is closed and no
    tensor that views the context's memory is alive any more, so a view can
    never outlive the memory it points at."""

    def __init__(self, lib, handle: ctypes.c_void_p):
        self.lib = lib
        self.handle = handle

    def __del__(self):
        try:
            if self.handle is not None and self.handle.value:
                self.lib.afd_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


class _DeviceArray:
    """Exposes library-owned device memory through __cuda_array_interface__;
    the tensor made from it keeps the owning context alive."""

    def __init__(self, ptr: int, shape, typestr: str, owner):
        self.__cuda_array_interface__ = {"shape": tuple(int(s) for s in shape), "typestr": typestr,
                                         "data": (int(ptr or 0), False), "version": 2,
                                         "strides": None}
        self._owner = owner


def _wrap(ptr, shape, dtype: torch.dtype, owner, device) -> torch.Tensor:
    base = {torch.int32: "<i4", torch.float32: "<f4", torch.bfloat16: "<i2",
            torch.float8_e4m3fn: "|u1", torch.uint8: "|u1"}[dtype]
    t = torch.as_tensor(_DeviceArray(ptr, shape, base, owner), device=device)
    if dtype == torch.bfloat16:
        t = t.view(torch.bfloat16)
    elif dtype == torch.float8_e4m3fn:
        t = t.view(torch.float8_e4m3fn)
    return t


def _stream_handle(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device.index)
    return int(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


@dataclass
class Receive:
    """One worker's received rows (zero-copy views of the context's arena)."""
    rows: torch.Tensor                 # [num_rows, H] bf16 or float8_e4m3fn
    row_scales: Optional[torch.Tensor]  # [num_rows, H/128] f32 (FP8)
    weights: torch.Tensor              # [num_rows] f32
    row_src: torch.Tensor              # [num_rows] i32
    ends: torch.Tensor                 # [E/F] i32 on the device
    host_counts: Optional[np.ndarray]  # [E/F] aligned counts (read_host_counts)
    num_rows: int
    receipt: int


class Buffer:
    """One context: A sources and F workers exchanging through this GPU's HBM."""

    def __init__(self, num_sources: int, num_workers: int, num_experts: int, top_k: int,
                 hidden: int, capacity: int, expert_alignment: int = 1, dtype: str = "bf16",
                 num_sms: int = 0, device=None, combine_mode: int = COMBINE_FUSED):
        self._lib = load_library()
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index or 0)
        self.cfg = Config(num_sources, num_workers, num_experts, top_k, hidden, capacity,
                          expert_alignment, FP8_E4M3 if dtype == "fp8" else BF16, num_sms,
                          combine_mode)
        self.dtype = dtype
        self.A, self.F, self.E, self.K, self.H = num_sources, num_workers, num_experts, top_k, hidden
        self.Ef = num_experts // max(num_workers, 1)
        self.capacity, self.alpha = capacity, expert_alignment
        h = ctypes.c_void_p()
        st = self._lib.afd_create(ctypes.byref(self.cfg), self.device.index, ctypes.byref(h))
        if st != OK:
            raise AfdError(st, "afd_create: " + self._lib.afd_status_string(st).decode())
        self._ctx = _Context(self._lib, h)
        self._h = h
        self._views = {}

    # the dtype the top-k IDs must have ("API contract": buffer.topk_idx_dtype)
    topk_idx_dtype = torch.int64

    # -- helpers ------------------------------------------------------------
    def _check(self, st: int, what: str):
        if st != OK:
            detail = self._lib.afd_error_detail(self._h).decode() if self._h else ""
            raise AfdError(st, f"{what}: {self._lib.afd_status_string(st).decode()}: {detail}")

    def _view(self, ptr, shape, dtype: torch.dtype) -> torch.Tensor:
        """A tensor over context-owned memory. The arenas never move, so the
        tensors are made once per (address, shape, dtype) and reused."""
        key = (int(ptr or 0), tuple(shape), dtype)
        t = self._views.get(key)
        if t is None:
            if len(self._views) >= 256:  # exact receive shapes vary with read_host_counts
                self._views.clear()
            t = _wrap(ptr, shape, dtype, self._ctx, self.device)
            self._views[key] = t
        return t

    @property
    def handle(self) -> int:
        return int(self._h.value or 0)

    def arena_rows(self) -> int:
        return int(self._lib.afd_arena_rows(self._h))

    def recv_rows_for_bucket(self, bucket: int) -> int:
        return int(self._lib.afd_recv_rows_for_bucket(self._h, bucket))

    # -- the four calls -------------------------------------------------------
    def source_dispatch(self, source: int, x: torch.Tensor, ids: torch.Tensor,
                        weights: torch.Tensor, x_scale: Optional[torch.Tensor] = None, *,
                        bucket: int, read_host_counts: bool = False, stream=None) -> None:
        T = int(x.shape[0]) if x is not None else 0
        if T:
            want = torch.float8_e4m3fn if self.dtype == "fp8" else torch.bfloat16
            if x.dtype != want or tuple(x.shape) != (T, self.H) or not x.is_contiguous():
                raise AfdError(ERR_ARG, f"x must be contiguous {want} [T, {self.H}]")
            if ids.dtype != torch.int64 or tuple(ids.shape) != (T, self.K) or not ids.is_contiguous():
                raise AfdError(ERR_ARG, f"ids must be contiguous int64 [T, {self.K}]")
            if weights.dtype != torch.float32 or tuple(weights.shape) != (T, self.K) \
                    or not weights.is_contiguous():
                raise AfdError(ERR_ARG, f"weights must be contiguous float32 [T, {self.K}]")
        sst = ssb = 0
        if x_scale is not None:
            if x_scale.dtype != torch.float32 or tuple(x_scale.shape) != (T, self.H // 128):
                raise AfdError(ERR_ARG, f"x_scale must be float32 [T, {self.H // 128}]")
            sst, ssb = x_scale.stride()
        st = self._lib.afd_source_dispatch(self._h, source, _ptr(x) if T else None,
                                           _ptr(ids) if T else None, _ptr(weights) if T else None,
                                           _ptr(x_scale) if T else None, sst, ssb, T, bucket,
                                           int(bool(read_host_counts)),
                                           _stream_handle(stream, self.device))
        self._check(st, "source_dispatch")

    def source_dispatch_cached(self, source: int, x: torch.Tensor, weights: Optional[torch.Tensor] = None,
                               x_scale: Optional[torch.Tensor] = None, *, bucket: int,
                               read_host_counts: bool = False, stream=None) -> None:
        """Dispatch with the routing (IDs, layout, receipts) of the last exchange;
        only the rows move. `weights` replaces the routing weights of the same
        IDs, or None keeps them."""
        T = int(x.shape[0]) if x is not None else 0
        if T:
            want = torch.float8_e4m3fn if self.dtype == "fp8" else torch.bfloat16
            if x.dtype != want or tuple(x.shape) != (T, self.H) or not x.is_contiguous():
                raise AfdError(ERR_ARG, f"x must be contiguous {want} [T, {self.H}]")
            if weights is not None and (weights.dtype != torch.float32 or
                                        tuple(weights.shape) != (T, self.K) or not weights.is_contiguous()):
                raise AfdError(ERR_ARG, f"weights must be contiguous float32 [T, {self.K}]")
        sst = ssb = 0
        if x_scale is not None:
            if x_scale.dtype != torch.float32 or tuple(x_scale.shape) != (T, self.H // 128):
                raise AfdError(ERR_ARG, f"x_scale must be float32 [T, {self.H // 128}]")
            sst, ssb = x_scale.stride()
        st = self._lib.afd_source_dispatch_cached(self._h, source, _ptr(x) if T else None,
                                                  _ptr(weights) if T else None,
                                                  _ptr(x_scale) if T else None, sst, ssb, T, bucket,
                                                  int(bool(read_host_counts)),
                                                  _stream_handle(stream, self.device))
        self._check(st, "source_dispatch_cached")

    def worker_receive(self, worker: int, *, bucket: int, read_host_counts: bool = False,
                       stream=None) -> Receive:
        r = Recv()
        st = self._lib.afd_worker_receive(self._h, worker, bucket, int(bool(read_host_counts)),
                                          _stream_handle(stream, self.device), ctypes.byref(r))
        self._check(st, "worker_receive")
        n = int(r.num_rows)
        rows_dtype = torch.float8_e4m3fn if self.dtype == "fp8" else torch.bfloat16
        hc = None
        if r.host_counts:
            hc = np.ctypeslib.as_array(ctypes.cast(r.host_counts, ctypes.POINTER(ctypes.c_int32)),
                                       shape=(self.Ef,)).copy()
        return Receive(
            rows=self._view(r.rows, (n, self.H), rows_dtype),
            row_scales=self._view(r.row_scales, (n, self.H // 128), torch.float32) if r.row_scales else None,
            weights=self._view(r.weights, (n,), torch.float32),
            row_src=self._view(r.row_src, (n,), torch.int32),
            ends=self._view(r.ends, (self.Ef,), torch.int32),
            host_counts=hc, num_rows=n, receipt=int(r.receipt))

    def worker_reply(self, worker: int, rows: torch.Tensor, receipt: int, stream=None) -> None:
        if rows.dtype != torch.bfloat16 or rows.dim() != 2 or rows.shape[1] != self.H \
                or not rows.is_contiguous():
            raise AfdError(ERR_ARG, f"reply rows must be contiguous bfloat16 [rows, {self.H}]")
        st = self._lib.afd_worker_reply(self._h, worker, _ptr(rows), int(rows.shape[0]),
                                        ctypes.c_uint64(receipt), _stream_handle(stream, self.device))
        self._check(st, "worker_reply")

    def source_collect(self, source: int, *, view: bool = False, out: Optional[torch.Tensor] = None,
                       num_tokens: Optional[int] = None, stream=None) -> torch.Tensor:
        """BF16 [T, H]. With view=True and one worker, a read-only view of the
        context's inbox (valid until the next source_dispatch)."""
        v = View()
        if out is None and not (view and self.F == 1):
            if num_tokens is None:
                raise AfdError(ERR_ARG, "pass out= or num_tokens=")
            out = torch.empty((num_tokens, self.H), dtype=torch.bfloat16, device=self.device)
        st = self._lib.afd_source_collect(self._h, source, _ptr(out), int(bool(view)),
                                          _stream_handle(stream, self.device), ctypes.byref(v))
        self._check(st, "source_collect")
        if v.is_view:
            return self._view(v.data, (int(v.num_tokens), int(v.row_stride)), torch.bfloat16)[:, : self.H]
        return out

    def source_collect_all(self, *, view: bool = False, outs=None, num_tokens=None, stream=None):
        """Every source's result with one call (one combine launch).
        Returns a list of BF16 [T_s, H] tensors (views with view=True and F == 1)."""
        if outs is None:
            if view and self.F == 1:
                outs = [None] * self.A
            else:
                if num_tokens is None:
                    raise AfdError(ERR_ARG, "pass outs= or num_tokens=")
                outs = [torch.empty((t, self.H), dtype=torch.bfloat16, device=self.device)
                        for t in num_tokens]
        ptrs = (ctypes.c_void_p * self.A)(*[_ptr(o) if o is not None else None for o in outs])
        views = (View * self.A)()
        st = self._lib.afd_source_collect_all(self._h, ptrs, int(bool(view)),
                                              _stream_handle(stream, self.device), views)
        self._check(st, "source_collect_all")
        res = []
        for s in range(self.A):
            v = views[s]
            if v.is_view:
                res.append(self._view(v.data, (int(v.num_tokens), int(v.row_stride)), torch.bfloat16)[:, : self.H])
            else:
                res.append(outs[s])
        return res

    # -- errors and lifetime ---------------------------------------------------
    def get_error(self):
        c, s, t, k = (ctypes.c_int32() for _ in range(4))
        st = self._lib.afd_get_error(self._h, ctypes.byref(c), ctypes.byref(s), ctypes.byref(t),
                                     ctypes.byref(k))
        self._check(st, "get_error")
        return c.value, s.value, t.value, k.value

    def clear_error(self, stream=None) -> None:
        self._check(self._lib.afd_clear_error(self._h, _stream_handle(stream, self.device)),
                    "clear_error")

    def reset_exchange(self) -> None:
        self._check(self._lib.afd_reset_exchange(self._h), "reset_exchange")

    def phase_stamps(self, clear: bool = False) -> np.ndarray:
        """The phase-timer build's %globaltimer stamps, uint64 STAMP_SHAPE
        (afd_phase_stamps); synchronizes the device. Raises AfdError with
        ERR_UNSUPPORTED on the default build."""
        out = np.zeros(STAMP_SHAPE, dtype=np.uint64)
        st = self._lib.afd_phase_stamps(self._h, out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
                                        out.size, int(bool(clear)))
        self._check(st, "phase_stamps")
        return out

    def set_wait_limit(self, polls: int) -> None:
        """Polls of each bulk row load before the scatter reports AFD_ERR_TIMEOUT
        (afd_set_wait_limit; 0 makes every first wait give up at once)."""
        self._check(self._lib.afd_set_wait_limit(self._h, polls), "set_wait_limit")

    def __enter__(self) -> "Buffer":
        return self

    def __exit__(self, *exc) -> None:
        self.close()

    def close(self) -> None:
        """Releases the context. Its memory is freed (after the device work
        completes) once no tensor viewing it is alive."""
        self._views = {}
        self._ctx = None
        self._h = ctypes.c_void_p()


def route_layout_noalloc(ids: torch.Tensor, num_experts: int, num_workers: int,
                         expert_alignment: int, ends: torch.Tensor, slots: torch.Tensor,
                         error: torch.Tensor, stream=None) -> None:
    """Routing layout into caller-provided outputs; the library allocates
    nothing (its scratch is a fixed device array). See
    afd_route_layout_noalloc in include/afd.h for the limits and rules."""
    lib = load_library()
    T, K = (int(ids.shape[0]), int(ids.shape[1])) if ids.dim() == 2 else (0, 1)
    for name, t, dt in (("ends", ends, torch.int32), ("slots", slots, torch.int32),
                        ("error", error, torch.int32), ("ids", ids, torch.int64)):
        if t.dtype != dt or not t.is_contiguous():
            raise AfdError(ERR_ARG, f"{name} must be contiguous {dt}")
    st = lib.afd_route_layout_noalloc(_ptr(ids) if T else None, T, K, num_experts, num_workers,
                                      expert_alignment, _ptr(ends), _ptr(slots) if T else None,
                                      _ptr(error), _stream_handle(stream, ids.device))
    if st != OK:
        raise AfdError(st, "afd_route_layout_noalloc: " + lib.afd_status_string(st).decode())


# -- the experts' side of an exchange (afd.h: no context, no state) -----------
# Forward only: with gradients enabled, inputs that require them are refused.
# A decode step's call is shorter on the GPU than on the host, so the binding
# asks PyTorch for the raw stream and device number where it has them: the
# public objects around them cost 1 us a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, on: torch.Tensor, stream, *args) -> None:
    """Calls a context-free entry point on a stream of the device of `on`, with
    that device current (the library works on the current one)."""
    lib = _lib or load_library()
    index, current = on.get_device(), _current_device()
    if index < 0:  # page-locked host memory
        index = current
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == current:
        st = getattr(lib, name)(*args, handle)
    else:
        with torch.cuda.device(index):
            st = getattr(lib, name)(*args, handle)
    if st != OK:
        raise AfdError(st, f"{name}: {lib.afd_status_string(st).decode()}")


_INT32 = 0x7fffffff
_grad_enabled = torch.is_grad_enabled


def _too_large(*sizes: int) -> AfdError:
    """The C ABI's sizes have 32 bits (ctypes would keep their low ones, and the
    call work on a part)."""
    return AfdError(ERR_UNSUPPORTED, f"sizes {sizes} must fit 32 bits")


def _no_backward() -> AfdError:
    """Autograd would take the result for a constant."""
    return AfdError(ERR_UNSUPPORTED, "no backward pass: inputs that require gradients are taken "
                    "under torch.no_grad() only, or detached")


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """A new tensor from the pool of the stream that will use it (what the
    allocator hands out on another one may still be in use there)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _want(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> int:
    """Checks a dense tensor; returns its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise AfdError(ERR_ARG, f"{name} must be contiguous {dtype} {list(shape)}, "
                       f"got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _want_rows(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> int:
    """Checks a [rows, columns] tensor whose rows may be strided; returns the
    row stride in elements."""
    if t.dtype is dtype and t.shape == shape:
        row, col = t.stride()
        if shape[0] <= 1:
            row = shape[1]
        if row >= shape[1] and (col == 1 or shape[1] <= 1):
            return row
    raise AfdError(ERR_ARG, f"{name} must be {dtype} {list(shape)} with dense rows, got {t.dtype} {list(t.shape)}")


def route_topk(logits: torch.Tensor, top_k: int, *, scoring: str = "softmax",
               bias: Optional[torch.Tensor] = None, renormalize: bool = True, scale: float = 1.0,
               live_tokens: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None, stream=None):
    """The router: ``(ids, weights)`` of every token's `top_k` experts, int64
    and float32 [T, top_k], as :meth:`Buffer.source_dispatch` takes them.

    `logits` is [T, E], bf16 or float32. Scores are softmax or sigmoid of the
    logits; `bias` (float32 [E]) is added to them for the selection only.
    Ties go to the lowest index; NaN and -inf are never selected and slots
    without an expert get ID -1 and weight 0. `live_tokens` (int32 [1], on the
    device) makes the tokens from there on padding. See afd_route_topk in
    include/afd.h."""
    if logits.dim() != 2 or logits.dtype not in (torch.bfloat16, torch.float32):
        raise AfdError(ERR_ARG, f"logits must be bfloat16 or float32 [T, E], got {logits.dtype}")
    if scoring not in SCORINGS:
        raise AfdError(ERR_ARG, f"scoring must be one of {sorted(SCORINGS)}, got {scoring!r}")
    T, E = logits.shape
    if T > _INT32 or E > _INT32 or not -_INT32 <= top_k <= _INT32:
        raise _too_large(T, E, top_k)
    if _grad_enabled() and (logits.requires_grad or (bias is not None and bias.requires_grad)
                            or (weights is not None and weights.requires_grad)):
        raise _no_backward()
    stride = _want_rows(logits, "logits", logits.dtype, (T, E))
    bias_ptr = None if bias is None else _want(bias, "bias", torch.float32, (E,))
    live_ptr = None if live_tokens is None else _want(live_tokens, "live_tokens", torch.int32, (1,))
    shape = (T, top_k)
    if ids is None:
        ids = _empty(shape, torch.int64, logits.device, stream)
    else:
        _want(ids, "ids", torch.int64, shape)
    if weights is None:
        weights = _empty(shape, torch.float32, logits.device, stream)
    else:
        _want(weights, "weights", torch.float32, shape)
    _call("afd_route_topk", ids, stream, logits.data_ptr(), FP32 if logits.dtype is torch.float32 else BF16, stride,
          bias_ptr, live_ptr, T, E, top_k, SCORINGS[scoring], bool(renormalize), scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def grouped_linear(x: torch.Tensor, weight: torch.Tensor, ends: torch.Tensor, *, expert_alignment: int = 1,
                   gated: bool = False, x_scale: Optional[torch.Tensor] = None,
                   weight_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' matrix product over received rows: ``out[r] = x[r] @
    weight[l].T`` for the rows of every expert l, BF16.

    `x` is [R, K] and `weight` [E/F, N, K], both bf16, or both float8_e4m3fn
    with `x_scale` [R, K/128] and `weight_scale` [E/F, N/128, K/128]. `ends`
    and `expert_alignment` are those of the exchange
    (:attr:`Receive.ends`). With `gated` the weight has the gate's rows first
    and the up projection's after them ([E/F, 2N, K]) and ``out = silu(gate) *
    up``. Rows outside every expert's range are left as they were (`out`) or
    unspecified (without `out`). `error` (int32 [1]) receives ERR_TIMEOUT if a
    bounded wait of the kernel gave up (:func:`set_product_wait_limit`); without
    it nothing tells of that. See afd_grouped_linear in include/afd.h."""
    if x.dim() != 2 or weight.dim() != 3 or x.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise AfdError(ERR_ARG, "x must be [R, K] bfloat16 or float8_e4m3fn and weight [G, N, K]")
    R, K = x.shape
    G, W = weight.shape[0], weight.shape[1]
    if G > _INT32 or W > _INT32 or K > _INT32 or not -_INT32 <= expert_alignment <= _INT32:
        raise _too_large(G, W, K, expert_alignment)
    if _grad_enabled() and (x.requires_grad or weight.requires_grad or (out is not None and out.requires_grad)
                            or (x_scale is not None and x_scale.requires_grad)
                            or (weight_scale is not None and weight_scale.requires_grad)):
        raise _no_backward()
    fp8 = x.dtype == torch.float8_e4m3fn
    if gated and W % 2:
        raise AfdError(ERR_ARG, f"a gated weight has an even number of rows, got {W}")
    N = W // 2 if gated else W
    x_stride = _want_rows(x, "x", x.dtype, (R, K))
    w_ptr = _want(weight, "weight", x.dtype, (G, W, K))
    ends_ptr = _want(ends, "ends", torch.int32, (G,))
    xs_ptr = ws_ptr = error_ptr = None
    if fp8:
        if x_scale is None or weight_scale is None or K % 128 or N % 128:
            raise AfdError(ERR_ARG, "float8_e4m3fn takes x_scale, weight_scale and K, N that are multiples of 128")
        xs_ptr = _want(x_scale, "x_scale", torch.float32, (R, K // 128))
        ws_ptr = _want(weight_scale, "weight_scale", torch.float32, (G, W // 128, K // 128))
    elif x_scale is not None or weight_scale is not None:
        raise AfdError(ERR_ARG, "bfloat16 rows take no scales")
    if out is None:
        out = _empty((R, N), torch.bfloat16, x.device, stream)
    out_stride = _want_rows(out, "out", torch.bfloat16, (R, N))
    if error is not None:
        error_ptr = _want(error, "error", torch.int32, (1,))
    _call("afd_grouped_linear", x, stream, x.data_ptr(), x_stride, xs_ptr, w_ptr, ws_ptr, ends_ptr, G, expert_alignment,
          R, K, N, FP8_E4M3 if fp8 else BF16, bool(gated), out.data_ptr(), out_stride, error_ptr)
    return out


def set_product_wait_limit(cycles: int = PRODUCT_WAIT_CYCLES) -> None:
    """The most clocks of an SM for which a wait inside :func:`grouped_linear`'s
    kernel lasts, for the process's calls from now on (the default: about two
    seconds; 0: give up at once). See afd_set_product_wait_limit in
    include/afd.h."""
    lib = _lib or load_library()
    if not 0 <= cycles < 1 << 63:
        raise AfdError(ERR_ARG, f"cycles must be in [0, 2^63), got {cycles}")
    lib.afd_set_product_wait_limit(cycles)


def gated_rows(h: torch.Tensor, ends: torch.Tensor, *, expert_alignment: int = 1,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gated activation over received rows, BF16: ``out[r] = silu(h[r, :N])
    * h[r, N:]`` for `h` [R, 2N]; rows outside every expert's range are left
    as they were. `out` may be ``h[:, :N]``. See afd_gated_rows in
    include/afd.h."""
    if h.dim() != 2 or h.shape[1] % 2:
        raise AfdError(ERR_ARG, "h must be bfloat16 [R, 2N]")
    R, N = h.shape[0], h.shape[1] // 2
    h_stride = _want_rows(h, "h", torch.bfloat16, (R, 2 * N))
    G = ends.numel()
    if G > _INT32 or N > _INT32 or not -_INT32 <= expert_alignment <= _INT32:
        raise _too_large(G, N, expert_alignment)
    if _grad_enabled() and (h.requires_grad or (out is not None and out.requires_grad)):
        raise _no_backward()
    ends_ptr = _want(ends, "ends", torch.int32, (G,))
    if out is None:
        out = _empty((R, N), torch.bfloat16, h.device, stream)
    out_stride = _want_rows(out, "out", torch.bfloat16, (R, N))
    _call("afd_gated_rows", ends, stream, h.data_ptr(), h_stride, ends_ptr, G, expert_alignment, R, N, out.data_ptr(),
          out_stride)
    return out


def adapter_add(base: torch.Tensor, x: torch.Tensor, down: torch.Tensor, up: torch.Tensor,
                token_slots: torch.Tensor, scales: torch.Tensor, *, row_src: Optional[torch.Tensor] = None,
                ends: Optional[torch.Tensor] = None, top_k: int = 1, x_scale: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Low-rank adapters of many requests beside a shared projection, BF16:
    ``out[r] = base[r] + scales[a] * up[a] @ (down[a] @ x[r])`` with a =
    ``token_slots[row_src[r] // top_k]`` (received rows: `row_src`, `ends` and
    `top_k` of the exchange, token_slots over [A * bucket] tokens) or
    ``token_slots[r]`` (a source's own tokens). A slot outside [0, S) means no
    adapter. `x` is bf16, or float8_e4m3fn with `x_scale` [R, K/128]; `down`
    is [S, rank, K], `up` [S, N, rank]; `out` defaults to `base` (in place). See afd_adapter_add in include/afd.h."""
    if base.dim() != 2 or x.dim() != 2 or down.dim() != 3:
        raise AfdError(ERR_ARG, "base must be [R, N], x [R, K], down [S, rank, K] and up [S, N, rank]")
    (R, N), K, (S, rank, _) = base.shape, x.shape[1], down.shape
    base_stride = _want_rows(base, "base", torch.bfloat16, (R, N))
    x_stride = _want_rows(x, "x", torch.bfloat16 if x_scale is None else torch.float8_e4m3fn, (R, K))
    xs_ptr = None if x_scale is None else _want(x_scale, "x_scale", torch.float32, (R, K // 128))
    down_ptr = _want(down, "down", torch.bfloat16, (S, rank, K))
    up_ptr = _want(up, "up", torch.bfloat16, (S, N, rank))
    scales_ptr = _want(scales, "scales", torch.float32, (S,))
    tokens = token_slots.numel()
    if tokens > _INT32 or S > _INT32 or rank > _INT32 or K > _INT32 or N > _INT32 or not -_INT32 <= top_k <= _INT32:
        raise _too_large(tokens, S, rank, K, N, top_k)
    if _grad_enabled() and (base.requires_grad or x.requires_grad or down.requires_grad or up.requires_grad
                            or scales.requires_grad or (out is not None and out.requires_grad)
                            or (x_scale is not None and x_scale.requires_grad)):
        raise _no_backward()
    slots_ptr = _want(token_slots, "token_slots", torch.int32, (tokens,))
    G, src_ptr, ends_ptr = 0, None, None
    if row_src is not None:
        if ends is None:
            raise AfdError(ERR_ARG, "row_src needs the exchange's ends, int32 [G]")
        G = ends.numel()
        if G > _INT32:
            raise _too_large(G)
        src_ptr = _want(row_src, "row_src", torch.int32, (R,))
        ends_ptr = _want(ends, "ends", torch.int32, (G,))
    elif tokens < R:
        raise AfdError(ERR_ARG, f"token_slots has {tokens} entries for {R} rows")
    if out is None:
        out, out_stride = base, base_stride
    else:
        out_stride = _want_rows(out, "out", torch.bfloat16, (R, N))
    size = (_lib or load_library()).afd_adapter_workspace_bytes(R, tokens, top_k if G else 0, S, rank, K, N)
    workspace = None
    if size > 0:
        on = x.device if x.is_cuda else torch.device("cuda", _current_device())
        workspace = _empty(size, torch.uint8, on, stream)
    _call("afd_adapter_add", x, stream, base.data_ptr(), base_stride, x.data_ptr(), x_stride, xs_ptr, down_ptr, up_ptr,
          slots_ptr, scales_ptr, src_ptr, ends_ptr, G, top_k, R, tokens, S, rank, K, N, out.data_ptr(), out_stride,
          None if workspace is None else workspace.data_ptr(), size)
    return out
