"""Python binding of libpkv (the C ABI in include/pkv.h) through ctypes.

Argument marshalling only: every step of the attention runs in libpkv's CUDA
kernels. PyTorch provides device memory and the current stream. Importing this
module does not need a GPU; loading the library does not either, but running it
does, and there is no CPU path: if libpkv.so is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK = 0
PKV_ERR_INVALID_ARG = 1
PKV_ERR_UNSUPPORTED = 2
PKV_ERR_CUDA = 3
PKV_ERR_OOM = 4
PKV_ERR_DEVICE_BOUNDS = 5
PKV_ERR_TIMEOUT = 6

PKV_PREFILL = 0
PKV_DECODE = 1
PKV_PREFILL_RAGGED = 2
PKV_BF16 = 0
PKV_F32 = 1
PKV_FP8_E4M3 = 2
PKV_FP8_E5M2 = 3
PKV_FP4_E2M1 = 5

# Element types of the K/V caches, by name and by torch dtype. A 4-bit cache is a uint8
# tensor of two values a byte (float4_e2m1fn_x2 is taken for it too).
KV_DTYPES = {"bf16": PKV_BF16, "e4m3": PKV_FP8_E4M3, "e5m2": PKV_FP8_E5M2, "e2m1": PKV_FP4_E2M1}
_KV_TORCH = {PKV_BF16: torch.bfloat16, PKV_FP8_E4M3: torch.float8_e4m3fn,
             PKV_FP8_E5M2: torch.float8_e5m2, PKV_FP4_E2M1: torch.uint8}
_KV_CODES = {v: k for k, v in _KV_TORCH.items()}
_FP4_X2 = getattr(torch, "float4_e2m1fn_x2", torch.uint8)
_KV_CODES[_FP4_X2] = PKV_FP4_E2M1
_SCALE_TYPES = (torch.float8_e4m3fn, torch.uint8)
_BLOCK = 16  # columns that share a block scale of a 4-bit cache

EXPORTED = ("pkv_plan_create", "pkv_run", "pkv_merge_state", "pkv_plan_destroy",
            "pkv_plan_get_info", "pkv_plan_device_status", "pkv_status_string",
            "pkv_last_error", "pkv_abi_version", "pkv_plan_set_timing_events",
            "pkv_decode_noalloc", "pkv_plan_create_capturable", "pkv_plan_update",
            "pkv_build_kv_indices", "pkv_plan_create_sinks", "pkv_norm_rope_append",
            "pkv_pages_workspace", "pkv_pages_extend", "pkv_pages_fork", "pkv_pages_free",
            "pkv_pages_compact", "pkv_copy_pages", "pkv_run_blocks", "pkv_norm_rope_append_blocks",
            "pkv_gather_kv", "pkv_plan_create_shared", "pkv_copy_pages_blocks")


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{status}]")
        self.status = status


class PlanDesc(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("batch_size", ctypes.c_int32),
        ("qo_indptr", ctypes.c_void_p),
        ("kv_indptr", ctypes.c_void_p),
        ("kv_last_page_len", ctypes.c_void_p),
        ("q_start", ctypes.c_void_p),
        ("kv_indices", ctypes.c_void_p),
        ("num_pages", ctypes.c_int32),
        ("num_qo_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("window_left", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
        ("fixed_split_size", ctypes.c_int32),
        ("disable_split_kv", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("logits_soft_cap", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("kv_dtype", ctypes.c_int32),
        ("wait_limit_us", ctypes.c_int32),
        ("wait_probe", ctypes.c_int32),
    ]


class PlanCaps(ctypes.Structure):
    _fields_ = [
        ("max_batch", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("max_total_q", ctypes.c_int64),
    ]


class PlanGroups(ctypes.Structure):
    _fields_ = [
        ("num_groups", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("group_indptr", ctypes.c_void_p),
        ("shared_pages", ctypes.c_void_p),
    ]


class AppendDesc(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("num_qo_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("max_position", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class GatherDesc(ctypes.Structure):
    _fields_ = [
        ("total", ctypes.c_int64),
        ("num_indices", ctypes.c_int64),
        ("batch_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
    ]


class PoolDesc(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("refs", ctypes.c_void_p),
        ("row_stride", ctypes.c_int64),
        ("num_rows", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_int64),
        ("status", ctypes.c_void_p),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("num_work_items", ctypes.c_int32),
        ("num_partials", ctypes.c_int32),
        ("mask_mode", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
        ("total_q", ctypes.c_int64),
        ("kernels_per_run", ctypes.c_int32),
        ("kv_tile", ctypes.c_int32),
    ]


_lib = None
_lock = threading.Lock()


def load_library(path: Optional[str] = None):
    """Load libpkv.so (built by paged_kv_sliding_gb300.build); raises if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"libpkv.so not found at {path}: build it with "
                "`python -m paged_kv_sliding_gb300.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        lib.pkv_plan_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(PlanDesc), vp]
        lib.pkv_plan_create.restype = ctypes.c_int
        lib.pkv_run.argtypes = [vp, vp, vp, vp, vp, vp, vp]
        lib.pkv_run.restype = ctypes.c_int
        lib.pkv_merge_state.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, vp]
        lib.pkv_merge_state.restype = ctypes.c_int
        lib.pkv_plan_destroy.argtypes = [vp]
        lib.pkv_plan_destroy.restype = ctypes.c_int
        lib.pkv_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
        lib.pkv_plan_get_info.restype = ctypes.c_int
        lib.pkv_plan_device_status.argtypes = [vp, ctypes.POINTER(i32)]
        lib.pkv_plan_device_status.restype = ctypes.c_int
        lib.pkv_status_string.argtypes = [ctypes.c_int]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_last_error.argtypes = []
        lib.pkv_last_error.restype = ctypes.c_char_p
        lib.pkv_plan_set_timing_events.argtypes = [vp, vp, vp]
        lib.pkv_plan_set_timing_events.restype = ctypes.c_int
        lib.pkv_decode_noalloc.argtypes = [ctypes.POINTER(PlanDesc), vp, vp, vp, vp, vp, vp]
        lib.pkv_decode_noalloc.restype = ctypes.c_int
        lib.pkv_plan_create_capturable.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(PlanDesc),
                                                    ctypes.POINTER(PlanCaps), vp]
        lib.pkv_plan_create_capturable.restype = ctypes.c_int
        lib.pkv_plan_create_sinks.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(PlanDesc), i32,
                                              ctypes.POINTER(PlanCaps), vp]
        lib.pkv_plan_create_sinks.restype = ctypes.c_int
        lib.pkv_plan_create_shared.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(PlanDesc), ctypes.POINTER(PlanGroups),
                                               i32, vp]
        lib.pkv_plan_create_shared.restype = ctypes.c_int
        lib.pkv_plan_update.argtypes = [vp, ctypes.POINTER(PlanDesc), vp]
        lib.pkv_plan_update.restype = ctypes.c_int
        lib.pkv_build_kv_indices.argtypes = [vp, i32, i64, vp, vp, vp, i32, vp, i64, vp, vp, i64, vp, vp]
        lib.pkv_build_kv_indices.restype = ctypes.c_int
        lib.pkv_norm_rope_append.argtypes = [ctypes.POINTER(AppendDesc)] + [vp] * 14
        lib.pkv_norm_rope_append.restype = ctypes.c_int
        lib.pkv_norm_rope_append_blocks.argtypes = [ctypes.POINTER(AppendDesc)] + [vp] * 16
        lib.pkv_norm_rope_append_blocks.restype = ctypes.c_int
        lib.pkv_run_blocks.argtypes = [vp] * 9
        lib.pkv_run_blocks.restype = ctypes.c_int
        lib.pkv_gather_kv.argtypes = [ctypes.POINTER(GatherDesc)] + [vp] * 12
        lib.pkv_gather_kv.restype = ctypes.c_int
        pool = ctypes.POINTER(PoolDesc)
        for name, args in (("pkv_pages_workspace", [i32, i32, ctypes.POINTER(i64)]),
                           ("pkv_pages_extend", [pool, vp, vp, i32, vp, i64, vp]),
                           ("pkv_pages_fork", [pool, vp, vp, i32, vp, vp, vp]),
                           ("pkv_pages_free", [pool, vp, i32, vp]),
                           ("pkv_pages_compact", [pool, pool, vp, vp, i32, vp, vp]),
                           ("pkv_copy_pages", [vp, vp, i32, i64, i32, i64, vp, vp, i32, vp, vp, vp]),
                           ("pkv_copy_pages_blocks", [vp, vp, vp, vp, i32, i64, i64, i32, i64, i64, vp, vp, i32, vp, vp, vp])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        lib.pkv_abi_version.argtypes = []
        lib.pkv_abi_version.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int, what: str):
    if status != PKV_OK:
        lib = load_library()
        msg = lib.pkv_last_error().decode() or lib.pkv_status_string(status).decode()
        raise PkvError(status, f"{what}: {msg}")


# The current stream's handle without a Stream object around it (a third of the host time
# of a small call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream=None) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


# Memory of calls on a stream other than the current one. PyTorch gives a dropped tensor's
# memory to the next one made on the same stream at once, though another stream may still
# be using it: what the binding makes and keeps for a caller therefore says where it is used.

def _on(stream, *tensors):
    """The tensors are used on `stream`: dropped, they are kept until it has come this far."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream))
    for t in tensors:
        t.record_stream(stream)


def _within(stream):
    """The torch operations of a block go to `stream` (None: the current one)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream))
    return torch.cuda.stream(stream)


def _made(stream, make, *args, **kw):
    """The result of a call on an explicit stream, made by make(...): that stream's own memory
    (what the current stream has just given up may still be in use there), with the current
    stream, on which the caller goes on with it, recorded."""
    with _within(stream):
        t = make(*args, **kw)
    _on(torch.cuda.current_stream(), t)
    return t


def _empty(stream, shape, dtype, device):
    """Memory for the result of a call, on whatever stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _made(stream, torch.empty, shape, dtype=dtype, device=device)


def _ptrs(*tensors):
    return [None if t is None else t.data_ptr() for t in tensors]


def _sig(t):
    """What a call's checks and its descriptor go by: a tensor's type, shape, strides and device."""
    return None if t is None else (t.dtype, t.shape, t.stride(), t.device)


def _host_i32(a):
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class Plan:
    """A plan: the batch layout, head shape, window and causal mode, fixed once.

    kv_indices is a device int32 tensor borrowed by the plan (kept alive here).
    Host index arrays are copied by the library.
    """

    _fp4_page = None  # 4-bit caches: the shape of a page

    def __init__(self, *, kind: str, kv_indptr, num_qo_heads: int, num_kv_heads: int, head_dim: int,
                 kv_indices: Optional[torch.Tensor] = None, kv_last_page_len=None,
                 page_size: int = 1, num_pages: int = 0, window_left: int = -1, causal: bool = True,
                 sm_scale: Optional[float] = None, qo_indptr=None, q_start=None,
                 fixed_split_size: int = -1, disable_split_kv: bool = False, stream=None,
                 capacity: Optional[dict] = None, logits_soft_cap: float = 0.0, k_scale: float = 1.0,
                 v_scale: float = 1.0, kv_dtype="bf16", wait_limit_us: int = 0, wait_probe: bool = False,
                 num_sinks: int = 0, group_indptr=None, shared_pages=None):
        """kind: "prefill", "decode" or "prefill_ragged" (K/V passed to run() are
        contiguous [total_kv, H_kv, d]; kv_indptr counts tokens; no page table).
        capacity={"max_batch": B, "max_total_q": Q}: a capturable plan (its run may
        be captured in a CUDA graph and replayed after update()).
        kv_dtype: element type of the caches, "bf16", "e4m3", "e5m2" or "e2m1" (or the torch
        dtype); the 8-bit ones are for paged (decode and prefill) plans, the 4-bit one, whose
        caches come with block scales, for decode plans.
        wait_limit_us: bound of every device-side wait (<= 0: 2 s); wait_probe: make
        each CTA's first consuming wait run out (tests of the timeout path).
        num_sinks: first keys of each request that stay visible under the window.
        group_indptr [G + 1], shared_pages [G] (host; decode): requests group_indptr[g] ..
        group_indptr[g + 1] - 1 share their first shared_pages[g] pages, which are then read
        once for all of them."""
        self._lib = load_library()
        self._handle = ctypes.c_void_p()
        self.kind = kind
        if isinstance(kv_dtype, torch.dtype):
            kv_dtype = _KV_CODES.get(kv_dtype, -1)
        elif isinstance(kv_dtype, str):
            kv_dtype = KV_DTYPES.get(kv_dtype, -1)
        self._kv_torch = _KV_TORCH.get(int(kv_dtype))
        kv_indptr = _host_i32(kv_indptr)
        ragged = kind == "prefill_ragged"
        if kv_last_page_len is None:
            if not ragged:
                raise ValueError("kv_last_page_len is required for paged plans")
            kv_last_page_len = np.ones(len(kv_indptr) - 1, dtype=np.int32)
        kv_last_page_len = _host_i32(kv_last_page_len)
        qo_indptr = _host_i32(qo_indptr)
        q_start = _host_i32(q_start)
        if kv_indices is None:
            if not ragged:
                raise ValueError("kv_indices is required for paged plans")
            kv_indices = torch.zeros(0, dtype=torch.int32, device="cuda")
        if kv_indices.dtype != torch.int32 or not kv_indices.is_cuda:
            raise ValueError("kv_indices must be a device int32 tensor")
        self._kv_indices = kv_indices.contiguous()
        d = PlanDesc()
        d.kind = {"decode": PKV_DECODE, "prefill": PKV_PREFILL, "prefill_ragged": PKV_PREFILL_RAGGED}[kind]
        d.batch_size = len(kv_indptr) - 1
        d.qo_indptr = None if qo_indptr is None else qo_indptr.ctypes.data
        d.kv_indptr = kv_indptr.ctypes.data
        d.kv_last_page_len = kv_last_page_len.ctypes.data
        d.q_start = None if q_start is None else q_start.ctypes.data
        d.kv_indices = self._kv_indices.data_ptr() if self._kv_indices.numel() else None
        d.num_pages = int(num_pages)
        d.num_qo_heads = int(num_qo_heads)
        d.num_kv_heads = int(num_kv_heads)
        d.head_dim = int(head_dim)
        d.page_size = int(page_size)
        d.window_left = int(window_left)
        d.causal = 1 if causal else 0
        d.sm_scale = float(sm_scale if sm_scale is not None else head_dim ** -0.5)
        d.fixed_split_size = int(fixed_split_size)
        d.disable_split_kv = 1 if disable_split_kv else 0
        d.dtype = PKV_BF16
        d.logits_soft_cap = float(logits_soft_cap)
        d.k_scale = float(k_scale)
        d.v_scale = float(v_scale)
        d.kv_dtype = int(kv_dtype)
        d.wait_limit_us = int(wait_limit_us)
        d.wait_probe = 1 if wait_probe else 0
        self._desc = d
        if d.kv_dtype == PKV_FP4_E2M1:
            self._fp4_page = (d.page_size, d.num_kv_heads, d.head_dim // 2)
        caps = None
        if capacity is not None:
            caps = PlanCaps()
            caps.max_batch = int(capacity["max_batch"])
            caps.max_total_q = int(capacity.get("max_total_q", capacity["max_batch"]))
        if group_indptr is not None or shared_pages is not None:
            group_indptr, shared_pages = _host_i32(group_indptr), _host_i32(shared_pages)
            if group_indptr is None or shared_pages is None or len(group_indptr) != len(shared_pages) + 1:
                raise ValueError("group_indptr [G + 1] and shared_pages [G] come together")
            if caps is not None:
                raise ValueError("plans of shared prefixes take no capacity")
            gr = PlanGroups(len(shared_pages), 0, group_indptr.ctypes.data, shared_pages.ctypes.data)
            _check(self._lib.pkv_plan_create_shared(ctypes.byref(self._handle), ctypes.byref(d), ctypes.byref(gr),
                                                    int(num_sinks), _stream_handle(stream)), "pkv_plan_create_shared")
        elif num_sinks:
            _check(self._lib.pkv_plan_create_sinks(ctypes.byref(self._handle), ctypes.byref(d), int(num_sinks),
                                                   None if caps is None else ctypes.byref(caps),
                                                   _stream_handle(stream)), "pkv_plan_create_sinks")
        elif caps is None:
            _check(self._lib.pkv_plan_create(ctypes.byref(self._handle), ctypes.byref(d),
                                             _stream_handle(stream)), "pkv_plan_create")
        else:
            _check(self._lib.pkv_plan_create_capturable(ctypes.byref(self._handle), ctypes.byref(d),
                                                        ctypes.byref(caps), _stream_handle(stream)),
                   "pkv_plan_create_capturable")
        self.num_qo_heads = int(num_qo_heads)
        self.head_dim = int(head_dim)
        self.info = self.get_info()

    def update(self, *, kv_indptr, kv_last_page_len, qo_indptr=None, q_start=None,
               fixed_split_size: int = -1, disable_split_kv: bool = False, stream=None):
        """Re-plan a capturable plan for a new batch (same heads, window, page pool and
        kv_indices tensor, whose contents the caller has rewritten)."""
        kv_indptr = _host_i32(kv_indptr)
        kv_last_page_len = _host_i32(kv_last_page_len)
        qo_indptr = _host_i32(qo_indptr)
        q_start = _host_i32(q_start)
        d = PlanDesc.from_buffer_copy(self._desc)
        d.batch_size = len(kv_last_page_len)
        d.qo_indptr = None if qo_indptr is None else qo_indptr.ctypes.data
        d.kv_indptr = kv_indptr.ctypes.data
        d.kv_last_page_len = kv_last_page_len.ctypes.data
        d.q_start = None if q_start is None else q_start.ctypes.data
        d.fixed_split_size = int(fixed_split_size)
        d.disable_split_kv = 1 if disable_split_kv else 0
        _check(self._lib.pkv_plan_update(self._handle, ctypes.byref(d), _stream_handle(stream)),
               "pkv_plan_update")
        self.info = self.get_info()

    def get_info(self) -> dict:
        info = PlanInfo()
        _check(self._lib.pkv_plan_get_info(self._handle, ctypes.byref(info)), "pkv_plan_get_info")
        return {k: getattr(info, k) for k, _ in PlanInfo._fields_}

    def run(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
            return_lse: bool = False, stream=None, k_block_scales: Optional[torch.Tensor] = None,
            v_block_scales: Optional[torch.Tensor] = None):
        """Attention for the planned batch; returns out (and lse when asked). A 4-bit cache
        ([num_pages, P, H_kv, d / 2] bytes) comes with its block scales, [num_pages, P, H_kv,
        d / 16] float8_e4m3fn."""
        for t, name, dt in ((q, "q", torch.bfloat16), (k_cache, "k_cache", self._kv_torch),
                            (v_cache, "v_cache", self._kv_torch)):
            if (t.dtype != dt and (dt, t.dtype) != (torch.uint8, _FP4_X2)) or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
        blocks = self._kv_torch == torch.uint8
        if blocks:
            # (uint8 may be bytes of another width, of which the scales' shape says nothing)
            page = self._fp4_page
            if page is not None and not (k_cache.shape[1:] == v_cache.shape[1:] == page and
                                         min(k_cache.shape[0], v_cache.shape[0]) >= self._desc.num_pages):
                raise ValueError(f"k_cache and v_cache must be [{self._desc.num_pages}, {page[0]}, {page[1]}, {page[2]}] bytes")
            _block_scales(k_cache, k_block_scales, "k_block_scales")
            _block_scales(v_cache, v_block_scales, "v_block_scales")
        elif k_block_scales is not None or v_block_scales is not None:
            raise ValueError("block scales belong to 4-bit caches")
        if out is None:
            out = torch.empty_like(q) if stream is None else _made(stream, torch.empty_like, q)
        if return_lse and lse is None:
            lse = (torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device) if stream is None else
                   _made(stream, torch.empty, q.shape[:2], dtype=torch.float32, device=q.device))
        if blocks:
            _check(self._lib.pkv_run_blocks(self._handle, *_ptrs(q, k_cache, k_block_scales, v_cache, v_block_scales, out,
                                                                 lse), _stream_handle(stream)), "pkv_run_blocks")
        else:
            _check(self._lib.pkv_run(self._handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                     _ptr(lse), _stream_handle(stream)), "pkv_run")
        return (out, lse) if (return_lse or lse is not None) else out

    def set_timing_events(self, ev_begin, ev_end):
        """Raw cudaEvent_t handles (ints) recorded around the main kernel of later runs."""
        _check(self._lib.pkv_plan_set_timing_events(self._handle, ctypes.c_void_p(ev_begin or 0),
                                                    ctypes.c_void_p(ev_end or 0)),
               "pkv_plan_set_timing_events")

    def device_status(self) -> int:
        st = ctypes.c_int32(0)
        _check(self._lib.pkv_plan_device_status(self._handle, ctypes.byref(st)),
               "pkv_plan_device_status")
        return st.value

    def close(self):
        if getattr(self, "_handle", None) is not None and self._handle.value:
            self._lib.pkv_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def build_kv_indices(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, kv_start: torch.Tensor,
                     kv_lens: torch.Tensor, loc_map: Optional[torch.Tensor] = None, capacity: Optional[int] = None,
                     kv_indptr: Optional[torch.Tensor] = None, kv_indices: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None):
    """kv_indptr, kv_indices of a batch built on the device from a request-to-slot
    table (device int32 tensors). `capacity` bounds kv_indices; when neither it nor
    kv_indices is given it is read from kv_lens (one host read)."""
    lib = load_library()
    for t, name in ((req_to_token, "req_to_token"), (req_pool_indices, "req_pool_indices"),
                    (kv_start, "kv_start"), (kv_lens, "kv_lens")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor")
    B = kv_lens.numel()
    if kv_indptr is None:
        kv_indptr = _empty(stream, (B + 1,), torch.int32, kv_lens.device)
    if kv_indices is None:
        if capacity is None:
            with _within(stream):  # behind whatever writes them there
                capacity = int(kv_lens.clamp(min=0).sum().item())
        kv_indices = _empty(stream, (max(1, capacity),), torch.int32, kv_lens.device)
    cap = kv_indices.numel() if capacity is None else min(int(capacity), kv_indices.numel())
    _check(lib.pkv_build_kv_indices(_ptr(req_to_token), req_to_token.shape[0], req_to_token.shape[1],
                                    _ptr(req_pool_indices), _ptr(kv_start), _ptr(kv_lens), B, _ptr(loc_map),
                                    0 if loc_map is None else loc_map.numel(), _ptr(kv_indptr), _ptr(kv_indices),
                                    cap, _ptr(status), _stream_handle(stream)), "pkv_build_kv_indices")
    return kv_indptr, kv_indices


def _rows(t: torch.Tensor, name: str):
    """[tokens, heads, d] bf16 on the device whose heads are contiguous within a token."""
    n, h, d = t.shape
    if t.dtype != torch.bfloat16 or not t.is_cuda or (t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d))):
        raise ValueError(f"{name} must be a CUDA bf16 tensor [tokens, heads, d] with contiguous heads")
    return n, h, d, t.stride(0) if n > 1 else h * d


def _want(t: Optional[torch.Tensor], name: str, dtype, shape=None):
    if t is not None and (t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or
                          (shape is not None and tuple(t.shape) != tuple(shape))):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor" + (f" of shape {tuple(shape)}" if shape else ""))


def _block_scales(cache: torch.Tensor, scales: Optional[torch.Tensor], name: str):
    """The block scales of a 4-bit cache: an e4m3 code for every 16 columns (8 bytes) of a row."""
    if scales is None:
        raise ValueError(f"a 4-bit cache needs {name}")
    *pages, width = cache.shape
    if (scales.dtype not in _SCALE_TYPES or not scales.is_cuda or not scales.is_contiguous() or
            scales.shape != (*pages, width * 2 // _BLOCK)):
        raise ValueError(f"{name} must be a contiguous CUDA float8_e4m3fn tensor of the cache's shape with head_dim / 16 columns")


def _here(dev: int, *tensors):
    """The tensors live on the current device, whose stream the call is launched on."""
    for t in tensors:
        if t is not None and t.device.index != dev:
            raise ValueError(f"a tensor on {t.device}, but the current device is cuda:{dev}")


# Checked descriptors of earlier calls by what they were made from (types, shapes, strides
# and scalars), which a layer's calls of one step share.
_append_descs: dict = {}


def _append_desc(dev, eps, weight_offset, interleaved, k_scale, v_scale, q, k, v, q_weight, k_weight, cos_sin, positions,
                 slots, q_out, k_out, k_cache, v_cache, k_block_scales, v_block_scales, status):
    d = AppendDesc()
    n = dim = None
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is None:
            continue
        tn, heads, td, stride = _rows(t, name)
        if n is not None and (tn != n or td != dim):
            raise ValueError("q, k and v must agree in tokens and head_dim")
        n, dim = tn, td
        setattr(d, name + "_stride", stride)
        if name == "q":
            d.num_qo_heads = heads
        elif name == "k":
            d.num_kv_heads = heads
        elif k is None or heads != d.num_kv_heads:
            raise ValueError("k and v must have the same heads")
    if n is None:
        raise ValueError("q or k is required")
    d.num_tokens, d.head_dim = n, dim
    _want(positions, "positions", torch.int32, (n,))
    _want(slots, "slots", torch.int64, (n,))
    _want(q_weight, "q_weight", torch.bfloat16, (dim,))
    _want(k_weight, "k_weight", torch.bfloat16, (dim,))
    _want(status, "status", torch.int32)
    if cos_sin is not None:
        _want(cos_sin, "cos_sin", torch.float32)
        d.max_position, d.rotary_dim = cos_sin.shape
        if positions is None:
            raise ValueError("cos_sin needs positions")
    if k_cache is not None or v_cache is not None:
        if k_cache is None or v_cache is None or slots is None or v is None:
            raise ValueError("k_cache, v_cache, v and slots come together")
        code = _KV_CODES.get(k_cache.dtype)
        fp4 = code == PKV_FP4_E2M1
        if code is None or k_cache.dim() != 4 or tuple(k_cache.shape[2:]) != (d.num_kv_heads, dim // 2 if fp4 else dim):
            raise ValueError("k_cache must be [num_pages, page_size, H_kv, d], bf16 or 8-bit, or [..., d / 2] bytes of 4-bit values")
        _want(k_cache, "k_cache", k_cache.dtype)
        _want(v_cache, "v_cache", k_cache.dtype, k_cache.shape)
        if fp4:
            _block_scales(k_cache, k_block_scales, "k_block_scales")
            _block_scales(v_cache, v_block_scales, "v_block_scales")
        d.num_pages, d.page_size, d.kv_dtype = k_cache.shape[0], k_cache.shape[1], code
    if (k_block_scales is not None or v_block_scales is not None) and d.kv_dtype != PKV_FP4_E2M1:
        raise ValueError("block scales belong to 4-bit caches")
    if q is not None:
        _want(q_out, "q_out", torch.bfloat16, (n, d.num_qo_heads, dim))
    if k is not None:
        _want(k_out, "k_out", torch.bfloat16, (n, d.num_kv_heads, dim))
    _here(dev, q, k, v, positions, cos_sin, slots, k_cache, v_cache, q_weight, k_weight, q_out, k_out, k_block_scales,
          v_block_scales, status)
    d.eps, d.weight_offset, d.interleaved = eps, weight_offset, 1 if interleaved else 0
    d.k_scale, d.v_scale = k_scale, v_scale
    return d


def norm_rope_append(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor] = None, *,
                     positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
                     slots: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                     v_cache: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_offset: float = 0.0,
                     interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0,
                     q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None, k_block_scales: Optional[torch.Tensor] = None,
                     v_block_scales: Optional[torch.Tensor] = None):
    """Normalise each head of q and k, rotate them by their tokens' positions and write k
    and v into the paged caches, in one pass; returns q_out (None without q).

    q [n, H_qo, d], k and v [n, H_kv, d] bf16, possibly slices of one projection (heads
    contiguous, any token stride); q_weight / k_weight [d] bf16 (None: no norm); cos_sin
    [max_position, rotary_dim] fp32 (cosines, then sines; None: no rotation); positions
    [n] int32; slots [n] int64 (page * page_size + offset; negative: a padding row, not
    written); caches [num_pages, P, H_kv, d] bf16, float8_e4m3fn or float8_e5m2, or 4-bit:
    [..., d / 2] uint8 with k_block_scales and v_block_scales [..., d / 16] float8_e4m3fn, which
    are written with them; or both None with k_out [n, H_kv, d]. status: device int32 word for
    out-of-range slots and positions."""
    lib = _lib or load_library()
    # Plain values before the descriptor is looked up: a tensor of one number would be found
    # by its identity, and with it the value that it had in an earlier call.
    if not (eps.__class__ is weight_offset.__class__ is k_scale.__class__ is v_scale.__class__ is float):
        eps, weight_offset, k_scale, v_scale = float(eps), float(weight_offset), float(k_scale), float(v_scale)
    if interleaved is not False and interleaved is not True:
        interleaved = bool(interleaved)
    if q is not None and q_out is None:
        q_out = _empty(stream, q.shape, torch.bfloat16, q.device)
    dev = torch.cuda.current_device()
    tensors = (q, k, v, q_weight, k_weight, cos_sin, positions, slots, q_out, k_out, k_cache, v_cache, k_block_scales,
               v_block_scales, status)
    key = (dev, eps, weight_offset, interleaved, k_scale, v_scale) + tuple(map(_sig, tensors))
    d = _append_descs.get(key)
    if d is None:
        d = _append_desc(dev, eps, weight_offset, interleaved, k_scale, v_scale, *tensors)
        if len(_append_descs) >= 1024:
            _append_descs.clear()
        _append_descs[key] = d
    if d.kv_dtype == PKV_FP4_E2M1:
        _check(lib.pkv_norm_rope_append_blocks(d, *_ptrs(*tensors), _stream_handle(stream)), "pkv_norm_rope_append_blocks")
    else:
        _check(lib.pkv_norm_rope_append(d, *_ptrs(*tensors[:12]), None if status is None else status.data_ptr(),
                                        _stream_handle(stream)), "pkv_norm_rope_append")
    return q_out


_gather_descs: dict = {}  # as _append_descs


def _gather_desc(dev, k_scale, v_scale, k_cache, v_cache, k_block_scales, v_block_scales, kv_indptr, kv_indices, kv_start,
                 out_indptr, k_out, v_out, status):
    d = GatherDesc()
    code = _KV_CODES.get(k_cache.dtype)
    if code is None or k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, H_kv, d], bf16 or 8-bit, or [..., d / 2] bytes of 4-bit values")
    _want(k_cache, "k_cache", k_cache.dtype)
    _want(v_cache, "v_cache", k_cache.dtype, k_cache.shape)
    if code == PKV_FP4_E2M1:
        _block_scales(k_cache, k_block_scales, "k_block_scales")
        _block_scales(v_cache, v_block_scales, "v_block_scales")
    elif k_block_scales is not None or v_block_scales is not None:
        raise ValueError("block scales belong to 4-bit caches")
    if kv_indptr.dim() != 1 or kv_indptr.shape[0] < 1:
        raise ValueError("kv_indptr must hold batch + 1 offsets")
    d.batch_size = kv_indptr.shape[0] - 1
    _want(kv_indptr, "kv_indptr", torch.int32)
    _want(out_indptr, "out_indptr", torch.int32, kv_indptr.shape)
    _want(kv_indices, "kv_indices", torch.int32)
    _want(kv_start, "kv_start", torch.int32, (d.batch_size,))
    _want(status, "status", torch.int32)
    dim = k_cache.shape[3] * (2 if code == PKV_FP4_E2M1 else 1)
    if k_out.dim() != 3 or tuple(k_out.shape[1:]) != (k_cache.shape[2], dim):
        raise ValueError("k_out must be [rows, H_kv, d]")
    _want(k_out, "k_out", torch.bfloat16)
    _want(v_out, "v_out", torch.bfloat16, k_out.shape)
    _here(dev, k_cache, v_cache, k_block_scales, v_block_scales, kv_indptr, kv_indices, kv_start, out_indptr, k_out, v_out,
          status)
    d.total, d.num_indices, d.num_kv_heads, d.head_dim = k_out.shape[0], kv_indices.numel(), k_cache.shape[2], dim
    d.num_pages, d.page_size, d.kv_dtype, d.k_scale, d.v_scale = k_cache.shape[0], k_cache.shape[1], code, k_scale, v_scale
    return d


def gather_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, *, kv_indptr: torch.Tensor, kv_indices: torch.Tensor,
              out_indptr: torch.Tensor, total: Optional[int] = None, kv_start: Optional[torch.Tensor] = None,
              k_scale: float = 1.0, v_scale: float = 1.0, k_block_scales: Optional[torch.Tensor] = None,
              v_block_scales: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              v_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Cached rows read back as contiguous bf16 K and V [total, H_kv, d], which a
    "prefill_ragged" plan takes: rows out_indptr[b] .. out_indptr[b + 1] - 1 are rows kv_start[b]
    (0), ... of request b, whose pages are kv_indices[kv_indptr[b] .. kv_indptr[b + 1] - 1] (device
    int32). Caches of every type; a 4-bit one comes with its block scales. Without outputs,
    `total` says how many rows to make. status: device int32 word for rows that the pages do
    not hold, which are zeros."""
    lib = _lib or load_library()
    if not (k_scale.__class__ is v_scale.__class__ is float):  # plain values, as in norm_rope_append
        k_scale, v_scale = float(k_scale), float(v_scale)
    if k_out is None or v_out is None:
        if total is None:
            raise ValueError("total, or k_out and v_out, are required")
        heads, dim = k_cache.shape[-2:]
        shape = (total, heads, dim * 2 if _KV_CODES.get(k_cache.dtype) == PKV_FP4_E2M1 else dim)
        k_out = _empty(stream, shape, torch.bfloat16, k_cache.device) if k_out is None else k_out
        v_out = _empty(stream, shape, torch.bfloat16, k_cache.device) if v_out is None else v_out
    dev = torch.cuda.current_device()
    tensors = (k_cache, v_cache, k_block_scales, v_block_scales, kv_indptr, kv_indices, kv_start, out_indptr, k_out, v_out,
               status)
    key = (dev, k_scale, v_scale) + tuple(map(_sig, tensors))
    d = _gather_descs.get(key)
    if d is None:
        d = _gather_desc(dev, k_scale, v_scale, *tensors)
        if len(_gather_descs) >= 1024:
            _gather_descs.clear()
        _gather_descs[key] = d
    _check(lib.pkv_gather_kv(d, *_ptrs(*tensors), _stream_handle(stream)), "pkv_gather_kv")
    return k_out, v_out


class PagePool:
    """The pages of a cache on the device: table [rows, max_pages] page ids, lens [rows]
    tokens and refs [num_pages] int32 (how many table entries in use name a page; 0: free),
    all CUDA tensors that stay the caller's. Calls are asynchronous on the current stream, or
    on `stream`, which the caller orders behind the one that the pool was made on; what they
    could not do is in device_status(). A pool's calls share its workspace, so they must not
    overlap on several streams; a pool outlives the graphs that its calls were captured in."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, *, page_size: int):
        self._lib = load_library()
        if table.dim() != 2 or lens.dim() != 1 or refs.dim() != 1 or lens.shape[0] != table.shape[0]:
            raise ValueError("table is [rows, max_pages], lens [rows], refs [num_pages]")
        for t, name in ((table, "table"), (lens, "lens"), (refs, "refs")):
            _want(t, name, torch.int32)
        _here(torch.cuda.current_device(), table, lens, refs)
        self.table, self.lens, self.refs, self.page_size = table, lens, refs, int(page_size)
        self._device = table.get_device()
        size = ctypes.c_int64()
        _check(self._lib.pkv_pages_workspace(table.shape[0], refs.shape[0], ctypes.byref(size)), "pkv_pages_workspace")
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=table.device)
        self._status = torch.zeros(1, dtype=torch.int32, device=table.device)
        d = PoolDesc()
        d.table, d.lens, d.refs = table.data_ptr(), lens.data_ptr(), refs.data_ptr()
        d.row_stride, d.num_rows, d.num_pages, d.page_size = table.shape[1], table.shape[0], refs.shape[0], self.page_size
        d.workspace, d.workspace_bytes, d.status = self._workspace.data_ptr(), size.value, self._status.data_ptr()
        self._desc = d
        self._streams = {_stream_handle()}  # whose memory this is, and those that it is recorded on

    @classmethod
    def empty(cls, *, num_rows: int, max_pages: int, num_pages: int, page_size: int, device="cuda") -> "PagePool":
        """A pool without tokens."""
        zeros = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        return cls(zeros(num_rows, max_pages), zeros(num_rows), zeros(num_pages), page_size=page_size)

    def _used_on(self, stream, handle):
        """A call's stream, which from now on may be using the pool's memory."""
        if handle not in self._streams:  # (a tensor stays recorded)
            _on(torch.cuda.current_stream() if stream is None else stream, self.table, self.lens, self.refs,
                self._workspace, self._status)
            self._streams.add(handle)

    def _index(self, *tensors):
        if torch.cuda.current_device() != self._device:
            raise ValueError(f"the pool is on cuda:{self._device}, which is not the current device")
        n = tensors[0].numel()
        for t in tensors:
            if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n or t.get_device() != self._device:
                raise ValueError("index arrays must be contiguous CUDA int32 tensors of one length, on the pool's device")
        return n

    def extend(self, rows: torch.Tensor, add: torch.Tensor, total: Optional[int] = None,
               slots: Optional[torch.Tensor] = None, stream=None):
        """rows[i] grows by add[i] tokens. With `total`, the sum of add, the new tokens' int64
        slots are returned, entry after entry."""
        n = self._index(rows, add)
        if slots is None and total is not None:
            slots = _empty(stream, (total,), torch.int64, self.table.device)
        elif slots is not None:
            _want(slots, "slots", torch.int64)
            _here(self._device, slots)
        handle = _stream_handle(stream)
        if handle not in self._streams:
            self._used_on(stream, handle)
        _check(self._lib.pkv_pages_extend(self._desc, rows.data_ptr(), add.data_ptr(), n,
                                          None if slots is None else slots.data_ptr(),
                                          0 if slots is None else slots.numel(), handle),
               "pkv_pages_extend")
        return slots

    def fork(self, parents: torch.Tensor, children: torch.Tensor, src: Optional[torch.Tensor] = None,
             dst: Optional[torch.Tensor] = None, stream=None):
        """children[i], an empty row, becomes a copy of parents[i]: full pages are shared, a
        partly filled last one is new. Returns (src, dst), the pages to copy (or -1)."""
        if src is None:
            src = torch.empty_like(parents) if stream is None else _made(stream, torch.empty_like, parents)
        if dst is None:
            dst = torch.empty_like(parents) if stream is None else _made(stream, torch.empty_like, parents)
        n = self._index(parents, children, src, dst)
        handle = _stream_handle(stream)
        if handle not in self._streams:
            self._used_on(stream, handle)
        _check(self._lib.pkv_pages_fork(self._desc, parents.data_ptr(), children.data_ptr(), n, src.data_ptr(),
                                        dst.data_ptr(), handle), "pkv_pages_fork")
        return src, dst

    def free(self, rows: torch.Tensor, stream=None):
        """The rows become empty; pages that no other row names are free again."""
        n = self._index(rows)
        handle = _stream_handle(stream)
        if handle not in self._streams:
            self._used_on(stream, handle)
        _check(self._lib.pkv_pages_free(self._desc, rows.data_ptr(), n, handle), "pkv_pages_free")

    def compact(self, out: Optional["PagePool"] = None, src: Optional[torch.Tensor] = None,
                dst: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None, stream=None):
        """The pages in use move to the lowest ids; the new table, lens and refs go to `out`
        (None: in place). Returns (src, dst, count): the pages to copy, and how many on the
        device. The caches' pages are the caller's to copy (copy_pages) before the new
        table is used."""
        if src is None:
            src = _empty(stream, (self.refs.shape[0] // 2,), torch.int32, self.table.device)
        if dst is None:
            dst = _empty(stream, src.shape, torch.int32, self.table.device)
        if count is None:
            count = _empty(stream, (1,), torch.int32, self.table.device)
        n = self._index(src, dst)
        self._index(count)
        out = self if out is None else out
        if out._device != self._device:
            raise ValueError(f"the pools are on cuda:{self._device} and cuda:{out._device}")
        handle = _stream_handle(stream)
        self._used_on(stream, handle)
        out._used_on(stream, handle)
        _check(self._lib.pkv_pages_compact(self._desc, out._desc, src.data_ptr(), dst.data_ptr(), n,
                                           count.data_ptr(), handle), "pkv_pages_compact")
        return src, dst, count

    def device_status(self) -> int:
        """Read and clear what earlier calls recorded (waits for the device)."""
        torch.cuda.synchronize(self.table.device)
        st = int(self._status.item())
        self._status.zero_()
        # cleared before the next call, on whatever stream, can record anything
        torch.cuda.synchronize(self.table.device)
        return st


def copy_pages(k_cache: torch.Tensor, v_cache: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
               count: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None,
               k_block_scales: Optional[torch.Tensor] = None, v_block_scales: Optional[torch.Tensor] = None):
    """Page dst[i] of both caches becomes page src[i]. Caches [num_pages, P, H_kv, d], or
    [layers, num_pages, P, H_kv, d] for every layer at once, contiguous, of any type; src
    and dst int32, negative ids skipped; count: a device int32 of how many pairs are
    meant (default: all). The block scales of a 4-bit cache ([..., d / 16]) are copied with it when
    they are given."""
    lib = _lib or load_library()
    shape, dev = k_cache.shape, torch.cuda.current_device()
    if shape != v_cache.shape or k_cache.dtype != v_cache.dtype or len(shape) not in (4, 5):
        raise ValueError("k_cache and v_cache must be [num_pages, P, H_kv, d] or [layers, num_pages, P, H_kv, d]")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if src.shape != dst.shape:
        raise ValueError("src and dst must have one length")
    ptrs = []
    for t in (src, dst, count, status):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype != torch.int32 or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError("src, dst, count and status must be contiguous int32 tensors on the current CUDA device")
        ptrs.append(t.data_ptr())
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError("the caches must be on the current CUDA device")
    layers = shape[0] if len(shape) == 5 else 1
    pages = shape[-4]
    layer_bytes = k_cache.numel() * k_cache.element_size() // layers if layers else 0
    if k_block_scales is not None or v_block_scales is not None:
        if _KV_CODES.get(k_cache.dtype) != PKV_FP4_E2M1:
            raise ValueError("block scales belong to 4-bit caches")
        _block_scales(k_cache, k_block_scales, "k_block_scales")
        _block_scales(v_cache, v_block_scales, "v_block_scales")
        if k_block_scales.get_device() != dev or v_block_scales.get_device() != dev:
            raise ValueError("the block scales must be on the current CUDA device")
        scale_bytes = k_block_scales.numel() // layers if layers else 0
        _check(lib.pkv_copy_pages_blocks(k_cache.data_ptr(), v_cache.data_ptr(), k_block_scales.data_ptr(),
                                         v_block_scales.data_ptr(), layers, layer_bytes, scale_bytes, pages,
                                         layer_bytes // pages if pages else 0, scale_bytes // pages if pages else 0, ptrs[0],
                                         ptrs[1], src.numel(), ptrs[2], ptrs[3], _stream_handle(stream)), "pkv_copy_pages_blocks")
        return
    _check(lib.pkv_copy_pages(k_cache.data_ptr(), v_cache.data_ptr(), layers, layer_bytes, pages,
                              layer_bytes // pages if pages else 0, ptrs[0], ptrs[1], src.numel(), ptrs[2], ptrs[3],
                              _stream_handle(stream)), "pkv_copy_pages")


def plan(**kw) -> Plan:
    return Plan(**kw)


def merge_state(v_a: torch.Tensor, s_a: torch.Tensor, v_b: torch.Tensor, s_b: torch.Tensor,
                v_out: Optional[torch.Tensor] = None, s_out: Optional[torch.Tensor] = None,
                stream=None):
    """(v, s) = merge((v_a, s_a), (v_b, s_b)); v: [tokens, heads, d] bf16 or fp32."""
    lib = load_library()
    if v_a.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("values must be bf16 or fp32")
    if v_a.shape != v_b.shape or v_a.dim() != 3 or s_a.shape != v_a.shape[:2] or s_b.shape != s_a.shape:
        raise ValueError("shape mismatch")
    if v_out is None:
        v_out = torch.empty_like(v_a) if stream is None else _made(stream, torch.empty_like, v_a)
    if s_out is None:
        s_out = torch.empty_like(s_a) if stream is None else _made(stream, torch.empty_like, s_a)
    dtype = PKV_BF16 if v_a.dtype == torch.bfloat16 else PKV_F32
    _check(lib.pkv_merge_state(_ptr(v_a), _ptr(s_a), _ptr(v_b), _ptr(s_b), _ptr(v_out), _ptr(s_out),
                               v_a.shape[0], v_a.shape[1], v_a.shape[2], dtype,
                               _stream_handle(stream)), "pkv_merge_state")
    return v_out, s_out


def plan_for(w, device="cuda", **over) -> Plan:
    """A Plan for a paged_kv_sliding_gb300.inputs.Workload (test/bench convenience)."""
    kv_indices = torch.as_tensor(w.kv_indices, dtype=torch.int32).to(device)
    args = dict(kind=w.kind, kv_indptr=w.kv_indptr, kv_indices=kv_indices,
                kv_last_page_len=w.kv_last_page_len, num_qo_heads=w.num_qo_heads,
                num_kv_heads=w.num_kv_heads, head_dim=w.head_dim, page_size=w.page_size,
                num_pages=w.num_pages, window_left=w.window_left, causal=w.causal,
                sm_scale=w.sm_scale, qo_indptr=None if w.kind == "decode" else w.qo_indptr,
                q_start=w.q_start, kv_dtype=w.k_cache.dtype)
    args.update(over)
    return Plan(**args)
