"""ctypes binding of libsplitkv (``include/splitkv.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libsplitkv.so``.  PyTorch supplies device memory and streams.
Loading fails loudly when the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsplitkv.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_WORKSPACE = 3
ERR_CUDA = 4
ERR_TIMEOUT = 5
ERR_DEVICE_CHECK = 6

GQA, MLA = 0, 1
F32, BF16 = 0, 1
PLAN_UNIFORM, PLAN_CRITICAL_WAVE = 0, 1


class SplitKVError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libsplitkv status {status}: {message}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim_qk", ctypes.c_int32), ("head_dim_v", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32), ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("qo_indptr", ctypes.c_void_p), ("seq_lens_host", ctypes.c_void_p),
        ("qo_indptr_host", ctypes.c_void_p),
        ("kv_fp8", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
    ]


class PlanParams(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32), ("uniform_splits", ctypes.c_int32),
        ("min_splits", ctypes.c_int32), ("max_splits", ctypes.c_int32),
        ("num_ctas", ctypes.c_int32), ("warps_per_cta", ctypes.c_int32),
        ("tile_tokens", ctypes.c_int32), ("decode_qlen_max", ctypes.c_int32),
        ("rho", ctypes.c_double), ("delta_attn", ctypes.c_double),
        ("delta_red", ctypes.c_double), ("gamma", ctypes.c_double),
        ("adopt_margin", ctypes.c_double),
        ("interleave", ctypes.c_int32), ("partial_dtype", ctypes.c_int32),
        ("trace", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class TraceRecord(ctypes.Structure):
    _fields_ = [("start_ns", ctypes.c_uint64), ("end_ns", ctypes.c_uint64), ("id", ctypes.c_int32),
                ("sm", ctypes.c_int32), ("kind", ctypes.c_int32), ("cta", ctypes.c_int32)]


class TraceStats(ctypes.Structure):
    _fields_ = [("records", ctypes.c_int32), ("sms", ctypes.c_int32), ("begin_ns", ctypes.c_double),
                ("end_ns", ctypes.c_double), ("tail_idle_sm_ns", ctypes.c_double),
                ("tail_idle_frac", ctypes.c_double)]


TRACE_ATTENTION, TRACE_REDUCTION, TRACE_CHUNK, TRACE_MLA_ITEM, TRACE_PAIR = 0, 1, 2, 3, 4
TRACE_DTYPE = np.dtype([("start_ns", "<u8"), ("end_ns", "<u8"), ("id", "<i4"), ("sm", "<i4"), ("kind", "<i4"),
                        ("cta", "<i4")])


class SeqModel(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int32), ("tasks_per_split", ctypes.c_int32),
                ("vectors", ctypes.c_int32), ("q_len", ctypes.c_int32)]


class ModelParams(ctypes.Structure):
    _fields_ = [
        ("num_ctas", ctypes.c_int32), ("warps_per_cta", ctypes.c_int32),
        ("q_heads", ctypes.c_int32), ("decode_qlen_max", ctypes.c_int32),
        ("rho", ctypes.c_double), ("delta_attn", ctypes.c_double),
        ("delta_red", ctypes.c_double), ("gamma", ctypes.c_double),
        ("adopt_margin", ctypes.c_double),
    ]


class KernelTime(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int32), ("pad", ctypes.c_int32), ("total_ms", ctypes.c_double)]


# splitkv_kv_rows and splitkv_verify, packed as bytes for each call (a fifth of the host time of
# filling a ctypes.Structure)
_KV_ROWS = struct.Struct("@PPqqqqii")
_VERIFY = struct.Struct("@iiiiPPPPqqPPPPPP")


class LatentLayer(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("w_kv_b", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse_out", ctypes.c_void_p)]


# splitkv_kernel ids, in order
KERNEL_NAMES = ["generic_partial_kernel", "gqa_engine_kernel", "mla_partial_kernel", "chunk_tc_kernel",
                "merge_states_kernel", "chunk_value_convert_kernel", "pair_tc_kernel", "mla_latent_convert_kernel",
                "kv_append_kernel", "kv_gather_kernel", "verify_drafts_kernel", "latent_rows_kernel", "latent_expand_kernel",
                "latent_attention_kernel", "latent_absorb_kernel", "latent_project_kernel"]

# name -> (restype, argtypes); this list mirrors include/splitkv.h
_vp, _i32, _i64, _dp = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_double)
_ip = ctypes.POINTER(ctypes.c_int32)
SIGNATURES = {
    "splitkv_plan_params_default": (None, [ctypes.POINTER(PlanParams)]),
    "splitkv_plan": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(PlanParams),
                                    ctypes.POINTER(ctypes.c_void_p)]),
    "splitkv_plan_destroy": (None, [_vp]),
    "splitkv_plan_num_tasks": (_i32, [_vp]),
    "splitkv_plan_num_chunk_tasks": (_i32, [_vp]),
    "splitkv_plan_num_pair_tasks": (_i32, [_vp]),
    "splitkv_plan_chunk_requests": (ctypes.c_int, [_vp, _ip]),
    "splitkv_plan_num_states": (_i64, [_vp]),
    "splitkv_plan_num_rows": (_i32, [_vp]),
    "splitkv_plan_splits": (ctypes.c_int, [_vp, _ip]),
    "splitkv_plan_state_indptr": (ctypes.c_int, [_vp, _ip]),
    "splitkv_plan_split_ranges": (ctypes.c_int, [_vp, _i32, _ip]),
    "splitkv_plan_interleaved": (_i32, [_vp]),
    "splitkv_plan_partial_dtype": (_i32, [_vp]),
    "splitkv_plan_trace_records": (_i32, [_vp]),
    "splitkv_plan_overlap_ctas": (_i32, [_vp]),
    "splitkv_trace_read": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "splitkv_trace_tail_idle": (ctypes.c_int, [_vp, _i32, _i32, _i32, ctypes.POINTER(TraceStats)]),
    "splitkv_plan_scores": (ctypes.c_int, [_vp, _dp]),
    "splitkv_plan_kernel_path": (_i32, [_vp]),
    "splitkv_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "splitkv_plan_upload": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp]),
    "splitkv_partial": (ctypes.c_int, [ctypes.POINTER(Problem), _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]),
    "merge_states": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp]),
    "merge_states_typed": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp]),
    "splitkv_decode": (ctypes.c_int, [ctypes.POINTER(Problem), _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]),
    "splitkv_decode_static": (ctypes.c_int, [ctypes.POINTER(Problem), _vp, _vp, _vp, _vp, _vp]),
    "splitkv_kv_append": (ctypes.c_int, [_vp, _vp, _vp, _vp]),                  # structs packed per call
    "splitkv_kv_gather": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _vp, _vp]),  # (splitkv_kv_rows, splitkv_verify)
    "splitkv_latent_plan": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_void_p)]),
    "splitkv_latent_plan_destroy": (None, [_vp]),
    "splitkv_latent_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "splitkv_latent_plan_num_tasks": (_i32, [_vp]),
    "splitkv_latent_plan_splits": (ctypes.c_int, [_vp, _ip]),
    "splitkv_latent_upload": (ctypes.c_int, [_vp, _vp, ctypes.c_size_t, _vp]),
    "splitkv_latent_expanded": (ctypes.c_int, [ctypes.POINTER(Problem), _vp, ctypes.POINTER(LatentLayer), _vp,
                                               ctypes.c_size_t, _vp, _vp]),
    "splitkv_latent_absorb_query": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(LatentLayer), _vp, _vp, _vp]),
    "splitkv_latent_project": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(LatentLayer), _vp, _i32, _vp, _vp,
                                              _vp, _vp]),
    "splitkv_latent_prefers_expanded": (_i32, [ctypes.POINTER(Problem)]),
    "splitkv_verify_drafts": (ctypes.c_int, [_vp, _vp, _vp]),
    "splitkv_read_device_error": (ctypes.c_int, [_vp, _vp, _i32, _ip, _vp]),
    "splitkv_read_static_device_error": (ctypes.c_int, [_i32, _ip, _vp]),
    "splitkv_last_error_message": (ctypes.c_char_p, []),
    "splitkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "splitkv_abi_version": (_i32, []),
    "splitkv_model_simulate": (ctypes.c_int, [ctypes.POINTER(SeqModel), _i32, _ip,
                                              ctypes.POINTER(ModelParams), _dp, _dp]),
    "splitkv_model_plan": (ctypes.c_int, [ctypes.POINTER(SeqModel), _i32, ctypes.POINTER(ModelParams),
                                          _i32, _i32, _ip, _dp]),
    "splitkv_profile_begin": (ctypes.c_int, []),
    "splitkv_debug_set_inject": (ctypes.c_int, [_i32]),
    "splitkv_profile_end": (ctypes.c_int, [ctypes.POINTER(KernelTime)]),
}

_lock = threading.Lock()
_lib = None


def load() -> ctypes.CDLL:
    """Load libsplitkv.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"` "
                    "(there is no CPU fallback)")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            _lib = lib
    return _lib


def _check(status: int):
    if status != OK:
        msg = load().splitkv_last_error_message().decode(errors="replace")
        raise SplitKVError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> Optional[int]:
    """The raw handle of `stream`, of the current stream when None."""
    if stream is None:
        if not torch.cuda.is_initialized():
            if not torch.cuda.is_available():
                return None   # argument checks still run; no launch can follow
            torch.cuda.init()
        # the handle alone: a torch.cuda.Stream object costs 3 us a call on the host
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class AttentionProblem:
    """A batch of attention over a paged KV cache (``splitkv_problem``).

    Tensors are on the GPU: ``q`` [total_q, Hq, D_qk]; GQA ``k_cache``/``v_cache``
    [num_pages, Hkv, P, D]; MLA ``k_cache`` [num_pages, P, 576] with
    ``v_cache=None``; ``page_table`` int32 [B, max_pages]; ``seq_lens`` int32
    [B]; ``qo_indptr`` int32 [B+1].  Host copies of the lengths are taken once
    here (or passed in) for the planner.  K/V caches of dtype uint8 hold E4M3
    codes (an FP8 KV cache) whose values are code * ``k_scale`` / ``v_scale``.
    """

    def __init__(self, *, q: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                 page_table: torch.Tensor, seq_lens: torch.Tensor, qo_indptr: torch.Tensor,
                 num_q_heads: int, num_kv_heads: int, head_dim_qk: int, head_dim_v: int,
                 page_size: int, scale: float, kind: str = "gqa",
                 seq_lens_host: Optional[Sequence[int]] = None,
                 qo_indptr_host: Optional[Sequence[int]] = None,
                 k_scale: Optional[float] = None, v_scale: Optional[float] = None):
        self.q, self.k_cache, self.v_cache = q, k_cache, v_cache
        self.page_table, self.seq_lens, self.qo_indptr = page_table, seq_lens, qo_indptr
        for name, t in (("page_table", page_table), ("seq_lens", seq_lens), ("qo_indptr", qo_indptr)):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous int32 tensor")
        for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
            if t is not None and not t.is_contiguous():
                raise TypeError(f"{name} must be contiguous")
        if q.dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {q.dtype}")
        self.kv_fp8 = k_cache.dtype == torch.uint8
        if self.kv_fp8 != (k_scale is not None and v_scale is not None):
            raise TypeError("uint8 (E4M3) K/V caches come with k_scale and v_scale, other caches without")
        self.k_scale = float(k_scale) if self.kv_fp8 else 1.0
        self.v_scale = float(v_scale) if self.kv_fp8 else 1.0
        self.seq_lens_host = np.ascontiguousarray(
            seq_lens.cpu().numpy() if seq_lens_host is None else seq_lens_host, dtype=np.int32)
        self.qo_indptr_host = np.ascontiguousarray(
            qo_indptr.cpu().numpy() if qo_indptr_host is None else qo_indptr_host, dtype=np.int32)
        self.kind = kind
        self.dtype = _DTYPES[q.dtype]
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.head_dim_qk, self.head_dim_v = head_dim_qk, head_dim_v
        self.page_size, self.scale = page_size, scale
        self.batch = int(seq_lens.shape[0])
        self._s = Problem(
            kind=GQA if kind == "gqa" else MLA, dtype=self.dtype, batch=self.batch,
            num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim_qk=head_dim_qk,
            head_dim_v=head_dim_v, page_size=page_size, num_pages=int(k_cache.shape[0]),
            max_pages_per_req=int(page_table.shape[1]), scale=float(scale),
            q=q.data_ptr(), k_cache=k_cache.data_ptr(),
            v_cache=(v_cache.data_ptr() if v_cache is not None else None),
            page_table=page_table.data_ptr(), seq_lens=seq_lens.data_ptr(),
            qo_indptr=qo_indptr.data_ptr(), seq_lens_host=self.seq_lens_host.ctypes.data,
            qo_indptr_host=self.qo_indptr_host.ctypes.data, kv_fp8=int(self.kv_fp8),
            k_scale=self.k_scale, v_scale=self.v_scale, reserved0=0)
        self.address = ctypes.addressof(self._s)

    @property
    def total_q(self) -> int:
        return int(self.qo_indptr_host[-1])

    @property
    def num_rows(self) -> int:
        return self.total_q * self.num_q_heads


def plan_params(mode: str = "critical_wave", **kw) -> PlanParams:
    p = PlanParams()
    load().splitkv_plan_params_default(ctypes.byref(p))
    p.mode = PLAN_UNIFORM if mode == "uniform" else PLAN_CRITICAL_WAVE
    for k, v in kw.items():
        if not hasattr(p, k):
            raise TypeError(f"unknown plan parameter {k}")
        setattr(p, k, v)
    return p


class Plan:
    """Owner of a ``splitkv_plan_t`` (host-side split plan and task list)."""

    def __init__(self, handle: ctypes.c_void_p, problem: AttentionProblem):
        self._h = handle
        self.batch = problem.batch
        lib = load()
        self.num_tasks = int(lib.splitkv_plan_num_tasks(handle))
        self.num_chunk_tasks = int(lib.splitkv_plan_num_chunk_tasks(handle))
        self.num_pair_tasks = int(lib.splitkv_plan_num_pair_tasks(handle))
        self.num_states = int(lib.splitkv_plan_num_states(handle))
        self.num_rows = int(lib.splitkv_plan_num_rows(handle))
        self.workspace_bytes = int(lib.splitkv_workspace_bytes(handle))
        self.kernel_path = int(lib.splitkv_plan_kernel_path(handle))
        self.trace_records = int(lib.splitkv_plan_trace_records(handle))
        self.overlap_ctas = int(lib.splitkv_plan_overlap_ctas(handle))

    @property
    def handle(self):
        return self._h

    def splits(self) -> np.ndarray:
        out = np.zeros(self.batch, dtype=np.int32)
        _check(load().splitkv_plan_splits(self._h, out.ctypes.data_as(_ip)))
        return out

    def state_indptr(self) -> np.ndarray:
        out = np.zeros(self.num_rows + 1, dtype=np.int32)
        _check(load().splitkv_plan_state_indptr(self._h, out.ctypes.data_as(_ip)))
        return out

    def split_ranges(self, b: int) -> np.ndarray:
        n = int(self.splits()[b])
        out = np.zeros(2 * n, dtype=np.int32)
        _check(load().splitkv_plan_split_ranges(self._h, b, out.ctypes.data_as(_ip)))
        return out.reshape(n, 2)

    @property
    def partial_dtype(self):
        """torch dtype of the plan's partial outputs (float32, or bfloat16)."""
        return torch.bfloat16 if load().splitkv_plan_partial_dtype(self._h) == BF16 else torch.float32

    @property
    def interleaved(self) -> bool:
        """True when split r of each request holds its pages r, r + n, r + 2n, ..."""
        return bool(load().splitkv_plan_interleaved(self._h))

    def chunk_requests(self) -> np.ndarray:
        """Per request: 1 when it runs on the chunk-tile kernel, 2 on the paired-tile
        kernel, else 0."""
        out = np.zeros(self.batch, dtype=np.int32)
        _check(load().splitkv_plan_chunk_requests(self._h, out.ctypes.data_as(_ip)))
        return out

    def scores(self) -> np.ndarray:
        out = np.zeros(4, dtype=np.float64)
        _check(load().splitkv_plan_scores(self._h, out.ctypes.data_as(_dp)))
        return out

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.splitkv_plan_destroy(h)
            self._h = None


def splitkv_plan(problem: AttentionProblem, params: Optional[PlanParams] = None) -> Plan:
    h = ctypes.c_void_p()
    _check(load().splitkv_plan(ctypes.byref(problem._s), ctypes.byref(params) if params is not None else None,
                               ctypes.byref(h)))
    return Plan(h, problem)


def alloc_workspace(plan: Plan, device=None) -> torch.Tensor:
    """A device byte buffer of the plan's workspace size (256-byte aligned by the allocator)."""
    t = torch.empty(max(256, plan.workspace_bytes), dtype=torch.uint8, device=device or "cuda")
    if t.data_ptr() % 256:
        raise RuntimeError("workspace allocation is not 256-byte aligned")
    return t


def splitkv_plan_upload(plan: Plan, workspace: torch.Tensor, stream=None):
    _check(load().splitkv_plan_upload(plan.handle, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def splitkv_partial(problem: AttentionProblem, plan: Plan, workspace: torch.Tensor, o_part: torch.Tensor,
                    lse_part: torch.Tensor, dev_error_word: Optional[torch.Tensor] = None, stream=None):
    _check(load().splitkv_partial(ctypes.byref(problem._s), plan.handle, _ptr(workspace), workspace.numel(),
                                  _ptr(o_part), _ptr(lse_part), _ptr(dev_error_word), _stream_handle(stream)))


def merge_states(o_part: torch.Tensor, lse_part: torch.Tensor, state_indptr: torch.Tensor, out: torch.Tensor,
                 lse_out: Optional[torch.Tensor] = None, stream=None):
    """merge_states for float32 o_part; merge_states_typed for bfloat16 o_part."""
    rows = int(state_indptr.shape[0]) - 1
    dim = int(o_part.shape[-1])
    if o_part.dtype == torch.float32:
        _check(load().merge_states(_ptr(o_part), _ptr(lse_part), _ptr(state_indptr), rows, dim, _ptr(out),
                                   _DTYPES[out.dtype], _ptr(lse_out), _stream_handle(stream)))
    else:
        _check(load().merge_states_typed(_ptr(o_part), _DTYPES[o_part.dtype], _ptr(lse_part), _ptr(state_indptr),
                                         rows, dim, _ptr(out), _DTYPES[out.dtype], _ptr(lse_out),
                                         _stream_handle(stream)))


def splitkv_decode(problem: AttentionProblem, plan: Plan, workspace: torch.Tensor, out: torch.Tensor,
                   lse_out: Optional[torch.Tensor] = None, dev_error_word: Optional[torch.Tensor] = None,
                   stream=None):
    _check(load().splitkv_decode(ctypes.byref(problem._s), plan.handle, _ptr(workspace), workspace.numel(),
                                 _ptr(out), _ptr(lse_out), _ptr(dev_error_word), _stream_handle(stream)))


def splitkv_decode_static(problem: AttentionProblem, plan: Plan, out: torch.Tensor,
                          lse_out: Optional[torch.Tensor] = None, dev_error_word: Optional[torch.Tensor] = None,
                          stream=None):
    """splitkv_decode for callers that cannot allocate device memory: the
    scratch is the library's own static device array (see include/splitkv.h)."""
    _check(load().splitkv_decode_static(ctypes.byref(problem._s), plan.handle, _ptr(out), _ptr(lse_out),
                                        _ptr(dev_error_word), _stream_handle(stream)))


def _kv_part(name: str, t: torch.Tensor, shape: tuple, dtype):
    """(token stride, head stride) of row tensor t, checked."""
    if t.shape != shape:
        raise TypeError(f"{name} rows have shape {tuple(t.shape)}, expected {shape}")
    if t.dtype is not dtype or dtype not in _DTYPES:
        raise TypeError("k and v rows differ in dtype" if t.dtype is not dtype else f"unsupported row dtype {dtype}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and shape[0] > 0:
        raise TypeError(f"the last axis of {name} rows must be contiguous")
    # (strides of axes of length 1 mean nothing)
    return st[0] if shape[0] > 1 else 0, st[1] if len(shape) == 3 and shape[1] > 1 else 0


def _kv_rows(problem: AttentionProblem, rows: int, k: torch.Tensor, v: Optional[torch.Tensor]) -> bytes:
    """The ``splitkv_kv_rows`` of row tensors: GQA [rows, Hkv, D] each; MLA [rows, 512]
    and [rows, 64], or [rows, 576] alone.  Any strides but a contiguous last axis."""
    dt = k.dtype
    if problem.kind == "gqa":
        if v is None:
            raise TypeError("a GQA cache takes key and value rows")
        shape = vshape = (rows, problem.num_kv_heads, problem.head_dim_qk)
    elif v is None:
        shape = (rows, problem.head_dim_qk)
    else:
        shape, vshape = (rows, problem.head_dim_v), (rows, problem.head_dim_qk - problem.head_dim_v)
    kt, kh = _kv_part("k", k, shape, dt)
    if v is None:
        return _KV_ROWS.pack(k.data_ptr(), 0, kt, kh, 0, 0, _DTYPES[dt], 0)
    vt, vh = _kv_part("v", v, vshape, dt)
    return _KV_ROWS.pack(k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, _DTYPES[dt], 0)


def kv_append(problem: AttentionProblem, k_new: torch.Tensor, v_new: Optional[torch.Tensor] = None,
              dev_error_word: Optional[torch.Tensor] = None, stream=None):
    """splitkv_kv_append: write the rows of the batch's new tokens (row qo_indptr[b] + i is
    the i-th of request b's last q_len tokens) into the problem's paged cache, quantised
    when the cache is E4M3.  GQA: k_new, v_new [total_q, Hkv, D]; MLA: k_new the latent
    columns [total_q, 512] and v_new the rotary columns [total_q, 64], or k_new
    [total_q, 576] alone.  float32 or bfloat16, any token and head strides."""
    rows = _kv_rows(problem, problem.total_q, k_new, v_new)
    st = (_lib or load()).splitkv_kv_append(problem.address, rows, _ptr(dev_error_word), _stream_handle(stream))
    if st:
        _check(st)


def kv_gather(problem: AttentionProblem, kv_indptr: torch.Tensor, k_out: torch.Tensor,
              v_out: Optional[torch.Tensor] = None, kv_begin: Optional[torch.Tensor] = None,
              dev_error_word: Optional[torch.Tensor] = None, stream=None):
    """splitkv_kv_gather: rows kv_indptr[b] .. kv_indptr[b+1]-1 of k_out / v_out become the
    (dequantised) cached tokens kv_begin[b] (0 without it) and following of request b.
    Shapes as kv_append's, over the rows of k_out; kv_indptr, kv_begin device int32."""
    _check_array("kv_indptr", kv_indptr, problem.batch + 1, torch.int32)
    if kv_begin is not None:
        _check_array("kv_begin", kv_begin, problem.batch, torch.int32)
    n = k_out.shape[0]
    rows = _kv_rows(problem, n, k_out, v_out)
    st = (_lib or load()).splitkv_kv_gather(problem.address, kv_indptr.data_ptr(), _ptr(kv_begin), n, rows,
                                            _ptr(dev_error_word), _stream_handle(stream))
    if st:
        _check(st)


def _check_array(name: str, t: torch.Tensor, n: int, dtype):
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() != n:
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of {n} entries")


class LatentPlan:
    """Owner of a ``splitkv_latent_plan_t`` (tasks and workspace of the expanded form)."""

    def __init__(self, problem: AttentionProblem):
        self._h = None
        h = ctypes.c_void_p()
        _check(load().splitkv_latent_plan(ctypes.byref(problem._s), ctypes.byref(h)))
        self._h = h
        self.batch = problem.batch
        self.num_tasks = int(load().splitkv_latent_plan_num_tasks(h))
        self.workspace_bytes = int(load().splitkv_latent_workspace_bytes(h))

    @property
    def handle(self):
        return self._h

    def splits(self) -> np.ndarray:
        out = np.zeros(self.batch, dtype=np.int32)
        _check(load().splitkv_latent_plan_splits(self._h, out.ctypes.data_as(_ip)))
        return out

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.splitkv_latent_plan_destroy(h)
            self._h = None


def latent_upload(plan: LatentPlan, workspace: torch.Tensor, stream=None):
    _check(load().splitkv_latent_upload(plan.handle, _ptr(workspace), workspace.numel(), _stream_handle(stream)))


def latent_layer(problem: AttentionProblem, q: Optional[torch.Tensor], w_kv_b: torch.Tensor, out: Optional[torch.Tensor],
                 lse: Optional[torch.Tensor] = None) -> LatentLayer:
    """The ``splitkv_latent_layer`` of q [total_q, H, 192] (any token stride that is a multiple of
    8), w_kv_b [H, 256, 512], out [total_q, H, 128], lse [total_q, H] float32; bfloat16 otherwise."""
    total, heads = problem.total_q, problem.num_q_heads
    for name, t, shape, dt in (("q", q, (total, heads, 192), torch.bfloat16), ("w_kv_b", w_kv_b, (heads, 256, 512), torch.bfloat16),
                               ("out", out, (total, heads, 128), torch.bfloat16), ("lse", lse, (total, heads), torch.float32)):
        if t is None:
            continue
        if t.dtype != dt or tuple(t.shape) != shape:
            raise TypeError(f"{name} must be {dt} of shape {shape}, got {t.dtype} {tuple(t.shape)}")
        if name == "q":
            if total > 0 and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != 192)):
                raise TypeError("the heads of a query token must be contiguous")
        elif not t.is_contiguous():
            raise TypeError(f"{name} must be contiguous")
    stride = heads * 192 if q is None or total <= 1 else q.stride(0)
    return LatentLayer(None if q is None else q.data_ptr(), stride, w_kv_b.data_ptr(), None if out is None else out.data_ptr(),
                       None if lse is None else lse.data_ptr())


def latent_expanded(problem: AttentionProblem, plan: LatentPlan, layer: LatentLayer, workspace: torch.Tensor,
                    dev_error_word: Optional[torch.Tensor] = None, stream=None):
    _check(load().splitkv_latent_expanded(ctypes.byref(problem._s), plan.handle, ctypes.byref(layer), _ptr(workspace),
                                          workspace.numel(), _ptr(dev_error_word), _stream_handle(stream)))


def latent_absorb_query(problem: AttentionProblem, layer: LatentLayer, q_abs: torch.Tensor,
                        dev_error_word: Optional[torch.Tensor] = None, stream=None):
    """splitkv_latent_absorb_query: q_abs [total_q, H, 576] bfloat16 from the layer's q."""
    _check_array("q_abs", q_abs, problem.total_q * problem.num_q_heads * 576, torch.bfloat16)
    _check(load().splitkv_latent_absorb_query(ctypes.byref(problem._s), ctypes.byref(layer), _ptr(q_abs),
                                              _ptr(dev_error_word), _stream_handle(stream)))


def latent_project(problem: AttentionProblem, layer: LatentLayer, o_part: torch.Tensor, lse_part: torch.Tensor,
                   state_indptr: torch.Tensor, dev_error_word: Optional[torch.Tensor] = None, stream=None):
    """splitkv_latent_project: merge o_part [num_states, 512] (float32 or bfloat16) and lse_part
    [num_states] by state_indptr [total_q * H + 1] int32 and project the rows to the layer's out."""
    if o_part.dtype not in _DTYPES:
        raise TypeError(f"unsupported o_part dtype {o_part.dtype}")
    _check_array("o_part", o_part, o_part.shape[0] * 512, o_part.dtype)
    _check_array("lse_part", lse_part, o_part.shape[0], torch.float32)
    _check_array("state_indptr", state_indptr, problem.total_q * problem.num_q_heads + 1, torch.int32)
    _check(load().splitkv_latent_project(ctypes.byref(problem._s), ctypes.byref(layer), _ptr(o_part), _DTYPES[o_part.dtype],
                                         _ptr(lse_part), _ptr(state_indptr), _ptr(dev_error_word), _stream_handle(stream)))


def latent_prefers_expanded(problem: AttentionProblem) -> bool:
    """Whether the expanded form is expected to be faster for the problem's lengths."""
    r = int(load().splitkv_latent_prefers_expanded(ctypes.byref(problem._s)))
    if r < 0:
        _check(ERR_INVALID_ARG)
    return bool(r)


def verify_drafts(tokens: torch.Tensor, qo_indptr: torch.Tensor, target_probs: torch.Tensor,
                  draft_probs: Optional[torch.Tensor], accept_u: torch.Tensor, sample_u: torch.Tensor,
                  out_tokens: Optional[torch.Tensor] = None, accepted: Optional[torch.Tensor] = None, *,
                  seq_lens: Optional[torch.Tensor] = None, seq_lens_out: Optional[torch.Tensor] = None,
                  dev_error_word: Optional[torch.Tensor] = None, stream=None):
    """splitkv_verify_drafts: accept drafted tokens against the target's probabilities and
    draw each request's next token.  Rows are the attention call's: tokens [total_q] int32
    (each request's last accepted token, then its drafts), target_probs and draft_probs
    [total_q, vocab] float32 (row r: the token after row r; draft_probs None: drafts
    proposed with certainty), accept_u [total_q], sample_u [batch].  With seq_lens the
    lengths without the refused drafts' slots go to seq_lens_out.  Returns (out_tokens,
    accepted)."""
    total, vocab, batch = tokens.shape[0], target_probs.shape[-1], qo_indptr.shape[0] - 1
    i32, f32 = torch.int32, torch.float32
    if out_tokens is None:
        out_tokens = torch.empty_like(tokens)
    if accepted is None:
        accepted = torch.empty(batch, dtype=i32, device=tokens.device)
    _check_array("tokens", tokens, total, i32)
    _check_array("qo_indptr", qo_indptr, batch + 1, i32)
    _check_array("accept_u", accept_u, total, f32)
    _check_array("sample_u", sample_u, batch, f32)
    _check_array("out_tokens", out_tokens, total, i32)
    _check_array("accepted", accepted, batch, i32)
    lens = lens_out = draft = 0
    if seq_lens is not None:
        _check_array("seq_lens", seq_lens, batch, i32)
        lens = seq_lens.data_ptr()
    if seq_lens_out is not None:
        _check_array("seq_lens_out", seq_lens_out, batch, i32)
        lens_out = seq_lens_out.data_ptr()
    target_stride = _check_probs(target_probs, total, vocab)
    draft_stride = vocab
    if draft_probs is not None:
        draft_stride = _check_probs(draft_probs, total, vocab)
        draft = draft_probs.data_ptr()
    v = _VERIFY.pack(batch, total, vocab, 0, qo_indptr.data_ptr(), tokens.data_ptr(), target_probs.data_ptr(), draft,
                     target_stride, draft_stride, accept_u.data_ptr(), sample_u.data_ptr(), lens, lens_out,
                     out_tokens.data_ptr(), accepted.data_ptr())
    st = (_lib or load()).splitkv_verify_drafts(v, _ptr(dev_error_word), _stream_handle(stream))
    if st:
        _check(st)
    return out_tokens, accepted


def _check_probs(t: torch.Tensor, total: int, vocab: int) -> int:
    """The row stride of probabilities t, checked."""
    if t.dtype is not torch.float32 or t.shape != (total, vocab):
        raise TypeError(f"probabilities must be float32 [{total}, {vocab}]")
    st = t.stride()
    if st[1] != 1 and vocab > 1 and total > 0:
        raise TypeError("probabilities must have contiguous rows")
    return st[0] if total > 1 else vocab


def read_device_error(dev_error_word: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      clear: bool = False, stream=None):
    """(status, raw word) of the device error word; synchronises the stream."""
    raw = ctypes.c_int32(0)
    st = load().splitkv_read_device_error(_ptr(dev_error_word), _ptr(workspace), 1 if clear else 0,
                                          ctypes.byref(raw), _stream_handle(stream))
    return st, raw.value


def read_static_device_error(clear: bool = False, stream=None):
    """(status, raw word) of the static array's error word (splitkv_decode_static
    calls made without an error word); synchronises the stream."""
    raw = ctypes.c_int32(0)
    st = load().splitkv_read_static_device_error(1 if clear else 0, ctypes.byref(raw), _stream_handle(stream))
    return st, raw.value


def trace_read(plan: Plan, workspace: torch.Tensor, stream=None) -> np.ndarray:
    """The plan's trace records from the workspace (structured numpy array with
    fields start_ns, end_ns, id, sm, kind, cta); synchronises the stream."""
    out = np.zeros(plan.trace_records, dtype=TRACE_DTYPE)
    _check(load().splitkv_trace_read(plan.handle, _ptr(workspace), workspace.numel(),
                                     ctypes.c_void_p(out.ctypes.data), _stream_handle(stream)))
    return out


def trace_tail_idle(records: np.ndarray, kinds=(TRACE_ATTENTION, TRACE_REDUCTION), num_sms: int = 0) -> dict:
    """Tail idle of the stage made of the records of the given kinds (LiquidCP
    Section 3: each SM's wait after its last task until the stage finishes,
    summed, over total SM-time)."""
    rec = np.ascontiguousarray(records, dtype=TRACE_DTYPE)
    mask = 0
    for k in kinds:
        mask |= 1 << int(k)
    st = TraceStats()
    _check(load().splitkv_trace_tail_idle(ctypes.c_void_p(rec.ctypes.data), len(rec), mask, num_sms,
                                          ctypes.byref(st)))
    return {f: getattr(st, f) for f, _ in TraceStats._fields_}


def _model_args(seqs, num_ctas, warps_per_cta, q_heads, rho, delta_attn, delta_red, gamma, adopt_margin,
                decode_qlen_max=16):
    arr = (SeqModel * len(seqs))()
    for i, s in enumerate(seqs):
        arr[i] = SeqModel(int(s[0]), int(s[1]), int(s[2]), int(s[3]))
    mp = ModelParams(num_ctas=num_ctas, warps_per_cta=warps_per_cta, q_heads=q_heads,
                     decode_qlen_max=decode_qlen_max, rho=rho, delta_attn=delta_attn, delta_red=delta_red,
                     gamma=gamma, adopt_margin=adopt_margin)
    return arr, mp


def model_simulate(seqs, splits, *, num_ctas, warps_per_cta=12, q_heads=1, rho=0.43, delta_attn=32.0,
                   delta_red=2.5, gamma=0.47, adopt_margin=0.10, decode_qlen_max=16):
    """(score, attention completion) of a split plan under the critical-wave
    model; ``seqs`` are (tiles, tasks_per_split, vectors, q_len) tuples."""
    arr, mp = _model_args(seqs, num_ctas, warps_per_cta, q_heads, rho, delta_attn, delta_red, gamma,
                          adopt_margin, decode_qlen_max)
    sp = np.ascontiguousarray(splits, dtype=np.int32)
    score, attn = ctypes.c_double(), ctypes.c_double()
    _check(load().splitkv_model_simulate(arr, len(seqs), sp.ctypes.data_as(_ip), ctypes.byref(mp),
                                         ctypes.byref(score), ctypes.byref(attn)))
    return score.value, attn.value


def model_plan(seqs, *, num_ctas, warps_per_cta=12, q_heads=1, rho=0.43, delta_attn=32.0, delta_red=2.5,
               gamma=0.47, adopt_margin=0.10, min_splits=1, max_splits=64, decode_qlen_max=16):
    """(splits, [base, chosen, search, reference] scores) from the planner."""
    arr, mp = _model_args(seqs, num_ctas, warps_per_cta, q_heads, rho, delta_attn, delta_red, gamma,
                          adopt_margin, decode_qlen_max)
    out = np.zeros(len(seqs), dtype=np.int32)
    sc = np.zeros(4, dtype=np.float64)
    _check(load().splitkv_model_plan(arr, len(seqs), ctypes.byref(mp), min_splits, max_splits,
                                     out.ctypes.data_as(_ip), sc.ctypes.data_as(_dp)))
    return out, sc


def profile_begin():
    """Start recording every kernel launch of the library (events on its stream)."""
    _check(load().splitkv_profile_begin())


def profile_end() -> dict:
    """Stop recording; {kernel name: (launches, total device ms)} for kernels that ran."""
    arr = (KernelTime * len(KERNEL_NAMES))()
    _check(load().splitkv_profile_end(arr))
    return {KERNEL_NAMES[k]: (int(arr[k].launches), float(arr[k].total_ms))
            for k in range(len(KERNEL_NAMES)) if arr[k].launches > 0}


def debug_set_inject(mode: int):
    """Test hook: 1 makes the persistent kernels withhold their tasks so their
    bounded waits expire (SPLITKV_ERR_TIMEOUT in the error word); 0 restores."""
    _check(load().splitkv_debug_set_inject(int(mode)))
