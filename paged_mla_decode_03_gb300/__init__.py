"""Batched paged MLA decode on GB300 (sm_103a): thin Python binding.

Every step of the computation runs in the CUDA kernels of ``libmla_decode.so``
behind the C ABI in ``include/mla_decode.h``; this module only marshals
arguments (torch tensors for device memory and streams) and caches plans.
There is no CPU fallback: if the library is missing, every call raises.

The high-level entry point mirrors the FlashInfer page
"prims_ts_batch_decode_with_kv_cache_mla" (signature): fixed
``[B, SQ, H, 576]`` or packed ``[total_q, H, 576]`` queries (``qo_indptr``),
a rank-3 or rank-4 paged cache, ``block_tables``/``seq_lens`` on the device,
caller-owned workspace, ``bmm1_scale``/``bmm2_scale``, causal or dense
masking, bf16 output and an optional natural-log LSE.  The cache is bf16, e4m3
or 4-bit; ``cache_append`` writes the newest tokens' rows (norm, rotation,
quantisation) and forms their query, ``cache_gather`` reads rows back, and
``rope_table`` makes the rotation table.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional, Tuple

import torch

__all__ = [
    "MLA_OK", "MlaDecodeError", "MlaDecodeParams", "load_library", "library_path",
    "mla_decode_plan", "mla_decode_run", "mla_decode_run_profiled", "mla_decode_run_dcp",
    "mla_decode_run_sparse", "mla_decode_destroy", "mla_decode_workspace_size",
    "mla_decode_status_offset", "mla_decode_status_string", "Plan", "decode",
    "HEAD_DIM_QK", "HEAD_DIM_V", "FP4_ROW_BYTES", "MlaCacheParams", "MlaRopeParams",
    "cache_append", "cache_gather", "rope_table",
]

HEAD_DIM_QK = 576
HEAD_DIM_V = 512
MLA_OK = 0
MLA_STATIC_WORKSPACE_BYTES = 48 * 1024 * 1024  # scratch of mla_decode_run_static_workspace
KV_BF16, KV_FP8_E4M3, KV_FP4_E2M1 = 0, 1, 2
KV_DTYPES = {"bf16": KV_BF16, "bfloat16": KV_BF16, torch.bfloat16: KV_BF16,
             "e4m3": KV_FP8_E4M3, "fp8": KV_FP8_E4M3, torch.float8_e4m3fn: KV_FP8_E4M3,
             "fp4": KV_FP4_E2M1, "e2m1": KV_FP4_E2M1}
FP4_ROW_BYTES = 324  # a 4-bit cache row: 288 bytes of e2m1 codes, 36 e4m3 scales
ROPE_STYLES = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "yarn": 2}
Q_BF16, Q_FP8_E4M3 = 0, 1
MASK_CAUSAL, MASK_DENSE = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmla_decode.so")
_lib = None


class MlaDecodeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {mla_decode_status_string(status)} ({status})")
        self.status = status


class MlaDecodeParams(ctypes.Structure):
    """Mirror of ``mla_decode_params`` (natural C alignment)."""
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("max_seq_len_q", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("packed", ctypes.c_int32),
        ("max_total_q", ctypes.c_int64),
        ("kv_dtype", ctypes.c_int32),
        ("mask", ctypes.c_int32),
        ("return_lse", ctypes.c_int32),
        ("device", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
        ("cp_world", ctypes.c_int32),
        ("cp_rank", ctypes.c_int32),
        ("sparse_top_k", ctypes.c_int32),
        ("e4m3_widen", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
    ]


class MlaCacheParams(ctypes.Structure):
    """Mirror of ``mla_cache_params`` (natural C alignment)."""
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("packed", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("num_heads", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32),
    ]


class MlaRopeParams(ctypes.Structure):
    """Mirror of ``mla_rope_params`` (natural C alignment)."""
    _fields_ = [
        ("max_position", ctypes.c_int32),
        ("scaling", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("amplitude", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_max_position", ctypes.c_double),
        ("beta_fast", ctypes.c_double),
        ("beta_slow", ctypes.c_double),
    ]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libmla_decode.so (built by ``paged_mla_decode_03_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                           "`python -m paged_mla_decode_03_gb300.build` (no fallback exists)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.mla_decode_plan.argtypes = [ctypes.POINTER(MlaDecodeParams), ctypes.POINTER(vp),
                                    ctypes.POINTER(sz)]
    lib.mla_decode_plan.restype = ctypes.c_int
    lib.mla_decode_run.argtypes = [vp, vp, vp, vp, vp, vp, i64, ctypes.c_float, ctypes.c_float,
                                   vp, vp, vp, sz, vp]
    lib.mla_decode_run.restype = ctypes.c_int
    lib.mla_decode_run_profiled.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, ctypes.c_float,
                                            ctypes.c_float, vp, vp, vp, sz, vp, vp, vp]
    lib.mla_decode_run_profiled.restype = ctypes.c_int
    lib.mla_decode_run_device_scales.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp,
                                                 sz, vp]
    lib.mla_decode_run_device_scales.restype = ctypes.c_int
    lib.mla_decode_host_staging_bytes.argtypes = [vp, i64]
    lib.mla_decode_host_staging_bytes.restype = sz
    lib.mla_decode_run_host.argtypes = [vp, vp, vp, vp, vp, vp, i64, ctypes.c_float,
                                        ctypes.c_float, vp, vp, vp, sz, vp, sz, vp]
    lib.mla_decode_run_host.restype = ctypes.c_int
    lib.mla_decode_run_dcp.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, ctypes.c_float,
                                       ctypes.c_float, vp, vp, vp, sz, vp]
    lib.mla_decode_run_dcp.restype = ctypes.c_int
    lib.mla_decode_run_sparse.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, ctypes.c_float,
                                          ctypes.c_float, vp, vp, vp, sz, vp]
    lib.mla_decode_run_sparse.restype = ctypes.c_int
    lib.mla_merge_states.argtypes = [vp, vp, i32, i64, ctypes.c_float, vp, vp, vp]
    lib.mla_merge_states.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.mla_rope_table.argtypes = [ctypes.POINTER(MlaRopeParams), vp, vp]
    lib.mla_rope_table.restype = ctypes.c_int
    lib.mla_cache_append.argtypes = [ctypes.POINTER(MlaCacheParams), vp, i64, vp, i64, vp, f32, vp,
                                     i32, i32, vp, vp, vp, vp, i64, f32, vp, vp, i64, i64, vp,
                                     i64, i64, f32, vp, vp, vp]
    lib.mla_cache_append.restype = ctypes.c_int
    lib.mla_cache_gather.argtypes = [ctypes.POINTER(MlaCacheParams), vp, vp, vp, vp, i64, f32, vp,
                                     vp, vp]
    lib.mla_cache_gather.restype = ctypes.c_int
    lib.mla_decode_destroy.argtypes = [vp]
    lib.mla_decode_destroy.restype = None
    lib.mla_decode_workspace_size.argtypes = [vp]
    lib.mla_decode_workspace_size.restype = sz
    lib.mla_decode_work_list_layout.argtypes = [vp, ctypes.POINTER(sz), ctypes.POINTER(sz),
                                                ctypes.POINTER(i32)]
    lib.mla_decode_work_list_layout.restype = ctypes.c_int
    lib.mla_decode_kernels_per_run.argtypes = [vp]
    lib.mla_decode_kernels_per_run.restype = i32
    lib.mla_decode_status_offset.argtypes = []
    lib.mla_decode_status_offset.restype = sz
    lib.mla_decode_status_string.argtypes = [ctypes.c_int]
    lib.mla_decode_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def mla_decode_status_string(status: int) -> str:
    return load_library().mla_decode_status_string(int(status)).decode()


def mla_decode_status_offset() -> int:
    return int(load_library().mla_decode_status_offset())


def mla_decode_plan(params: MlaDecodeParams) -> Tuple[int, int]:
    """-> (plan handle, workspace bytes).  Raises MlaDecodeError on failure."""
    lib = load_library()
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    rc = lib.mla_decode_plan(ctypes.byref(params), ctypes.byref(handle), ctypes.byref(ws))
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_plan")
    return handle.value, ws.value


def mla_decode_destroy(plan: Optional[int]) -> None:
    if plan:
        load_library().mla_decode_destroy(ctypes.c_void_p(plan))


def mla_decode_workspace_size(plan: int) -> int:
    return int(load_library().mla_decode_workspace_size(ctypes.c_void_p(plan)))


def mla_decode_work_list_layout(plan: int) -> Tuple[int, int, int]:
    """(items offset, worker-ranges offset, workers) of a plan's work list in
    the workspace (see include/mla_decode.h); for tests and tools."""
    a, b, n = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int32()
    rc = load_library().mla_decode_work_list_layout(ctypes.c_void_p(plan), ctypes.byref(a),
                                                    ctypes.byref(b), ctypes.byref(n))
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_work_list_layout")
    return a.value, b.value, n.value


def mla_decode_kernels_per_run(plan: int) -> int:
    """Kernels one run of the plan launches (see include/mla_decode.h)."""
    return int(load_library().mla_decode_kernels_per_run(ctypes.c_void_p(plan)))


def _nbytes(x) -> int:
    if x is None or isinstance(x, int):
        return 0
    return x.numel() * x.element_size()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def mla_decode_run(plan: int, query, kv_cache, block_tables, seq_lens, qo_indptr, total_q: int,
                   bmm1_scale: float, bmm2_scale: float, out, lse, workspace,
                   workspace_bytes: Optional[int] = None, stream=None) -> None:
    """Enqueue one decode (arguments: tensors or raw device pointers)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.mla_decode_run(ctypes.c_void_p(plan), _ptr(query), _ptr(kv_cache), _ptr(block_tables),
                            _ptr(seq_lens), _ptr(qo_indptr), int(total_q), float(bmm1_scale),
                            float(bmm2_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                            int(workspace_bytes), stream)
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_run")


def mla_decode_run_dcp(plan: int, query, kv_cache, block_tables, seq_lens, qo_indptr,
                       total_q: int, seq_lens_global, bmm1_scale: float, bmm2_scale: float,
                       out, lse, workspace, workspace_bytes: Optional[int] = None,
                       stream=None) -> None:
    """One decode-context-parallel rank's decode (``mla_decode_run_dcp``):
    ``seq_lens`` are the rank's local row counts, ``seq_lens_global`` the
    global KV lengths the causal bound is taken against (None for dense)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.mla_decode_run_dcp(ctypes.c_void_p(plan), _ptr(query), _ptr(kv_cache),
                                _ptr(block_tables), _ptr(seq_lens), _ptr(qo_indptr), int(total_q),
                                _ptr(seq_lens_global), float(bmm1_scale), float(bmm2_scale),
                                _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                stream)
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_run_dcp")


def mla_decode_run_sparse(plan: int, query, kv_cache, block_tables, seq_lens, qo_indptr,
                          total_q: int, sparse_indices, bmm1_scale: float, bmm2_scale: float,
                          out, lse, workspace, workspace_bytes: Optional[int] = None,
                          stream=None) -> None:
    """Sparse top-k decode (``mla_decode_run_sparse``): ``sparse_indices`` is
    an int32 CUDA tensor ``[tokens, k]`` of logical KV positions per query
    token; entries outside ``[0, seq_lens[b])`` are unused."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if isinstance(sparse_indices, torch.Tensor) and (
            sparse_indices.dtype != torch.int32 or not sparse_indices.is_cuda
            or not sparse_indices.is_contiguous()):
        raise TypeError("sparse_indices must be a contiguous int32 CUDA tensor")
    rc = lib.mla_decode_run_sparse(ctypes.c_void_p(plan), _ptr(query), _ptr(kv_cache),
                                   _ptr(block_tables), _ptr(seq_lens), _ptr(qo_indptr),
                                   int(total_q), _ptr(sparse_indices), float(bmm1_scale),
                                   float(bmm2_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                   int(workspace_bytes), stream)
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_run_sparse")


def mla_decode_host_staging_bytes(plan: int, total_q: int = 0) -> int:
    """Device staging bytes of ``mla_decode_run_host`` for one step."""
    return int(load_library().mla_decode_host_staging_bytes(ctypes.c_void_p(plan), int(total_q)))


def mla_decode_run_host(plan: int, h_query, kv_cache, h_block_tables, h_seq_lens, h_qo_indptr,
                        total_q: int, bmm1_scale: float, bmm2_scale: float, h_out, h_lse,
                        staging, workspace, staging_bytes: Optional[int] = None,
                        workspace_bytes: Optional[int] = None, stream=None) -> None:
    """Enqueue one decode whose query, metadata and results are host buffers
    (CPU tensors, ideally pinned); ``kv_cache``, ``staging`` and ``workspace``
    are device buffers.  The copies are enqueued on ``stream`` with the decode."""
    lib = load_library()
    if staging_bytes is None:
        staging_bytes = _nbytes(staging)
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = lib.mla_decode_run_host(ctypes.c_void_p(plan), _ptr(h_query), _ptr(kv_cache),
                                 _ptr(h_block_tables), _ptr(h_seq_lens), _ptr(h_qo_indptr),
                                 int(total_q), float(bmm1_scale), float(bmm2_scale), _ptr(h_out),
                                 _ptr(h_lse), _ptr(staging), int(staging_bytes), _ptr(workspace),
                                 int(workspace_bytes), stream)
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_run_host")


def mla_decode_run_device_scales(plan: int, query, kv_cache, block_tables, seq_lens, qo_indptr,
                                 total_q: int, bmm1_scale, bmm2_scale, out, lse, workspace,
                                 workspace_bytes: Optional[int] = None, stream=None) -> None:
    """``mla_decode_run`` with the two scales read from device memory at run
    time (``bmm1_scale`` / ``bmm2_scale``: one-element fp32 CUDA tensors or
    raw device pointers), so a captured graph sees new values at every replay."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    for t in (bmm1_scale, bmm2_scale):
        if isinstance(t, torch.Tensor) and (t.dtype != torch.float32 or not t.is_cuda
                                            or t.numel() != 1):
            raise TypeError("device scales must be one-element fp32 CUDA tensors")
    rc = lib.mla_decode_run_device_scales(
        ctypes.c_void_p(plan), _ptr(query), _ptr(kv_cache), _ptr(block_tables), _ptr(seq_lens),
        _ptr(qo_indptr), int(total_q), _ptr(bmm1_scale), _ptr(bmm2_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), int(workspace_bytes), stream)
    if rc != 0:
        raise MlaDecodeError(rc, "mla_decode_run_device_scales")


def mla_decode_run_profiled(plan: int, query, kv_cache, block_tables, seq_lens, qo_indptr,
                            total_q: int, bmm1_scale: float, bmm2_scale: float, out, lse,
                            workspace, workspace_bytes: Optional[int] = None, stream=None,
                            events=None, sparse_indices=None) -> None:
    """``mla_decode_run`` (``mla_decode_run_sparse`` with ``sparse_indices``)
    that also records ``events = (before, after)`` (torch.cuda.Event) around
    the decode kernel on the same stream."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    if stream is None:
        stream = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        raise TypeError("stream must be a torch.cuda.Stream")
    ev0 = ev1 = None
    if events is not None:
        # make sure the events exist (torch creates them lazily on first record)
        events[0].record(stream)
        events[1].record(stream)
        ev0, ev1 = events[0].cuda_event, events[1].cuda_event
    rc = lib.mla_decode_run_profiled(ctypes.c_void_p(plan), _ptr(query), _ptr(kv_cache),
                                     _ptr(block_tables), _ptr(seq_lens), _ptr(qo_indptr),
                                     int(total_q), _ptr(sparse_indices), float(bmm1_scale),
                                     float(bmm2_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                     int(workspace_bytes), stream.cuda_stream, ev0, ev1)
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_decode_run_profiled")


class Plan:
    """Owns one C plan; ``run`` enqueues a decode with it."""

    def __init__(self, *, batch: int, num_heads: int, max_seq_len_q: int, max_seq_len: int,
                 page_size: int, max_pages_per_req: int, num_pages: int, packed: bool,
                 max_total_q: int = 0, kv_dtype: str = "bf16", causal: bool = True,
                 return_lse: bool = False, device: int = 0, q_dtype: str = "bf16",
                 cp_world: int = 1, cp_rank: int = 0, sparse_top_k: int = 0,
                 e4m3_widen: bool = False, window: int = 0, sinks: int = 0):
        if kv_dtype not in KV_DTYPES:
            raise ValueError(f"kv_dtype must be one of {list(KV_DTYPES)}, got {kv_dtype!r}")
        for name, v in (("window", window), ("sinks", sinks)):
            if not -2 ** 31 <= v < 2 ** 31:  # (ctypes would cut it to its low 32 bits)
                raise ValueError(f"{name} = {v} does not fit 32 bits")
        self.params = MlaDecodeParams(
            batch=batch, num_heads=num_heads, max_seq_len_q=max_seq_len_q,
            max_seq_len=max_seq_len, page_size=page_size, max_pages_per_req=max_pages_per_req,
            num_pages=num_pages, packed=int(bool(packed)), max_total_q=max_total_q,
            kv_dtype=KV_DTYPES[kv_dtype],
            mask=MASK_CAUSAL if causal else MASK_DENSE, return_lse=int(bool(return_lse)),
            device=device,
            q_dtype=Q_FP8_E4M3 if q_dtype in ("e4m3", "fp8", torch.float8_e4m3fn) else Q_BF16,
            cp_world=cp_world, cp_rank=cp_rank, sparse_top_k=sparse_top_k,
            e4m3_widen=int(bool(e4m3_widen)), window=window, sinks=sinks)
        self.cp_world = cp_world
        self.sparse_top_k = sparse_top_k
        self.handle, self.workspace_bytes = mla_decode_plan(self.params)

    def run(self, query, kv_cache, block_tables, seq_lens, out, *, qo_indptr=None, total_q=0,
            lse=None, workspace=None, bmm1_scale=1.0, bmm2_scale=1.0, stream=None,
            seq_lens_global=None, sparse_indices=None):
        """Scales are Python floats, or one-element fp32 CUDA tensors (then both
        must be, and the kernels read them when they run).  A plan with
        ``cp_world`` > 1 runs one DCP rank's decode (``seq_lens_global``: the
        global KV lengths, required under causal masking); a plan with
        ``sparse_top_k`` > 0 a sparse top-k decode over ``sparse_indices``."""
        if self.sparse_top_k > 0:
            mla_decode_run_sparse(self.handle, query, kv_cache, block_tables, seq_lens,
                                  qo_indptr, total_q, sparse_indices, bmm1_scale, bmm2_scale,
                                  out, lse, workspace, None, stream)
            return
        if self.cp_world > 1:
            mla_decode_run_dcp(self.handle, query, kv_cache, block_tables, seq_lens, qo_indptr,
                               total_q, seq_lens_global, bmm1_scale, bmm2_scale, out, lse,
                               workspace, None, stream)
            return
        if isinstance(bmm1_scale, torch.Tensor) or isinstance(bmm2_scale, torch.Tensor):
            mla_decode_run_device_scales(self.handle, query, kv_cache, block_tables, seq_lens,
                                         qo_indptr, total_q, bmm1_scale, bmm2_scale, out, lse,
                                         workspace, None, stream)
            return
        mla_decode_run(self.handle, query, kv_cache, block_tables, seq_lens, qo_indptr, total_q,
                       bmm1_scale, bmm2_scale, out, lse, workspace, None, stream)

    def staging_bytes(self, total_q: int = 0) -> int:
        """Device staging bytes ``run_host`` needs for a step of ``total_q`` rows."""
        return mla_decode_host_staging_bytes(self.handle, total_q)

    def run_host(self, h_query, kv_cache, h_block_tables, h_seq_lens, h_out, *, staging,
                 workspace, h_qo_indptr=None, total_q=0, h_lse=None, bmm1_scale=1.0,
                 bmm2_scale=1.0, stream=None):
        """One step with host-side query, metadata and results (see
        ``mla_decode_run_host``); returns once the copies and kernels are enqueued."""
        for name, t in (("h_query", h_query), ("h_block_tables", h_block_tables),
                        ("h_seq_lens", h_seq_lens), ("h_out", h_out), ("h_qo_indptr", h_qo_indptr),
                        ("h_lse", h_lse)):
            if isinstance(t, torch.Tensor) and (t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous host tensor")
        mla_decode_run_host(self.handle, h_query, kv_cache, h_block_tables, h_seq_lens,
                            h_qo_indptr, total_q, bmm1_scale, bmm2_scale, h_out, h_lse, staging,
                            workspace, None, None, stream)

    def close(self):
        if self.handle:
            mla_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_plans: Dict[tuple, Plan] = {}


def decode(query: torch.Tensor, kv_cache: torch.Tensor, workspace_buffer: torch.Tensor,
           block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, *,
           qo_indptr: Optional[torch.Tensor] = None, max_seq_len_q: Optional[int] = None,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
           bmm1_scale=1.0, bmm2_scale=1.0, mask_type: str = "causal",
           return_lse: bool = False, cp_world: int = 1, cp_rank: int = 0,
           causal_seqlens_kv_global: Optional[torch.Tensor] = None,
           sparse_indices: Optional[torch.Tensor] = None, e4m3_widen: bool = False,
           window: int = 0, sinks: int = 0):
    """Paged MLA decode.  Returns ``out`` (and ``lse`` when ``return_lse``).

    ``query``: bf16 or float8_e4m3fn (quantised with a q_scale the caller folds
    into ``bmm1_scale``), ``[B, SQ, H, 576]`` (qo_indptr None) or ``[total_q, H, 576]``.
    ``kv_cache``: bf16 or float8_e4m3fn, ``[pages, page_size, 576]`` or
    ``[pages, 1, page_size, 576]``, or 4-bit, uint8 ``[pages, page_size, 324]``
    (``MLA_KV_FP4_E2M1`` in the header).  ``workspace_buffer`` must hold at least
    the plan's workspace bytes (see ``Plan``).  Plans are cached per static key.
    ``bmm1_scale`` / ``bmm2_scale``: floats, or one-element fp32 CUDA tensors the
    kernels read at run time (for scales that change between graph replays).
    ``cp_world`` / ``cp_rank`` / ``causal_seqlens_kv_global``: one rank of a
    decode-context-parallel decode (the vLLM FlashInferMLAImpl page's DCP
    keyword arguments); ``seq_lens`` are then the rank's local row counts.
    ``sparse_indices``: int32 ``[tokens, k]`` logical KV positions per query
    token (sparse top-k, ``sparse_mla_top_k`` = k); the listed positions in
    ``[0, seq_lens[b])`` replace the mask.
    ``e4m3_widen``: with an e4m3 cache, widen every e4m3 value exactly to bf16
    and multiply on bf16 tensor cores instead of the FP8 ones (see
    ``mla_decode_params.e4m3_widen`` in ``include/mla_decode.h``).
    ``window`` > 0: a query row sees the last ``window`` rows up to its bound, and
    the first ``sinks`` rows.  Over a 4-bit cache and with a window every tensor has to be
    contiguous, of its type and count and on the query's device (ValueError).
    """
    if query.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or not query.is_cuda:
        raise ValueError("query must be a bf16 or float8_e4m3fn CUDA tensor")
    q_dtype = "bf16" if query.dtype == torch.bfloat16 else "e4m3"
    kv_cache, kind = _cache_kind(kv_cache)
    kv_dtype = ("bf16", "e4m3", "fp4")[kind]
    if kind == KV_FP4_E2M1 or window:
        _check_decode(query, kv_cache, workspace_buffer, block_tables, seq_lens, qo_indptr, out,
                      lse if return_lse else None, causal_seqlens_kv_global)
    packed = qo_indptr is not None
    q_shape = query.shape
    H = q_shape[-2]
    B = seq_lens.shape[0]
    pages, page_size, _ = kv_cache.shape
    width = block_tables.shape[1]
    dev = query.get_device()
    if packed:
        if max_seq_len_q is None:
            raise ValueError("max_seq_len_q is required for packed launches")
        total_q = q_shape[0]
        sq = int(max_seq_len_q)
        out_shape = (total_q, H, HEAD_DIM_V)
        lse_shape = (total_q, H)
    else:
        total_q = 0
        sq = q_shape[1]
        out_shape = (B, sq, H, HEAD_DIM_V)
        lse_shape = (B * sq, H)
    causal = mask_type == "causal"
    if mask_type not in ("causal", "dense"):
        raise ValueError(mask_type)
    top_k = int(sparse_indices.shape[-1]) if sparse_indices is not None else 0
    key = (B, H, sq, int(max_seq_len), page_size, width, pages, packed, total_q, kv_dtype, causal,
           bool(return_lse), dev, q_dtype, int(cp_world), int(cp_rank), top_k, bool(e4m3_widen),
           int(window), int(sinks))
    plan = _plans.get(key)
    if plan is None:
        plan = Plan(batch=B, num_heads=H, max_seq_len_q=sq, max_seq_len=int(max_seq_len),
                    page_size=page_size, max_pages_per_req=width, num_pages=pages, packed=packed,
                    max_total_q=total_q, kv_dtype=kv_dtype, causal=causal, return_lse=return_lse,
                    device=dev, q_dtype=q_dtype, cp_world=int(cp_world),
                    cp_rank=int(cp_rank), sparse_top_k=top_k, e4m3_widen=e4m3_widen,
                    window=int(window), sinks=int(sinks))
        _plans[key] = plan
    if workspace_buffer.numel() * workspace_buffer.element_size() < plan.workspace_bytes:
        raise ValueError(f"workspace_buffer needs {plan.workspace_bytes} bytes")
    if out is None:
        out = torch.empty(out_shape, dtype=torch.bfloat16, device=query.device)
    if return_lse and lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=query.device)
    plan.run(query, kv_cache, block_tables, seq_lens, out, qo_indptr=qo_indptr, total_q=total_q,
             lse=lse if return_lse else None, workspace=workspace_buffer,
             bmm1_scale=bmm1_scale, bmm2_scale=bmm2_scale, stream=_raw_stream(dev),
             seq_lens_global=causal_seqlens_kv_global if causal else None,
             sparse_indices=sparse_indices)
    return (out, lse) if return_lse else out


def merge_states(o_parts: torch.Tensor, lse_parts: torch.Tensor, *, scale: float = 1.0,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 stream=None):
    """Merge partial attention states of the same rows by their natural-log
    LSEs (``mla_merge_states``): ``o_parts`` bf16 ``[n, ..., 512]``,
    ``lse_parts`` fp32 ``[n, ...]`` (the leading dims after ``n`` flattened to
    rows).  Returns ``(out, lse)`` with the parts' row shape; what the call makes belongs to
    ``stream`` (the current one), where the kernel runs."""
    if o_parts.dtype != torch.bfloat16 or lse_parts.dtype != torch.float32:
        raise TypeError("o_parts must be bf16 and lse_parts fp32")
    if not (o_parts.is_cuda and lse_parts.is_cuda):
        raise ValueError("merge_states runs on the GPU")
    n = int(o_parts.shape[0])
    row_shape = tuple(o_parts.shape[1:-1])
    if o_parts.shape[-1] != HEAD_DIM_V or tuple(lse_parts.shape) != (n,) + row_shape:
        raise ValueError("o_parts [n, ..., 512] and lse_parts [n, ...] disagree")
    rows = 1
    for d in row_shape:
        rows *= int(d)
    with _made_on(stream, o_parts.get_device()):
        o_parts = o_parts.contiguous()
        lse_parts = lse_parts.contiguous()
        if out is None:
            out = torch.empty(row_shape + (HEAD_DIM_V,), dtype=torch.bfloat16,
                              device=o_parts.device)
        if lse is None:
            lse = torch.empty(row_shape, dtype=torch.float32, device=o_parts.device)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = load_library().mla_merge_states(_ptr(o_parts), _ptr(lse_parts), n, rows, float(scale),
                                         _ptr(out), _ptr(lse), stream)
    if rc != 0:
        raise MlaDecodeError(rc, "mla_merge_states")
    return out, lse


def _cache_kind(kv_cache: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """The cache as [pages, page_size, row], and its KV_* type."""
    if kv_cache.dim() == 4:
        if kv_cache.shape[1] != 1:
            raise ValueError("rank-4 kv_cache must be [pages, 1, page_size, row]")
        kv_cache = kv_cache.squeeze(1)
    if kv_cache.dim() != 3:
        raise ValueError("kv_cache must be [pages, page_size, row]")
    row = kv_cache.shape[2]
    if kv_cache.dtype == torch.uint8 and row == FP4_ROW_BYTES:
        kind = KV_FP4_E2M1
    elif row != HEAD_DIM_QK:
        raise ValueError("kv_cache must be [pages, page_size, 576], or uint8 "
                         "[pages, page_size, 324] for 4 bits")
    elif kv_cache.dtype == torch.bfloat16:
        kind = KV_BF16
    elif kv_cache.dtype in (torch.float8_e4m3fn, torch.uint8):
        kind = KV_FP8_E4M3
    else:
        raise ValueError(f"unsupported kv_cache dtype {kv_cache.dtype}")
    return kv_cache, kind


# cache_append, cache_gather and decode run every layer of every step, so a call's
# checks are plain comparisons, and the message is worked out once one has failed.

def _is_int32(t: torch.Tensor, dev: int, shape) -> bool:
    return (t.dtype is torch.int32 and t.get_device() == dev and t.shape == shape
            and t.is_contiguous())


def _rows(name: str, t: torch.Tensor, dev: int, shape) -> Tuple[int, ...]:
    """The strides of a bf16 tensor of that shape with a contiguous last dim."""
    strides = t.stride()
    if not (t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == shape
            and (strides[-1] == 1 or t.numel() == 0)):
        _refuse(name, t, "a bf16 tensor with a contiguous last dim", dev, shape)
    return strides


def _refuse(name: str, t, what: str, dev: int, shape) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    raise ValueError(f"{name} must be {what} of shape {tuple(shape)} on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


_INT32 = "a contiguous int32 tensor"


def _stream_of(stream, dev: int) -> int:
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _made_on(stream, dev: int):
    """A context whose allocations and copies belong to ``stream``, where a call that was
    given one runs: memory of the current stream may still be in use there, and would be
    given away while the kernel writes it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(stream, device=torch.device("cuda", dev)) if stream > 1
                  else torch.cuda.default_stream(dev))  # (0 and 1: the legacy default stream)
    return torch.cuda.stream(stream)


try:  # the same handle without the Stream object around it (a microsecond and a half less)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:  # pragma: no cover - a torch without CUDA
    def _raw_stream(dev: int) -> int:
        return torch.cuda.current_stream(dev).cuda_stream


_cache_params: Dict[tuple, MlaCacheParams] = {}


def _params_of(*key) -> MlaCacheParams:
    """The parameter record of a static key (fields in order), made once."""
    p = _cache_params.get(key)
    if p is None:
        if len(_cache_params) >= 1024:
            _cache_params.clear()
        p = _cache_params[key] = MlaCacheParams(*key)
    return p


def _check_decode(query, kv_cache, workspace, block_tables, seq_lens, qo_indptr, out, lse,
                  global_lens) -> None:
    """What ``decode`` asks of its tensors over a 4-bit cache or with a window: the kernels
    take their types, counts and strides for granted."""
    dev = query.get_device()
    packed = qo_indptr is not None
    shape = query.shape
    if not (len(shape) == (3 if packed else 4) and shape[-1] == HEAD_DIM_QK
            and query.is_contiguous()):
        _refuse("query", query, "a contiguous tensor", dev,
                ("tokens", "heads", 576) if packed else ("batch", "tokens", "heads", 576))
    if kv_cache.get_device() != dev or not kv_cache.is_contiguous():
        _refuse("kv_cache", kv_cache, "a contiguous tensor", dev, kv_cache.shape)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("workspace_buffer", workspace, "a contiguous tensor", dev, workspace.shape)
    batch = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    if batch < 0 or not _is_int32(seq_lens, dev, (batch,)):
        _refuse("seq_lens", seq_lens, _INT32, dev, ("batch",))
    if not packed and shape[0] != batch:
        raise ValueError(f"query holds {shape[0]} requests, seq_lens {batch}")
    if block_tables.dim() != 2 or not _is_int32(block_tables, dev, (batch, block_tables.shape[1])):
        _refuse("block_tables", block_tables, _INT32, dev, (batch, "pages"))
    if packed and not _is_int32(qo_indptr, dev, (batch + 1,)):
        _refuse("qo_indptr", qo_indptr, _INT32, dev, (batch + 1,))
    if global_lens is not None and not _is_int32(global_lens, dev, (batch,)):
        _refuse("causal_seqlens_kv_global", global_lens, _INT32, dev, (batch,))
    rows = query.numel() // HEAD_DIM_QK
    if out is not None and not (out.dtype is torch.bfloat16 and out.get_device() == dev
                                and out.numel() == rows * HEAD_DIM_V and out.is_contiguous()):
        _refuse("out", out, "a contiguous bf16 tensor", dev, (*shape[:-1], HEAD_DIM_V))
    if lse is not None and not (lse.dtype is torch.float32 and lse.get_device() == dev
                                and lse.numel() == rows and lse.is_contiguous()):
        _refuse("lse", lse, "a contiguous fp32 tensor", dev, shape[:-1])


def _cache_call(kv_cache, block_tables, seq_lens, qo_indptr, q_len, total_q, status):
    """Checks that ``cache_append`` and ``cache_gather`` share -> (device, the
    parameters' first seven fields)."""
    dev = kv_cache.get_device()
    if dev < 0 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous CUDA tensor")
    kv_cache, kind = _cache_kind(kv_cache)
    pages, page_size, _ = kv_cache.shape
    batch = seq_lens.shape[0]
    if not _is_int32(seq_lens, dev, (batch,)):
        _refuse("seq_lens", seq_lens, _INT32, dev, (batch,))
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [batch, pages]")
    width = block_tables.shape[1]
    if not _is_int32(block_tables, dev, (batch, width)):
        _refuse("block_tables", block_tables, _INT32, dev, (batch, width))
    if (qo_indptr is None) == (q_len is None):
        raise ValueError("give qo_indptr (packed) or q_len (the same for every request)")
    if q_len is None:
        if not _is_int32(qo_indptr, dev, (batch + 1,)):
            _refuse("qo_indptr", qo_indptr, _INT32, dev, (batch + 1,))
    elif q_len < 1 or total_q != batch * q_len:
        raise ValueError(f"{total_q} tokens are not {batch} requests of {q_len}")
    if status is not None and not _is_int32(status, dev, (1,)):
        _refuse("status", status, _INT32, dev, (1,))
    return dev, (batch, int(q_len is None), q_len or 0, page_size, width, kind, pages)


def _call_on(dev: int, fn, *args) -> int:
    """``fn(*args)`` with ``dev`` current (the kernels launch on the current device)."""
    if torch.cuda.current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def rope_table(max_position: int, *, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original_max_position: int = 4096, beta_fast: float = 32.0,
               beta_slow: float = 1.0, amplitude: float = 1.0, device=None,
               stream=None) -> torch.Tensor:
    """The rotation table of ``cache_append`` (``mla_rope_table``): fp32
    ``[max_position, 64]``, 32 cosines then 32 sines per position, from angles in
    64 bits.  ``scaling``: None, ``"linear"`` (every frequency divided by
    ``factor``) or ``"yarn"`` (frequencies that turn fewer than ``beta_slow``
    times over ``original_max_position`` divided by ``factor``, those that turn
    more than ``beta_fast`` times kept, a linear blend between).  ``amplitude``
    multiplies cosines and sines.  The table is made on ``stream`` (the current one) and
    belongs to it."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}, got {scaling!r}")
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise ValueError("rope_table runs on the GPU")
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    p = MlaRopeParams(max_position=max_position, scaling=ROPE_SCALINGS[scaling], base=base,
                      amplitude=amplitude, factor=factor,
                      original_max_position=original_max_position, beta_fast=beta_fast,
                      beta_slow=beta_slow)
    with _made_on(stream, dev.index):
        table = torch.empty((max(max_position, 0), 64), dtype=torch.float32, device=dev)
    rc = _call_on(dev.index, load_library().mla_rope_table, ctypes.byref(p),
                  table.data_ptr() if max_position > 0 else 16, _stream_of(stream, dev.index))
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_rope_table")
    return table


def cache_append(latent: torch.Tensor, k_pe: torch.Tensor, kv_cache: torch.Tensor,
                 block_tables: torch.Tensor, seq_lens: torch.Tensor, *,
                 rope_table: torch.Tensor, norm_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, rope_style: str = "interleaved",
                 qo_indptr: Optional[torch.Tensor] = None, q_len: Optional[int] = None,
                 positions: Optional[torch.Tensor] = None, kv_scale: float = 1.0,
                 q_nope: Optional[torch.Tensor] = None, q_pe: Optional[torch.Tensor] = None,
                 query: Optional[torch.Tensor] = None, q_scale: float = 1.0,
                 status: Optional[torch.Tensor] = None, stream=None):
    """Norm, rotate, quantise and store the newest tokens' cache rows, and form
    their query rows in the same launch (``mla_cache_append``).

    ``latent`` bf16 ``[T, 512]`` and ``k_pe`` bf16 ``[T, 64]`` (row strides
    free): the tokens of all requests, ``q_len`` each or packed by
    ``qo_indptr``.  ``seq_lens`` already counts them: token i of a request of q
    tokens goes to position ``seq_lens[b] - q + i``.  ``kv_cache``: bf16, e4m3
    (``[pages, page_size, 576]``) or 4-bit (uint8 ``[pages, page_size, 324]``);
    its values are divided by ``kv_scale``.  ``norm_weight`` bf16 ``[512]``:
    RMS norm of the latent first (None: no norm).  ``q_pe`` bf16 ``[T, H, 64]``
    and ``q_nope`` bf16 ``[T, H, 512]`` (strides free) give ``query``
    ``[T, H, 576]`` (or ``[B, q_len, H, 576]``), made as bf16 when not given (rows
    of tokens without a place in the cache are zeros then, and stay as they were in a
    given one); an e4m3 one is divided by ``q_scale``; without ``q_nope`` only the RoPE dims
    of a given bf16 ``query`` are written.  ``status``: int32 ``[1]``, contract
    violations are ORed in (see ``include/mla_decode.h``).  Returns ``query``; one that the
    call makes belongs to ``stream`` (the current one), where the kernel runs."""
    if latent.dim() != 2 or not latent.is_cuda:
        raise ValueError("latent must be a CUDA tensor [tokens, 512]")
    T = latent.shape[0]
    dev, key = _cache_call(kv_cache, block_tables, seq_lens, qo_indptr, q_len, T, status)
    lat_row = _rows("latent", latent, dev, (T, 512))[0]
    pe_row = _rows("k_pe", k_pe, dev, (T, 64))[0]
    w_ptr = None
    if norm_weight is not None:
        _rows("norm_weight", norm_weight, dev, (512,))
        w_ptr = norm_weight.data_ptr()
    if not (rope_table.dtype is torch.float32 and rope_table.get_device() == dev
            and rope_table.dim() == 2 and rope_table.shape[1] == 64 and rope_table.is_contiguous()):
        _refuse("rope_table", rope_table, "a contiguous fp32 tensor", dev, ("positions", 64))
    style = ROPE_STYLES.get(rope_style)
    if style is None:
        raise ValueError(f"rope_style must be one of {list(ROPE_STYLES)}, got {rope_style!r}")
    if positions is not None and not _is_int32(positions, dev, (T,)):
        _refuse("positions", positions, _INT32, dev, (T,))
    H = q_dtype = 0
    n_ptr = p_ptr = q_ptr = None
    n_token = n_head = p_token = p_head = 0
    if q_pe is not None:
        if q_pe.dim() != 3:
            raise ValueError("q_pe must be [tokens, heads, 64]")
        H = q_pe.shape[1]
        p_token, p_head, _ = _rows("q_pe", q_pe, dev, (T, H, 64))
        if query is None:
            if q_nope is None:
                raise ValueError("without q_nope, query must be given (its latent part stays)")
            with _made_on(stream, dev):
                query = torch.zeros((T, H, HEAD_DIM_QK), dtype=torch.bfloat16,
                                    device=latent.device)
        if query.dtype is torch.float8_e4m3fn:
            q_dtype = Q_FP8_E4M3
        elif query.dtype is not torch.bfloat16:
            _refuse("query", query, "a contiguous bf16 or float8_e4m3fn tensor", dev, (T, H, 576))
        if query.get_device() != dev or not query.is_contiguous() or not (
                query.shape == (T, H, 576)
                or (q_len is not None and query.shape == (key[0], q_len, H, 576))):
            _refuse("query", query, "a contiguous bf16 or float8_e4m3fn tensor", dev, (T, H, 576))
        p_ptr, q_ptr = q_pe.data_ptr(), query.data_ptr()
        if q_nope is not None:
            n_token, n_head, _ = _rows("q_nope", q_nope, dev, (T, H, 512))
            n_ptr = q_nope.data_ptr()
    elif query is not None or q_nope is not None:
        raise ValueError("query and q_nope go with q_pe")
    if T == 1:  # the stride of a dim of one element is any number, and never applied
        lat_row = pe_row = n_token = p_token = 0
    rc = _call_on(
        dev, load_library().mla_cache_append, _params_of(*key, H, q_dtype), latent.data_ptr(),
        lat_row, k_pe.data_ptr(), pe_row, w_ptr, eps,
        rope_table.data_ptr(), rope_table.shape[0], style, _ptr(positions),
        block_tables.data_ptr(), seq_lens.data_ptr(), _ptr(qo_indptr), T, kv_scale,
        kv_cache.data_ptr(), n_ptr, n_token, n_head, p_ptr, p_token, p_head, q_scale, q_ptr,
        _ptr(status), _raw_stream(dev) if stream is None else _stream_of(stream, dev))
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_cache_append")
    return query


def cache_gather(kv_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, *,
                 total_q: Optional[int] = None, qo_indptr: Optional[torch.Tensor] = None,
                 q_len: Optional[int] = None, kv_scale: float = 1.0,
                 out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Cache rows as bf16 ``[total_q, 576]``, times ``kv_scale``
    (``mla_cache_gather``): the rows of each request's last ``q_len`` positions,
    or, packed by ``qo_indptr`` (then ``total_q`` or ``out`` is needed), of its
    last ``qo_indptr[b + 1] - qo_indptr[b]``; the running sum of ``seq_lens``
    reads whole sequences.  Rows of ``out`` that no position belongs to, or whose
    page id is bad (flagged in ``status``), stay as they were.  An ``out`` that the call
    makes has zeros there and belongs to ``stream`` (the current one), where the kernel runs."""
    if total_q is None:
        if out is not None:
            total_q = int(out.shape[0])
        elif q_len is not None:
            total_q = int(seq_lens.shape[0]) * q_len
        else:
            raise ValueError("total_q is needed for packed rows")
    dev, key = _cache_call(kv_cache, block_tables, seq_lens, qo_indptr, q_len, total_q, status)
    if out is None:
        with _made_on(stream, dev):
            out = torch.zeros((total_q, HEAD_DIM_QK), dtype=torch.bfloat16, device=kv_cache.device)
    elif not (out.dtype is torch.bfloat16 and out.get_device() == dev
              and out.shape == (total_q, HEAD_DIM_QK) and out.is_contiguous()):
        _refuse("out", out, "a contiguous bf16 tensor", dev, (total_q, HEAD_DIM_QK))
    rc = _call_on(dev, load_library().mla_cache_gather, _params_of(*key, 0, 0),
                  kv_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
                  _ptr(qo_indptr), total_q, kv_scale, out.data_ptr(), _ptr(status),
                  _raw_stream(dev) if stream is None else _stream_of(stream, dev))
    if rc != MLA_OK:
        raise MlaDecodeError(rc, "mla_cache_gather")
    return out


def dcp_gather(out: torch.Tensor, lse: torch.Tensor, group=None):
    """The exchange step of decode-context parallelism: all-gather this rank's
    partial state (``out`` [..., 512], ``lse`` [...]) over ``group`` (a
    torch.distributed process group; default the world) into stacked
    ``[world, ...]`` tensors, to be merged with ``merge_states``."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    outs = [torch.empty_like(out) for _ in range(world)]
    lses = [torch.empty_like(lse) for _ in range(world)]
    dist.all_gather(outs, out.contiguous(), group=group)
    dist.all_gather(lses, lse.contiguous(), group=group)
    return torch.stack(outs), torch.stack(lses)
