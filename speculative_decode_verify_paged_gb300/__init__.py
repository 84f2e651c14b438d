"""Block attention for speculative-decoding verify and draft over a paged KV cache, on GB300.

A thin ctypes binding over ``libspec_attn.so`` (C ABI in ``include/spec_attn.h``).
Every step of the computation runs in the library's CUDA kernels; this module
only marshals arguments: torch tensors are passed as device pointers and the
current torch CUDA stream is used unless another is given.  The calls around
the attention (step tables, norm and rotation, cross attention) go through a
small extension module (``csrc/binding.cpp``) with the same checks.  There is no CPU
path: if the library is missing, every call raises.

Names follow the C ABI::

    plan = spec_attn_plan_create(num_reqs=..., total_q_rows=..., max_w=..., ...,
                                 seq_lens=host_seq_lens, q_indptr=host_q_indptr)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    spec_attn_run(plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, ws)
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libspec_attn.so")

SPEC_ATTN_OK = 0
SPEC_ATTN_E_INVALID_ARG = -1
SPEC_ATTN_E_UNSUPPORTED = -2
SPEC_ATTN_E_WORKSPACE_TOO_SMALL = -3
SPEC_ATTN_E_CUDA = -4
SPEC_ATTN_E_DEVICE_CHECK = -5

SPEC_ATTN_MASK_CAUSAL_IN_BLOCK = 0
SPEC_ATTN_MASK_NON_CAUSAL = 1
SPEC_ATTN_KV_BF16 = 0
SPEC_ATTN_KV_NVFP4 = 1
SPEC_ATTN_MAX_W = 16
SPEC_ATTN_VARIANT_AUTO = 0
SPEC_ATTN_VARIANT_CUDA_CORE = 1
SPEC_ATTN_VARIANT_TCGEN05 = 2

SPEC_ATTN_DEV_BAD_PAGE = 0x1
SPEC_ATTN_DEV_BAD_SEQ_LEN = 0x2
SPEC_ATTN_DEV_BAD_WINDOW = 0x4
SPEC_ATTN_DEV_WAIT_TIMEOUT = 0x8
SPEC_ATTN_DEV_OUT_OF_PAGES = 0x10
SPEC_ATTN_DEV_BAD_FREE_LIST = 0x20
SPEC_ATTN_DEV_BAD_TREE = 0x40
SPEC_ATTN_TREE_MAX_W = 1024

# every symbol include/spec_attn.h declares
EXPORTED_SYMBOLS = (
    "spec_attn_plan_create", "spec_attn_plan_destroy", "spec_attn_plan_get_info",
    "spec_attn_run", "spec_attn_run_traced", "spec_attn_plan_set_timing_events",
    "spec_attn_reset_device_status", "spec_attn_check_device_status",
    "spec_attn_status_string", "spec_attn_last_cuda_error", "spec_attn_version",
    "spec_attn_run_noalloc", "spec_attn_noalloc_check_device_status", "spec_attn_append_kv",
    "spec_attn_run_append", "spec_attn_run_dense_block", "spec_attn_build_tables",
    "spec_attn_norm_rope_plan_create", "spec_attn_norm_rope_plan_destroy", "spec_attn_norm_rope",
    "spec_attn_norm_rope_append", "spec_attn_cross_plan_create", "spec_attn_cross_plan_destroy",
    "spec_attn_run_cross", "spec_attn_masked_plan_create", "spec_attn_masked_plan_destroy",
    "spec_attn_masked_plan_get_info", "spec_attn_masked_plan_set_test_stall", "spec_attn_run_masked",
    "spec_attn_build_tree", "spec_attn_accept_tree", "spec_attn_move_kv",
)


class SpecAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class spec_attn_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("total_q_rows", ctypes.c_int32), ("max_w", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("block_table_stride", ctypes.c_int32), ("mask_mode", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("max_seq_len", ctypes.c_int64),
        ("force_splits", ctypes.c_int32), ("kernel_variant", ctypes.c_int32),
        ("w_invariant", ctypes.c_int32), ("fixed_keys_per_split", ctypes.c_int32),
        ("window_left", ctypes.c_int32), ("kv_page_stride", ctypes.c_int64),
        ("scale_page_stride", ctypes.c_int64), ("dense_block_kv", ctypes.c_int32),
        ("early_metadata", ctypes.c_int32), ("test_stall", ctypes.c_int32),
        ("early_context_kv", ctypes.c_int32),
    ]


class spec_attn_plan_info(ctypes.Structure):
    _fields_ = [
        ("kernel_variant", ctypes.c_int32), ("keys_per_split", ctypes.c_int32),
        ("max_splits", ctypes.c_int32), ("row_groups", ctypes.c_int32),
        ("grid_x", ctypes.c_int32), ("grid_y", ctypes.c_int32), ("grid_z", ctypes.c_int32),
        ("block_threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
        ("uses_merge", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class spec_attn_tables_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("max_rows", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("block_table_stride", ctypes.c_int32), ("max_w", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int64),
    ]


class spec_attn_norm_rope_problem(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
        ("eps", ctypes.c_float), ("rot_scale", ctypes.c_float), ("q_row_stride", ctypes.c_int64),
        ("k_row_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64), ("q_out_row_stride", ctypes.c_int64),
        ("k_out_row_stride", ctypes.c_int64), ("kv_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("reserved", ctypes.c_int32), ("kv_page_stride", ctypes.c_int64),
        ("scale_page_stride", ctypes.c_int64),
    ]


class spec_attn_cross_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("total_q_rows", ctypes.c_int32), ("max_q_rows", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("total_kv_rows", ctypes.c_int32), ("max_kv_len", ctypes.c_int32), ("sm_scale", ctypes.c_float),
        ("force_splits", ctypes.c_int32), ("kv_row_stride", ctypes.c_int64),
    ]


class spec_attn_masked_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("total_q_rows", ctypes.c_int32), ("max_w", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("block_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("tree", ctypes.c_int32),
        ("window_left", ctypes.c_int32), ("sink_keys", ctypes.c_int32), ("mask_row_words", ctypes.c_int32),
        ("force_splits", ctypes.c_int32), ("max_seq_len", ctypes.c_int64), ("kv_page_stride", ctypes.c_int64),
        ("scale_page_stride", ctypes.c_int64),
    ]


class spec_attn_masked_plan_info(ctypes.Structure):
    _fields_ = [
        ("query_tiles", ctypes.c_int32), ("key_streams", ctypes.c_int32), ("ctas_per_sm", ctypes.c_int32),
        ("tiles_per_split", ctypes.c_int32), ("max_splits", ctypes.c_int32), ("join", ctypes.c_int32),
        ("longest_first", ctypes.c_int32), ("grid_x", ctypes.c_int32), ("grid_y", ctypes.c_int32),
        ("grid_z", ctypes.c_int32), ("block_threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
        ("num_sms", ctypes.c_int32), ("workspace_bytes", ctypes.c_size_t),
    ]


class spec_attn_tree_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("total_rows", ctypes.c_int32), ("max_w", ctypes.c_int32),
        ("mask_row_words", ctypes.c_int32), ("window_left", ctypes.c_int32), ("sink_keys", ctypes.c_int32),
        ("path_stride", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class spec_attn_move_problem(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("num_layers", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("block_table_stride", ctypes.c_int32), ("kv_dtype", ctypes.c_int32), ("path_stride", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("max_seq_len", ctypes.c_int64), ("kv_page_stride", ctypes.c_int64),
        ("scale_page_stride", ctypes.c_int64),
    ]


_lib = None
_lock = threading.Lock()


def load_library(path: Optional[str] = None):
    """Load libspec_attn.so (built by ``build.build()``); raise if it is absent."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libspec_attn.so not found at {p}; build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.spec_attn_plan_create.restype = i32
        lib.spec_attn_plan_create.argtypes = [ctypes.POINTER(spec_attn_problem), vp, vp,
                                              ctypes.POINTER(vp), ctypes.POINTER(sz)]
        lib.spec_attn_plan_destroy.restype = i32
        lib.spec_attn_plan_destroy.argtypes = [vp]
        lib.spec_attn_plan_get_info.restype = i32
        lib.spec_attn_plan_get_info.argtypes = [vp, ctypes.POINTER(spec_attn_plan_info)]
        run_args = [vp, vp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp, vp]
        lib.spec_attn_run.restype = i32
        lib.spec_attn_run.argtypes = run_args + [vp, sz, vp]
        lib.spec_attn_run_traced.restype = i32
        lib.spec_attn_run_traced.argtypes = run_args + [vp, vp, sz, vp]
        lib.spec_attn_plan_set_timing_events.restype = i32
        lib.spec_attn_plan_set_timing_events.argtypes = [vp, vp, vp]
        lib.spec_attn_reset_device_status.restype = i32
        lib.spec_attn_reset_device_status.argtypes = [vp, vp]
        lib.spec_attn_check_device_status.restype = i32
        lib.spec_attn_check_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.spec_attn_status_string.restype = ctypes.c_char_p
        lib.spec_attn_status_string.argtypes = [i32]
        lib.spec_attn_last_cuda_error.restype = i32
        lib.spec_attn_last_cuda_error.argtypes = []
        lib.spec_attn_version.restype = i32
        lib.spec_attn_version.argtypes = []
        lib.spec_attn_run_noalloc.restype = i32
        lib.spec_attn_run_noalloc.argtypes = run_args + [vp]
        lib.spec_attn_noalloc_check_device_status.restype = i32
        lib.spec_attn_noalloc_check_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        cache_args = [vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp, vp]
        lib.spec_attn_append_kv.restype = i32
        lib.spec_attn_append_kv.argtypes = [vp, vp, vp] + cache_args + [vp, sz, vp]
        lib.spec_attn_run_append.restype = i32
        lib.spec_attn_run_append.argtypes = [vp, vp, vp, vp] + cache_args + [vp, vp, vp, sz, vp]
        lib.spec_attn_run_dense_block.restype = i32
        lib.spec_attn_run_dense_block.argtypes = [vp] * 13 + [sz, vp]
        lib.spec_attn_build_tables.restype = i32
        lib.spec_attn_build_tables.argtypes = [ctypes.POINTER(spec_attn_tables_problem)] + [vp] * 12 + [sz, vp]
        lib.spec_attn_norm_rope_plan_create.restype = i32
        lib.spec_attn_norm_rope_plan_create.argtypes = [ctypes.POINTER(spec_attn_norm_rope_problem), vp, vp,
                                                        ctypes.POINTER(vp)]
        lib.spec_attn_norm_rope_plan_destroy.restype = i32
        lib.spec_attn_norm_rope_plan_destroy.argtypes = [vp]
        lib.spec_attn_norm_rope.restype = i32
        lib.spec_attn_norm_rope.argtypes = [vp, i32] + [vp] * 8
        lib.spec_attn_norm_rope_append.restype = i32
        lib.spec_attn_norm_rope_append.argtypes = ([vp, i32] + [vp] * 12 + [ctypes.c_float, ctypes.c_float, vp, sz, vp])
        lib.spec_attn_cross_plan_create.restype = i32
        lib.spec_attn_cross_plan_create.argtypes = [ctypes.POINTER(spec_attn_cross_problem), ctypes.POINTER(vp),
                                                    ctypes.POINTER(sz)]
        lib.spec_attn_cross_plan_destroy.restype = i32
        lib.spec_attn_cross_plan_destroy.argtypes = [vp]
        lib.spec_attn_run_cross.restype = i32
        lib.spec_attn_run_cross.argtypes = [vp] * 10 + [sz, vp]
        lib.spec_attn_masked_plan_create.restype = i32
        lib.spec_attn_masked_plan_create.argtypes = [ctypes.POINTER(spec_attn_masked_problem), ctypes.POINTER(vp),
                                                     ctypes.POINTER(sz)]
        lib.spec_attn_masked_plan_destroy.restype = i32
        lib.spec_attn_masked_plan_destroy.argtypes = [vp]
        lib.spec_attn_masked_plan_get_info.restype = i32
        lib.spec_attn_masked_plan_get_info.argtypes = [vp, ctypes.POINTER(spec_attn_masked_plan_info)]
        lib.spec_attn_masked_plan_set_test_stall.restype = i32
        lib.spec_attn_masked_plan_set_test_stall.argtypes = [vp, i32]
        lib.spec_attn_run_masked.restype = i32
        lib.spec_attn_run_masked.argtypes = [vp] * 6 + [ctypes.c_float, ctypes.c_float] + [vp] * 8 + [sz, vp]
        lib.spec_attn_build_tree.restype = i32
        lib.spec_attn_build_tree.argtypes = [ctypes.POINTER(spec_attn_tree_problem)] + [vp] * 6 + [sz, vp]
        lib.spec_attn_accept_tree.restype = i32
        lib.spec_attn_accept_tree.argtypes = [ctypes.POINTER(spec_attn_tree_problem)] + [vp] * 10 + [sz, vp]
        lib.spec_attn_move_kv.restype = i32
        lib.spec_attn_move_kv.argtypes = [ctypes.POINTER(spec_attn_move_problem)] + [vp] * 10 + [sz, vp]
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load_library().spec_attn_status_string(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(status: int, what: str):
    if status != SPEC_ATTN_OK:
        raise SpecAttnError(status, what)


def _host_i32(t):
    """Host int32 array (torch tensor / sequence) -> (ctypes pointer, keepalive)."""
    if t is None:
        return None, None
    import numpy as np
    if hasattr(t, "detach"):
        t = t.detach().cpu().numpy()
    a = np.ascontiguousarray(np.asarray(t, dtype=np.int32))
    return a.ctypes.data_as(ctypes.c_void_p), a


def _dptr(t, what, dtype=None, contiguous=True):
    """Device pointer of a CUDA tensor.  contiguous=False admits a view whose
    layout the plan describes (a pool with a page stride)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Plan:
    """Owns a spec_attn_plan* (destroyed with this object)."""

    def __init__(self, handle, workspace_bytes, problem):
        self._lib = load_library()
        self.handle = handle
        self.workspace_bytes = int(workspace_bytes)
        self.problem = problem
        info = spec_attn_plan_info()
        _check(self._lib.spec_attn_plan_get_info(handle, ctypes.byref(info)), "spec_attn_plan_get_info")
        self.info = {name: getattr(info, name) for name, _ in spec_attn_plan_info._fields_}

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None:
            try:
                self._lib.spec_attn_plan_destroy(h)
            except Exception:
                pass

    def set_timing_events(self, begin, end):
        b = None if begin is None else ctypes.c_void_p(begin.cuda_event)
        e = None if end is None else ctypes.c_void_p(end.cuda_event)
        _check(self._lib.spec_attn_plan_set_timing_events(self.handle, b, e),
               "spec_attn_plan_set_timing_events")


def spec_attn_plan_create(*, num_reqs, total_q_rows, max_w, num_q_heads, num_kv_heads, head_dim,
                          num_pages, block_table_stride, max_seq_len, mask_mode=0, kv_dtype=0,
                          page_size=16, sm_scale=0.0, force_splits=0, kernel_variant=0,
                          seq_lens=None, q_indptr=None, w_invariant=0, fixed_keys_per_split=0,
                          window_left=0, kv_page_stride=0, scale_page_stride=0, dense_block_kv=0,
                          early_metadata=0, test_stall=0, early_context_kv=0) -> Plan:
    lib = load_library()
    prob = spec_attn_problem(num_reqs, total_q_rows, max_w, num_q_heads, num_kv_heads, head_dim,
                             page_size, num_pages, block_table_stride, mask_mode, kv_dtype,
                             float(sm_scale), int(max_seq_len), force_splits, kernel_variant,
                             int(w_invariant), int(fixed_keys_per_split), int(window_left),
                             int(kv_page_stride), int(scale_page_stride), int(dense_block_kv),
                             int(early_metadata), int(test_stall), int(early_context_kv))
    sl, _k1 = _host_i32(seq_lens)
    qi, _k2 = _host_i32(q_indptr)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib.spec_attn_plan_create(ctypes.byref(prob), sl, qi, ctypes.byref(handle), ctypes.byref(ws)),
           "spec_attn_plan_create")
    return Plan(handle, ws.value, prob)


def _pool_ptrs(plan, k_pool, v_pool, k_scales, v_scales):
    """Pool pointers; a plan with a page stride takes strided views."""
    import torch
    fp4 = plan.problem.kv_dtype == SPEC_ATTN_KV_NVFP4
    dense = plan.problem.kv_page_stride == 0
    dense_sc = plan.problem.scale_page_stride == 0
    return [_dptr(k_pool, "k_pool", torch.uint8 if fp4 else torch.bfloat16, dense),
            _dptr(v_pool, "v_pool", torch.uint8 if fp4 else torch.bfloat16, dense),
            _dptr(k_scales, "k_scales", torch.uint8, dense_sc), _dptr(v_scales, "v_scales", torch.uint8, dense_sc)]


def _run_args(plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, k_scales, v_scales,
              k_gscale, v_gscale):
    import torch
    return [plan.handle,
            _dptr(q, "q", torch.bfloat16),
            *_pool_ptrs(plan, k_pool, v_pool, k_scales, v_scales),
            ctypes.c_float(k_gscale), ctypes.c_float(v_gscale),
            _dptr(block_table, "block_table", torch.int32), _dptr(seq_lens, "seq_lens", torch.int32),
            _dptr(q_indptr, "q_indptr", torch.int32), _dptr(o, "o", torch.bfloat16),
            _dptr(lse, "lse", torch.float32)]


def spec_attn_run(plan: Plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, workspace,
                  k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0, stream=None):
    """Launch one attention call (asynchronous).  Raises SpecAttnError on a bad status."""
    lib = load_library()
    args = _run_args(plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, k_scales,
                     v_scales, k_gscale, v_gscale)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.spec_attn_run(*args, _dptr(workspace, "workspace"), ctypes.c_size_t(ws_bytes),
                             _stream_handle(stream)), "spec_attn_run")


def spec_attn_run_traced(plan: Plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, trace,
                         workspace, k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0,
                         stream=None):
    import torch
    lib = load_library()
    args = _run_args(plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, k_scales,
                     v_scales, k_gscale, v_gscale)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.spec_attn_run_traced(*args, _dptr(trace, "trace", torch.int64), _dptr(workspace, "workspace"),
                                    ctypes.c_size_t(ws_bytes), _stream_handle(stream)),
           "spec_attn_run_traced")


def spec_attn_run_noalloc(plan: Plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse,
                          k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0, stream=None):
    """spec_attn_run for callers that cannot allocate device memory: the
    library's built-in scratch array stands in for the workspace (calls that
    may overlap on the GPU must be serialised by the caller)."""
    lib = load_library()
    args = _run_args(plan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse, k_scales,
                     v_scales, k_gscale, v_gscale)
    _check(lib.spec_attn_run_noalloc(*args, _stream_handle(stream)), "spec_attn_run_noalloc")


def spec_attn_noalloc_check_device_status(stream=None) -> int:
    """Device-status bits the last spec_attn_run_noalloc call on the current
    device left (and clear them); 0 means no device check tripped."""
    bits = ctypes.c_uint32()
    st = load_library().spec_attn_noalloc_check_device_status(_stream_handle(stream), ctypes.byref(bits))
    if st not in (SPEC_ATTN_OK, SPEC_ATTN_E_DEVICE_CHECK):
        _check(st, "spec_attn_noalloc_check_device_status")
    return int(bits.value)


def _cache_args(plan, k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale, block_table, seq_lens,
                q_indptr):
    import torch
    return [*_pool_ptrs(plan, k_pool, v_pool, k_scales, v_scales),
            ctypes.c_float(k_gscale), ctypes.c_float(v_gscale),
            _dptr(block_table, "block_table", torch.int32), _dptr(seq_lens, "seq_lens", torch.int32),
            _dptr(q_indptr, "q_indptr", torch.int32)]


def spec_attn_append_kv(plan: Plan, k_new, v_new, k_pool, v_pool, block_table, seq_lens, q_indptr, workspace,
                        k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0, stream=None):
    """Write the windows' new K/V rows ([total_rows, Hkv, d] bf16) into their
    cache slots, quantising for NVFP4 caches (asynchronous)."""
    import torch
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.spec_attn_append_kv(plan.handle, _dptr(k_new, "k_new", torch.bfloat16),
                                   _dptr(v_new, "v_new", torch.bfloat16),
                                   *_cache_args(plan, k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale,
                                                block_table, seq_lens, q_indptr),
                                   _dptr(workspace, "workspace"), ctypes.c_size_t(ws_bytes),
                                   _stream_handle(stream)), "spec_attn_append_kv")


def spec_attn_run_append(plan: Plan, q, k_new, v_new, k_pool, v_pool, block_table, seq_lens, q_indptr, o, lse,
                         workspace, k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0, stream=None):
    """KV append, then the attention call, on one stream (asynchronous)."""
    import torch
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.spec_attn_run_append(plan.handle, _dptr(q, "q", torch.bfloat16),
                                    _dptr(k_new, "k_new", torch.bfloat16), _dptr(v_new, "v_new", torch.bfloat16),
                                    *_cache_args(plan, k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale,
                                                 block_table, seq_lens, q_indptr),
                                    _dptr(o, "o", torch.bfloat16), _dptr(lse, "lse", torch.float32),
                                    _dptr(workspace, "workspace"), ctypes.c_size_t(ws_bytes),
                                    _stream_handle(stream)), "spec_attn_run_append")


def spec_attn_run_dense_block(plan: Plan, q, block_k, block_v, k_pool, v_pool, block_table, seq_lens, q_indptr,
                              o, lse, workspace, trace=None, stream=None):
    """Attention with the window's own keys from dense block tensors
    ([total_rows, Hkv, d] bf16) and the context from the cache (asynchronous)."""
    import torch
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size()
    dense = plan.problem.kv_page_stride == 0
    _check(lib.spec_attn_run_dense_block(
        plan.handle, _dptr(q, "q", torch.bfloat16), _dptr(block_k, "block_k", torch.bfloat16),
        _dptr(block_v, "block_v", torch.bfloat16), _dptr(k_pool, "k_pool", torch.bfloat16, dense),
        _dptr(v_pool, "v_pool", torch.bfloat16, dense), _dptr(block_table, "block_table", torch.int32),
        _dptr(seq_lens, "seq_lens", torch.int32), _dptr(q_indptr, "q_indptr", torch.int32),
        _dptr(o, "o", torch.bfloat16), _dptr(lse, "lse", torch.float32), _dptr(trace, "trace", torch.int64),
        _dptr(workspace, "workspace"), ctypes.c_size_t(ws_bytes), _stream_handle(stream)),
        "spec_attn_run_dense_block")


def spec_attn_reset_device_status(workspace, stream=None):
    _check(load_library().spec_attn_reset_device_status(_dptr(workspace, "workspace"),
                                                        _stream_handle(stream)),
           "spec_attn_reset_device_status")


def spec_attn_check_device_status(workspace, stream=None) -> int:
    """Return the device-status bits (and clear them); 0 means no device check tripped."""
    bits = ctypes.c_uint32()
    st = load_library().spec_attn_check_device_status(_dptr(workspace, "workspace"),
                                                      _stream_handle(stream), ctypes.byref(bits))
    if st not in (SPEC_ATTN_OK, SPEC_ATTN_E_DEVICE_CHECK):
        _check(st, "spec_attn_check_device_status")
    return int(bits.value)


def spec_attn_version() -> int:
    return load_library().spec_attn_version()


def spec_attn_last_cuda_error() -> int:
    return load_library().spec_attn_last_cuda_error()


# --------------------------------------------------------------------------- #
# Around the attention call: step tables, norm and rotation of q and k
# --------------------------------------------------------------------------- #
_calls = None


def _native():
    """The extension module that checks these calls' tensors and makes them."""
    global _calls
    if _calls is None:
        import importlib.machinery
        import importlib.util
        import torch  # noqa: F401  (the module uses the libraries that torch loads)
        load_library()
        path = os.path.join(HERE, "_build", "spec_attn_calls.so")
        if not os.path.exists(path):
            raise RuntimeError(f"spec_attn_calls.so not found at {path}; build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        loader = importlib.machinery.ExtensionFileLoader("spec_attn_calls", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("spec_attn_calls", loader))
        loader.exec_module(mod)
        _calls = mod
    return _calls


def spec_attn_build_tables(ctx_lens, window_lens, prev_seq_lens, prev_free_count, free_pages, block_table, seq_lens,
                           q_indptr, free_count, positions, slot_map, workspace, *, page_size=16, max_w=SPEC_ATTN_MAX_W,
                           max_seq_len, stream=None):
    """seq_lens, q_indptr, the grown block table and every row's position and
    cache slot from the requests' lengths (asynchronous).  seq_lens may be
    prev_seq_lens or ctx_lens, free_count may be prev_free_count."""
    _check((_calls or _native()).build_tables(
        (page_size, max_w, max_seq_len), ctx_lens, window_lens, prev_seq_lens, prev_free_count, free_pages, block_table,
        seq_lens, q_indptr, free_count, positions, slot_map, workspace, stream), "spec_attn_build_tables")


def rope_inv_freq(rot_dim: int, base: float = 10000.0):
    """The usual frequencies of rot_dim rotated elements: base^(-2 j / rot_dim)."""
    return [base ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)]


def rope_pair_axis(sections, interleaved: bool = False):
    """Axis of each rotated pair for ``sections`` pairs per axis: axis by axis,
    or (interleaved) the axes in turn while they have pairs left."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


class NormRopePlan:
    """Owns a spec_attn_norm_rope_plan* (destroyed with this object)."""

    def __init__(self, handle, problem):
        self._lib = load_library()
        self.handle = handle
        self.problem = problem
        p = problem
        # (in the order the native calls read them)
        self.spec = (handle.value, p.num_q_heads, p.num_kv_heads, p.head_dim, p.num_axes, p.q_row_stride, p.k_row_stride,
                     p.v_row_stride, p.q_out_row_stride, p.k_out_row_stride, p.kv_dtype, p.page_size, p.num_pages,
                     p.kv_page_stride, p.scale_page_stride)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None:
            try:
                self._lib.spec_attn_norm_rope_plan_destroy(h)
            except Exception:
                pass


def spec_attn_norm_rope_plan_create(*, num_q_heads, num_kv_heads, head_dim, inv_freq, rot_dim=None, pair_axis=None,
                                    num_axes=1, interleaved=0, eps=1e-6, rot_scale=1.0, q_row_stride=0,
                                    k_row_stride=0, v_row_stride=0, q_out_row_stride=0, k_out_row_stride=0,
                                    kv_dtype=0, page_size=0, num_pages=0, kv_page_stride=0,
                                    scale_page_stride=0) -> NormRopePlan:
    """``inv_freq``: rot_dim / 2 radians per position (a host sequence, doubles);
    ``pair_axis``: the position axis of each pair.  ``page_size`` and
    ``num_pages`` describe the cache that spec_attn_norm_rope_append writes."""
    rot_dim = head_dim if rot_dim is None else rot_dim
    freq = [float(x) for x in inv_freq]
    axis = None if pair_axis is None else [int(a) for a in pair_axis]
    if len(freq) != rot_dim // 2 or (axis is not None and len(axis) != rot_dim // 2):
        raise ValueError(f"inv_freq and pair_axis must have rot_dim / 2 = {rot_dim // 2} entries")
    if axis is not None and any(a < 0 or a > 255 for a in axis):
        raise ValueError("pair_axis entries must be position axes")
    prob = spec_attn_norm_rope_problem(
        num_q_heads, num_kv_heads, head_dim, rot_dim, int(interleaved), num_axes, float(eps), float(rot_scale),
        q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, k_out_row_stride, kv_dtype, page_size, num_pages,
        0, kv_page_stride, scale_page_stride)
    handle = ctypes.c_void_p()
    _check(load_library().spec_attn_norm_rope_plan_create(
        ctypes.byref(prob), (ctypes.c_double * max(1, len(freq)))(*freq),
        None if axis is None else (ctypes.c_uint8 * max(1, len(axis)))(*axis), ctypes.byref(handle)),
        "spec_attn_norm_rope_plan_create")
    return NormRopePlan(handle, prob)


def spec_attn_norm_rope(plan: NormRopePlan, q, k, q_weight, k_weight, positions, q_out, k_out, stream=None):
    """Norm and rotation of q [n, Hq, d] and k [n, Hkv, d] (asynchronous).
    ``positions`` [num_axes, n] int32; weights [d] fp32 or None (no norm);
    the outputs may be the inputs."""
    _check((_calls or _native()).norm_rope(plan.spec, q, k, q_weight, k_weight, positions, q_out, k_out, stream),
           "spec_attn_norm_rope")


def spec_attn_norm_rope_append(plan: NormRopePlan, q, k, v, q_weight, k_weight, positions, slot_map, q_out, k_pool,
                               v_pool, workspace, k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0,
                               stream=None):
    """spec_attn_norm_rope with K and V written into the cache slots that
    ``slot_map`` [n] int64 names (asynchronous); rows with a negative slot are skipped."""
    _check((_calls or _native()).norm_rope_append(
        plan.spec, q, k, v, q_weight, k_weight, positions, slot_map, q_out, k_pool, v_pool, workspace, k_scales, v_scales,
        k_gscale, v_gscale, stream), "spec_attn_norm_rope_append")


class CrossPlan:
    """Owns a spec_attn_cross_plan* (destroyed with this object)."""

    def __init__(self, handle, workspace_bytes, problem):
        self._lib = load_library()
        self.handle = handle
        self.workspace_bytes = int(workspace_bytes)
        self.problem = problem
        p = problem
        self.spec = (handle.value, p.num_reqs, p.total_q_rows, p.num_q_heads, p.num_kv_heads, p.head_dim,
                     p.total_kv_rows, p.kv_row_stride)   # (in the order the native call reads them)

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None:
            try:
                self._lib.spec_attn_cross_plan_destroy(h)
            except Exception:
                pass


def spec_attn_cross_plan_create(*, num_reqs, total_q_rows, max_q_rows, num_q_heads, num_kv_heads, head_dim,
                                total_kv_rows, max_kv_len, sm_scale=0.0, force_splits=0, kv_row_stride=0) -> CrossPlan:
    prob = spec_attn_cross_problem(num_reqs, total_q_rows, max_q_rows, num_q_heads, num_kv_heads, head_dim,
                                   total_kv_rows, max_kv_len, float(sm_scale), force_splits, kv_row_stride)
    handle, ws = ctypes.c_void_p(), ctypes.c_size_t()
    _check(load_library().spec_attn_cross_plan_create(ctypes.byref(prob), ctypes.byref(handle), ctypes.byref(ws)),
           "spec_attn_cross_plan_create")
    return CrossPlan(handle, ws.value, prob)


def spec_attn_run_cross(plan: CrossPlan, q, k, v, q_indptr, kv_start, kv_len, o, lse, workspace, stream=None):
    """Attention of each request's query rows to its range of state rows
    (asynchronous).  ``lse`` may be None."""
    _check((_calls or _native()).run_cross(plan.spec, q, k, v, q_indptr, kv_start, kv_len, o, lse, workspace, stream),
           "spec_attn_run_cross")


# --------------------------------------------------------------------------- #
# Drafted trees, and windows with sinks
# --------------------------------------------------------------------------- #
class MaskedPlan:
    """Owns a spec_attn_masked_plan* (destroyed with this object)."""

    def __init__(self, handle, workspace_bytes, problem):
        self._lib = load_library()
        self.handle = handle
        self.workspace_bytes = int(workspace_bytes)
        self.problem = problem
        p = problem
        # (in the order the native call reads them)
        self.spec = (handle.value, p.num_reqs, p.total_q_rows, p.num_q_heads, p.num_kv_heads, p.head_dim, p.num_pages,
                     p.page_size, p.block_table_stride, p.kv_dtype, p.kv_page_stride, p.scale_page_stride, p.tree,
                     p.mask_row_words or -(-p.max_w // 32))

    @property
    def info(self):
        """What the plan decided (spec_attn_masked_plan_info), by name."""
        info = spec_attn_masked_plan_info()
        _check(self._lib.spec_attn_masked_plan_get_info(self.handle, ctypes.byref(info)),
               "spec_attn_masked_plan_get_info")
        return {name: getattr(info, name) for name, _ in spec_attn_masked_plan_info._fields_}

    def set_test_stall(self, stall):
        """Testing only: let the waits of this plan's calls run out."""
        _check(self._lib.spec_attn_masked_plan_set_test_stall(self.handle, int(stall)),
               "spec_attn_masked_plan_set_test_stall")

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h is not None:
            try:
                self._lib.spec_attn_masked_plan_destroy(h)
            except Exception:
                pass


def spec_attn_masked_plan_create(*, num_reqs, total_q_rows, max_w, num_q_heads, num_kv_heads, head_dim, num_pages,
                                 block_table_stride, max_seq_len, kv_dtype=0, page_size=16, sm_scale=0.0, tree=0,
                                 window_left=0, sink_keys=0, mask_row_words=0, force_splits=0, kv_page_stride=0,
                                 scale_page_stride=0) -> MaskedPlan:
    prob = spec_attn_masked_problem(num_reqs, total_q_rows, max_w, num_q_heads, num_kv_heads, head_dim, page_size,
                                    num_pages, block_table_stride, kv_dtype, float(sm_scale), int(tree), window_left,
                                    sink_keys, mask_row_words, force_splits, int(max_seq_len), int(kv_page_stride),
                                    int(scale_page_stride))
    # (ctypes drops the bits that a field does not hold: a window of 2^32 would be none)
    given = dict(num_reqs=num_reqs, total_q_rows=total_q_rows, max_w=max_w, num_q_heads=num_q_heads,
                 num_kv_heads=num_kv_heads, head_dim=head_dim, page_size=page_size, num_pages=num_pages,
                 block_table_stride=block_table_stride, kv_dtype=kv_dtype, tree=tree, window_left=window_left,
                 sink_keys=sink_keys, mask_row_words=mask_row_words, force_splits=force_splits, max_seq_len=max_seq_len,
                 kv_page_stride=kv_page_stride, scale_page_stride=scale_page_stride)
    if any(getattr(prob, name) != int(value) for name, value in given.items()):
        _check(SPEC_ATTN_E_UNSUPPORTED, "spec_attn_masked_plan_create")
    handle, ws = ctypes.c_void_p(), ctypes.c_size_t()
    _check(load_library().spec_attn_masked_plan_create(ctypes.byref(prob), ctypes.byref(handle), ctypes.byref(ws)),
           "spec_attn_masked_plan_create")
    return MaskedPlan(handle, ws.value, prob)


def spec_attn_run_masked(plan: MaskedPlan, q, k_pool, v_pool, block_table, seq_lens, q_indptr, row_mask, positions, o,
                         lse, workspace, k_scales=None, v_scales=None, k_gscale=1.0, v_gscale=1.0, stream=None):
    """Attention over the paged cache under tree masks, or under a sliding
    window with sinks (asynchronous).  ``row_mask`` [rows, words] int32 for
    trees, ``positions`` [rows] int32 for trees with a window; else None."""
    _check((_calls or _native()).run_masked(plan.spec, q, k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale,
                                            block_table, seq_lens, q_indptr, row_mask, positions, o, lse, workspace,
                                            stream), "spec_attn_run_masked")


def spec_attn_build_tree(parents, seq_lens, q_indptr, positions, row_mask, workspace, *, max_w, window_left=0,
                         sink_keys=0, stream=None):
    """Positions [rows] and ancestor masks [rows, words] int32 of every
    request's tree from its nodes' parents (asynchronous)."""
    _check((_calls or _native()).build_tree((max_w, window_left, sink_keys), parents, seq_lens, q_indptr, positions,
                                            row_mask, workspace, stream), "spec_attn_build_tree")


def spec_attn_accept_tree(parents, draft_tokens, target_tokens, seq_lens, q_indptr, path, accept_lens, next_tokens,
                          ctx_lens, workspace, *, max_w, stream=None):
    """The accepted path of every request's tree (asynchronous).  Tokens int64;
    ctx_lens may be seq_lens if the caller keeps a copy of those: the move and
    the next step's tables take the lengths as they were."""
    _check((_calls or _native()).accept_tree((max_w,), parents, draft_tokens, target_tokens, seq_lens, q_indptr, path,
                                             accept_lens, next_tokens, ctx_lens, workspace, stream),
           "spec_attn_accept_tree")


def spec_attn_move_kv(k_pools, v_pools, block_table, seq_lens, q_indptr, path, accept_lens, workspace, *, max_seq_len,
                      k_scales=None, v_scales=None, stream=None):
    """Move the accepted nodes' keys and values into place in every layer's
    cache (asynchronous).  Pools and scales: lists of one tensor [pages, Hkv,
    page_size, row] a layer; layers share shapes and strides.  ``seq_lens`` as
    spec_attn_accept_tree took them, window included, not the ctx_lens that it
    wrote: with those, accepted text would be overwritten."""
    _check((_calls or _native()).move_kv((max_seq_len,), k_pools, v_pools, k_scales, v_scales, block_table, seq_lens,
                                         q_indptr, path, accept_lens, workspace, stream), "spec_attn_move_kv")


# --------------------------------------------------------------------------- #
# Convenience: run a workload (from .workloads) that lives on the GPU
# --------------------------------------------------------------------------- #
class DeviceWorkload:
    """A workload's tensors moved to a CUDA device, plus output and workspace buffers."""

    def __init__(self, wl, device="cuda", force_splits=0, kernel_variant=0, host_lens=True, w_invariant=0,
                 fixed_keys_per_split=0, append_rows=None, mode="run", interleave=False, early_metadata=0,
                 early_context_kv=0):
        """``append_rows``: (k_new, v_new) [total_rows, Hkv, d] bf16 for the KV
        append.  ``mode``: what :meth:`run` launches -- "run" (attention),
        "run_append" (append, then attention) or "append" (the append alone).
        ``interleave``: K and V pages (and NVFP4 scale pages) share one
        allocation [num_pages, 2, Hkv, page_size, row], so the pools are views
        with a page stride of twice their dense page."""
        import torch
        assert mode in ("run", "run_append", "append")
        assert mode == "run" or append_rows is not None
        self.wl = wl
        self.mode = mode
        dev = torch.device(device)
        self.q = wl.q.to(dev)
        kv_stride = sc_stride = 0
        if interleave:
            both = torch.stack([wl.k_pool, wl.v_pool], 1).to(dev)          # [pages, 2, Hkv, ps, row]
            self.kv_storage = both
            self.k_pool, self.v_pool = both[:, 0], both[:, 1]
            kv_stride = both[0].numel() * both.element_size()
            self.k_scales = self.v_scales = None
            if wl.k_scales is not None:
                sboth = torch.stack([wl.k_scales, wl.v_scales], 1).to(dev)
                self.scale_storage = sboth
                self.k_scales, self.v_scales = sboth[:, 0], sboth[:, 1]
                sc_stride = sboth[0].numel()
        else:
            self.k_pool = wl.k_pool.to(dev)
            self.v_pool = wl.v_pool.to(dev)
            self.k_scales = None if wl.k_scales is None else wl.k_scales.to(dev)
            self.v_scales = None if wl.v_scales is None else wl.v_scales.to(dev)
        self.block_table = wl.block_table.to(dev)
        self.seq_lens = wl.seq_lens.to(dev)
        self.q_indptr = wl.q_indptr.to(dev)
        self.o = torch.zeros(wl.total_rows, wl.num_q_heads, wl.head_dim, dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros(wl.total_rows, wl.num_q_heads, dtype=torch.float32, device=dev)
        self.plan = spec_attn_plan_create(
            num_reqs=wl.num_reqs, total_q_rows=wl.total_rows, max_w=max(1, wl.max_w),
            num_q_heads=wl.num_q_heads, num_kv_heads=wl.num_kv_heads, head_dim=wl.head_dim,
            num_pages=wl.num_pages, block_table_stride=int(wl.block_table.shape[1]),
            max_seq_len=max(1, wl.max_seq_len), mask_mode=wl.mask_mode, kv_dtype=wl.kv_dtype,
            page_size=wl.page_size, sm_scale=wl.sm_scale, force_splits=force_splits,
            kernel_variant=kernel_variant, seq_lens=wl.seq_lens if host_lens else None,
            q_indptr=wl.q_indptr if host_lens else None, w_invariant=w_invariant,
            fixed_keys_per_split=fixed_keys_per_split, window_left=wl.window_left, kv_page_stride=kv_stride,
            scale_page_stride=sc_stride, dense_block_kv=int(wl.block_k is not None),
            early_metadata=early_metadata, early_context_kv=early_context_kv)
        self.workspace = torch.zeros(max(256, self.plan.workspace_bytes), dtype=torch.uint8, device=dev)
        self.block_k = None if wl.block_k is None else wl.block_k.to(dev)
        self.block_v = None if wl.block_v is None else wl.block_v.to(dev)
        self.k_new = self.v_new = None
        if append_rows is not None:
            self.k_new = append_rows[0].to(dev).contiguous()
            self.v_new = append_rows[1].to(dev).contiguous()

    def run(self, stream=None):
        if self.mode == "append":
            spec_attn_append_kv(self.plan, self.k_new, self.v_new, self.k_pool, self.v_pool, self.block_table,
                                self.seq_lens, self.q_indptr, self.workspace, self.k_scales, self.v_scales,
                                self.wl.k_gscale, self.wl.v_gscale, stream)
        elif self.mode == "run_append":
            spec_attn_run_append(self.plan, self.q, self.k_new, self.v_new, self.k_pool, self.v_pool,
                                 self.block_table, self.seq_lens, self.q_indptr, self.o, self.lse, self.workspace,
                                 self.k_scales, self.v_scales, self.wl.k_gscale, self.wl.v_gscale, stream)
        elif self.block_k is not None:
            spec_attn_run_dense_block(self.plan, self.q, self.block_k, self.block_v, self.k_pool, self.v_pool,
                                      self.block_table, self.seq_lens, self.q_indptr, self.o, self.lse,
                                      self.workspace, stream=stream)
        else:
            spec_attn_run(self.plan, self.q, self.k_pool, self.v_pool, self.block_table, self.seq_lens,
                          self.q_indptr, self.o, self.lse, self.workspace, self.k_scales, self.v_scales,
                          self.wl.k_gscale, self.wl.v_gscale, stream)

    def run_traced(self, trace, stream=None):
        if self.block_k is not None:
            spec_attn_run_dense_block(self.plan, self.q, self.block_k, self.block_v, self.k_pool, self.v_pool,
                                      self.block_table, self.seq_lens, self.q_indptr, self.o, self.lse,
                                      self.workspace, trace=trace, stream=stream)
            return
        spec_attn_run_traced(self.plan, self.q, self.k_pool, self.v_pool, self.block_table,
                             self.seq_lens, self.q_indptr, self.o, self.lse, trace, self.workspace,
                             self.k_scales, self.v_scales, self.wl.k_gscale, self.wl.v_gscale, stream)

    def device_status(self) -> int:
        return spec_attn_check_device_status(self.workspace)
