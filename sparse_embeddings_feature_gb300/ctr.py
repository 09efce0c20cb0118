"""Thin Python binding of libctr (the C-ABI declared in include/ctr.h).

Every function here has the name of the C call it wraps and only marshals
arguments: torch tensors become device pointers, the current CUDA stream is
passed along, and a negative ctr_status becomes a CtrError.  All computation
happens in libctr's CUDA kernels; there is no CPU fallback.  If the library
cannot be built or loaded the first call raises.

The calls of the expert layer and of the layers around it are short enough that
reading their arguments here costs more than the kernels: in the usual layouts (dense tensors, the current
stream) csrc/calls.cpp reads them, and what it does not take comes back here.
"""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
import threading
import warnings
from typing import Optional, Sequence

import numpy as np
import torch

from . import build as _build

F32, BF16 = 0, 1
POOL_SUM, POOL_MEAN = 0, 1
DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
# status codes (ctr_status in include/ctr.h)
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE = 0, -1, -2, -3
ERR_INDEX_OUT_OF_RANGE, ERR_CUDA, ERR_TIMEOUT, ERR_NOT_IMPLEMENTED, ERR_BAD_OFFSETS = -4, -5, -6, -7, -8
ERR_BAD_VALUE = -9
MAX_EXPERTS, MAX_CHOICES = 512, 16

_lock = threading.Lock()
_lib = None
_calls = None
_p = C.c_void_p
_i32, _i64, _u64, _f32, _sz = C.c_int32, C.c_int64, C.c_uint64, C.c_float, C.c_size_t

# name -> (restype, argtypes), mirroring include/ctr.h
_SIGS = {
    "ctr_status_string": (C.c_char_p, [C.c_int]),
    "ctr_version": (C.c_int, []),
    "ctr_set_timing_events": (C.c_int, [C.c_int, _p, _p]),
    "ctr_launch_count": (C.c_uint64, []),
    "ctr_set_tma_gather": (C.c_int, [C.c_int]),
    "ctr_set_tile_slices": (C.c_int, [C.c_int]),
    "ctr_set_wait_limit_ns": (C.c_uint64, [C.c_uint64]),
    "ctr_status_reset": (C.c_int, [_p, _p]),
    "ctr_check_status": (C.c_int, [_p, _p]),
    "ctr_fill_table": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, C.c_int, _u64, _f32, _p]),
    "ctr_dedup_workspace_size": (_sz, [_i64, _i32, _i32, _i64]),
    "ctr_dedup": (C.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i64, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "ctr_dedup_phases": (C.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i64, _p, _p, _p, _p, _p, _p, _p, _i32, _p, _sz,
                                   _p]),
    "ctr_gather_rows": (C.c_int, [_p, C.c_int, _i32, _i64, _p, _p, _i64, _p, _p, _sz, _p]),
    "ctr_embedding_bag_workspace_size": (_sz, []),
    "ctr_embedding_bag_fwd": (C.c_int, [_p, C.c_int, _i32, _i64, _p, C.c_int, _i64, _p, _i32, _i32, _p, _p, _i32, C.c_int,
                                        _p, C.c_int, _i64, _i64, _p, _sz, _p]),
    "ctr_embedding_bag_fwd_fm": (C.c_int, [_p, C.c_int, _i32, _i64, _p, C.c_int, _i64, _p, _i32, _i32, _p, _p, _i32,
                                           C.c_int, _p, C.c_int, _i64, _i64, _p, _p, _sz, _p]),
    "ctr_interaction_workspace_size": (_sz, []),
    "ctr_dot_interaction": (C.c_int, [_p, C.c_int, _i32, _i32, _i32, _p, _p, _sz, _p]),
    "ctr_dot_interaction_bwd": (C.c_int, [_p, _p, _i32, _i32, _i32, _p, _p, _sz, _p]),
    "ctr_bwd_update_workspace_size": (_sz, [_i64, _i32]),
    "ctr_embedding_bag_bwd_update": (C.c_int, [_p, _i64, _i64, _p, _i32, _i32, C.c_int, _p, _p, _p, _p, _i64, _f32,
                                               _p, C.c_int, _i32, _i64, _p, _p, _sz, _p]),
    "ctr_interaction_width": (C.c_int64, [_i32, _i32, C.c_int]),
    "ctr_embedding_bag_bwd_update_opt": (C.c_int, [_p, _i64, _i64, _p, _i32, _i32, C.c_int, _p, _p, _p, _p, _i64,
                                                   _f32, _p, C.c_int, _i32, _i64, _p, C.c_int, _p, _p, _sz, _p]),
    "ctr_dot_interaction_mode": (C.c_int, [_p, C.c_int, _i32, _i32, _i32, C.c_int, _p, _p, _sz, _p]),
    "ctr_dot_interaction_bwd_mode": (C.c_int, [_p, _p, _i32, _i32, _i32, C.c_int, _p, _p, _sz, _p]),
    "ctr_embedding_bag_bwd_update_phases": (C.c_int, [_p, _i64, _i64, _p, _i32, _i32, C.c_int, _p, _p, _p, _p, _i64,
                                                      _f32, _p, C.c_int, _i32, _i64, _p, C.c_int, _p, _sz, _p]),
    "ctr_set_route_cluster": (C.c_int, [C.c_int]),
    "ctr_expert_route_workspace_size": (_sz, [_i64, _i32, _i32]),
    "ctr_expert_route": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _i32, C.c_int, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "ctr_expert_route_bwd": (C.c_int, [_p, _p, C.c_int, _i64, _i32, _i64, _i32, C.c_int, _p, _p, _i64, _p, _sz, _p]),
    "ctr_expert_workspace_size": (_sz, []),
    "ctr_expert_dispatch": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _i32, _p, _p, _p, _i64, _p, _sz, _p]),
    "ctr_expert_combine": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _i32, _p, _p, _p, _i64, _p, _sz, _p]),
    "ctr_expert_combine_bwd": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _i32, _p, _i64, _p, _p, _p, _p, _i64, _p, _p,
                                         _sz, _p]),
    "ctr_fp8_padded_rows": (C.c_int64, [_i64, _i32]),
    "ctr_fp8_quantize_rows": (C.c_int, [_p, C.c_int, _i64, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _sz, _p]),
    "ctr_fp8_quantize_rows_cols": (C.c_int, [_p, C.c_int, _i64, _i64, _i64, _i64, _p, _p, _i32, C.c_int, _p, _p, _i64,
                                             _p, _p, _p, _sz, _p]),
    "ctr_fp8_quantize_blocks": (C.c_int, [_p, C.c_int, _i32, _i64, _i64, _p, _p, _p, _p, _p, _sz, _p]),
    "ctr_fp8_matmul_workspace_size": (_sz, [_i64, _i32, _i64, _i64]),
    "ctr_fp8_matmul": (C.c_int, [_p, _p, _i64, _p, _p, _p, _i64, _i32, _i64, _i64, _p, C.c_int, _i64, _p, _sz, _p]),
    "ctr_fp8_matmul_wgrad": (C.c_int, [_p, _p, _p, _p, _p, _i64, _i32, _i64, _i64, _p, C.c_int, _p, _sz, _p]),
    "ctr_expert_route_balanced": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _i32, C.c_int, _p, _i32, _i32, C.c_int, _f32, _p,
                                            _p, _p, _p, _p, _p, _sz, _p]),
    "ctr_expert_route_balanced_bwd": (C.c_int, [_p, _p, C.c_int, _i64, _i32, _i64, _i32, C.c_int, C.c_int, _f32, _p, _p,
                                                _i64, _p, _sz, _p]),
    "ctr_dense_workspace_size": (_sz, [_i64, _i64, _i64, C.c_int, C.c_int, C.c_int]),
    "ctr_dense": (C.c_int, [_p, C.c_int, _i64, _i64, _i64, _p, _i64, _i64, _p, C.c_int, _p, _i64, _p, _i64, _p, _i64, _p,
                            _sz, _p]),
    "ctr_dense_bwd": (C.c_int, [_p, C.c_int, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _p, _i64, C.c_int, _p, _i64,
                                C.c_int, _p, _i64, _p, _p, _sz, _p]),
    "ctr_rms_norm_workspace_size": (_sz, [_i64, _i32]),
    "ctr_rms_norm": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _p, _i64, _p, _f32, _p, _i64, _p, _i64, _p, _p, _i64, _p,
                               _sz, _p]),
    "ctr_rms_norm_bwd": (C.c_int, [_p, C.c_int, _i64, _i32, _i64, _p, _i64, _p, _i64, _p, _f32, _p, _i64, _p, _p, _sz,
                                   _p]),
    "ctr_clip_grads_workspace_size": (_sz, []),
    "ctr_clip_grads": (C.c_int, [_p, _p, _p, _p, _i32, _f32, _p, _p, _sz, _p]),
}


class CtrError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} returned {status} ({status_string(status)})")
        self.status = status


def lib() -> C.CDLL:
    """Load libctr.so, building it first if the sources changed.  Raises if that fails."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libctr not found at {path}")
            L = C.CDLL(path)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


class _NoCalls:
    """In the place of csrc/calls.cpp where it cannot be compiled or loaded: takes no call."""

    def __getattr__(self, name):
        return lambda *args: None


def _usual():
    """The calls in their usual layouts (csrc/calls.cpp): each returns its status, or None if it did not take it."""
    global _calls
    if _calls is None:
        lib()
        with _lock:
            path = _build.build_calls() if _calls is None else None
            if path is not None:
                try:
                    loader = importlib.machinery.ExtensionFileLoader("ctr_calls", path)
                    calls = importlib.util.module_from_spec(importlib.util.spec_from_loader("ctr_calls", loader))
                    loader.exec_module(calls)
                    _calls = calls
                except ImportError as e:
                    warnings.warn(f"{path} cannot be loaded, the layers' calls read their arguments in Python: {e}",
                                  RuntimeWarning)
            if _calls is None:
                _calls = _NoCalls()
    return _calls


def _took(name: str, st: Optional[int]) -> bool:
    if st:
        raise CtrError(name, st)
    return st is not None


def library_path() -> str:
    return _build.LIB


def status_string(status: int) -> str:
    return lib().ctr_status_string(int(status)).decode()


def _ok(name: str, st: int) -> None:
    if st != 0:
        raise CtrError(name, st)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    # the current stream's handle, without building a torch.cuda.Stream object on every call
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream


_raw_stream = torch._C._cuda_getCurrentRawStream


def _host_i32(a) -> C.Array:
    a = np.ascontiguousarray(a, dtype=np.int32)
    return (C.c_int32 * a.size)(*a.tolist())


def _host_i64(a) -> C.Array:
    a = np.ascontiguousarray(a, dtype=np.int64)
    return (C.c_int64 * a.size)(*a.tolist())


def _dev(t: torch.Tensor, what: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t


KERNEL_GATHER, KERNEL_BWD_TILES, KERNEL_BWD_PIECES, KERNEL_SORT, KERNEL_INTERACTION, KERNEL_INTERACTION_BWD, \
    KERNEL_GATHER_ROWS = 1, 2, 3, 4, 5, 6, 7


def ctr_set_timing_events(kernel: int, before=None, after=None) -> None:
    """Record torch.cuda.Events around every later launch of `kernel` (None, None: off).

    The events must already have been recorded once, so that torch has created them.
    """
    b = None if before is None else C.c_void_p(before.cuda_event)
    e = None if after is None else C.c_void_p(after.cuda_event)
    _ok("ctr_set_timing_events", lib().ctr_set_timing_events(int(kernel), b, e))


def ctr_launch_count() -> int:
    """Kernel launches the library has issued in this process so far."""
    return int(lib().ctr_launch_count())


def ctr_set_tma_gather(on: bool) -> bool:
    """Select the TMA row-gather variant of the fp32 d=128 pooled gather; returns the previous setting."""
    return bool(lib().ctr_set_tma_gather(1 if on else 0))


def ctr_set_wait_limit_ns(ns: int) -> int:
    """Wall-clock limit of each radix-pass look-back wait of ctr_dedup (diagnostics); returns the previous."""
    return int(lib().ctr_set_wait_limit_ns(int(ns)))


def ctr_set_tile_slices(mode: int) -> int:
    """Short-run pass of the fp32 d=128 SGD row update: 0 automatic, 1 never sliced, 2 always in
    64-column slices; returns the previous mode."""
    return int(lib().ctr_set_tile_slices(int(mode)))


# ---------------------------------------------------------------------------
# status / workspace
# ---------------------------------------------------------------------------
def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zeroed device buffer usable as a libctr workspace (torch allocations are 512-byte aligned)."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device or "cuda")


def ctr_status_reset(ws: torch.Tensor, stream=None) -> None:
    _ok("ctr_status_reset", lib().ctr_status_reset(_ptr(ws), _stream(stream)))


def ctr_check_status(ws: torch.Tensor, stream=None) -> int:
    return int(lib().ctr_check_status(_ptr(ws), _stream(stream)))


def ctr_dedup_workspace_size(n_ids: int, num_fields: int, batch: int, total_rows: int) -> int:
    return int(lib().ctr_dedup_workspace_size(n_ids, num_fields, batch, total_rows))


def ctr_embedding_bag_workspace_size() -> int:
    return int(lib().ctr_embedding_bag_workspace_size())


def ctr_interaction_workspace_size() -> int:
    return int(lib().ctr_interaction_workspace_size())


def ctr_bwd_update_workspace_size(n_ids: int, d: int) -> int:
    return int(lib().ctr_bwd_update_workspace_size(n_ids, d))


# ---------------------------------------------------------------------------
# calls
# ---------------------------------------------------------------------------
def ctr_fill_table(table: torch.Tensor, d: int, row0: int, gen_kind: int, seed: int, scale: float,
                   stream=None) -> None:
    _dev(table, "table")
    rows = table.numel() // d
    _ok("ctr_fill_table", lib().ctr_fill_table(_ptr(table), DTYPES[table.dtype], rows, d, row0, gen_kind,
                                               C.c_uint64(seed & ((1 << 64) - 1)), scale, _stream(stream)))


def ctr_dedup(ids: torch.Tensor, offsets: torch.Tensor, num_fields: int, batch: int, bag_to_table: Sequence[int],
              row_base: Sequence[int], unique_rows: torch.Tensor, n_unique: torch.Tensor,
              inverse: Optional[torch.Tensor], sorted_pos: Optional[torch.Tensor], sorted_bag: Optional[torch.Tensor],
              run_offsets: Optional[torch.Tensor], unique_offsets: Optional[torch.Tensor], ws: torch.Tensor,
              n_ids: Optional[int] = None, stream=None) -> None:
    n = int(ids.numel()) if n_ids is None else int(n_ids)
    rb = np.asarray(row_base, dtype=np.int64)
    st = lib().ctr_dedup(_ptr(ids), _ptr(offsets), num_fields, batch, _host_i32(bag_to_table), _host_i64(rb),
                         rb.size - 1, n, _ptr(unique_rows), _ptr(n_unique), _ptr(inverse), _ptr(sorted_pos),
                         _ptr(sorted_bag), _ptr(run_offsets), _ptr(unique_offsets), _ptr(ws), ws.numel(),
                         _stream(stream))
    _ok("ctr_dedup", st)


DEDUP_PREPARE, DEDUP_SORT, DEDUP_ALL = 1, 2, 3


def ctr_dedup_phases(ids: torch.Tensor, offsets: torch.Tensor, num_fields: int, batch: int,
                     bag_to_table: Sequence[int], row_base: Sequence[int], unique_rows: torch.Tensor,
                     n_unique: torch.Tensor, inverse: Optional[torch.Tensor], sorted_pos: Optional[torch.Tensor],
                     sorted_bag: Optional[torch.Tensor], run_offsets: Optional[torch.Tensor],
                     unique_offsets: Optional[torch.Tensor], phases: int, ws: torch.Tensor,
                     n_ids: Optional[int] = None, stream=None) -> None:
    n = int(ids.numel()) if n_ids is None else int(n_ids)
    rb = np.asarray(row_base, dtype=np.int64)
    st = lib().ctr_dedup_phases(_ptr(ids), _ptr(offsets), num_fields, batch, _host_i32(bag_to_table),
                                _host_i64(rb), rb.size - 1, n, _ptr(unique_rows), _ptr(n_unique), _ptr(inverse),
                                _ptr(sorted_pos), _ptr(sorted_bag), _ptr(run_offsets), _ptr(unique_offsets),
                                int(phases), _ptr(ws), ws.numel(), _stream(stream))
    _ok("ctr_dedup_phases", st)


def ctr_gather_rows(table: torch.Tensor, d: int, unique_rows: torch.Tensor, n_unique: torch.Tensor, U: torch.Tensor,
                    ws: torch.Tensor, stream=None) -> None:
    total_rows = table.numel() // d
    capacity = U.numel() // d
    st = lib().ctr_gather_rows(_ptr(table), DTYPES[table.dtype], d, total_rows, _ptr(unique_rows), _ptr(n_unique),
                               capacity, _ptr(U), _ptr(ws), ws.numel(), _stream(stream))
    _ok("ctr_gather_rows", st)


def ctr_embedding_bag_fwd(table: torch.Tensor, d: int, indices: torch.Tensor, offsets: torch.Tensor,
                          num_fields: int, batch: int, bag_to_table: Optional[Sequence[int]],
                          row_base: Optional[Sequence[int]], pool: int, out: torch.Tensor, out_stride_b: int,
                          out_stride_f: int, ws: torch.Tensor, total_rows: Optional[int] = None,
                          n_indices: Optional[int] = None, stream=None, fm_out: Optional[torch.Tensor] = None) -> None:
    """Pooled gather; with fm_out (fp32 [F*B]) the ctr_embedding_bag_fwd_fm call, which also
    writes each bag's FM second-order term."""
    total = int(table.numel() // d) if total_rows is None else int(total_rows)
    if bag_to_table is not None:
        rb = np.asarray(row_base, dtype=np.int64)
        b2t, rbp, T = _host_i32(bag_to_table), _host_i64(rb), rb.size - 1
    else:
        b2t, rbp, T = None, None, 0
    n_idx = int(indices.numel()) if n_indices is None else int(n_indices)
    args = (_ptr(table), DTYPES[table.dtype], d, total, _ptr(indices), 1 if indices.dtype == torch.int32 else 0, n_idx,
            _ptr(offsets), num_fields, batch, b2t, rbp, T, pool, _ptr(out), DTYPES[out.dtype], out_stride_b,
            out_stride_f)
    if fm_out is None:
        st = lib().ctr_embedding_bag_fwd(*args, _ptr(ws), ws.numel(), _stream(stream))
        _ok("ctr_embedding_bag_fwd", st)
    else:
        st = lib().ctr_embedding_bag_fwd_fm(*args, _ptr(fm_out), _ptr(ws), ws.numel(), _stream(stream))
        _ok("ctr_embedding_bag_fwd_fm", st)


def ctr_dot_interaction(X: torch.Tensor, n: int, d: int, out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    batch = X.numel() // (n * d)
    st = lib().ctr_dot_interaction(_ptr(X), DTYPES[X.dtype], batch, n, d, _ptr(out), _ptr(ws), ws.numel(),
                                   _stream(stream))
    _ok("ctr_dot_interaction", st)


def ctr_dot_interaction_bwd(dout: torch.Tensor, X: torch.Tensor, n: int, d: int, dX: torch.Tensor,
                            ws: torch.Tensor, stream=None) -> None:
    batch = X.numel() // (n * d)
    st = lib().ctr_dot_interaction_bwd(_ptr(dout), _ptr(X), batch, n, d, _ptr(dX), _ptr(ws), ws.numel(),
                                       _stream(stream))
    _ok("ctr_dot_interaction_bwd", st)


INTERACT_CROSS, INTERACT_WITH_SELF, INTERACT_FULL_GRAM = 0, 1, 2


def ctr_interaction_width(n: int, d: int, mode: int) -> int:
    return int(lib().ctr_interaction_width(n, d, mode))


def ctr_dot_interaction_mode(X: torch.Tensor, n: int, d: int, mode: int, out: torch.Tensor, ws: torch.Tensor,
                             stream=None) -> None:
    batch = X.numel() // (n * d)
    st = lib().ctr_dot_interaction_mode(_ptr(X), DTYPES[X.dtype], batch, n, d, int(mode), _ptr(out), _ptr(ws),
                                        ws.numel(), _stream(stream))
    _ok("ctr_dot_interaction_mode", st)


def ctr_dot_interaction_bwd_mode(dout: torch.Tensor, X: torch.Tensor, n: int, d: int, mode: int, dX: torch.Tensor,
                                 ws: torch.Tensor, stream=None) -> None:
    batch = X.numel() // (n * d)
    st = lib().ctr_dot_interaction_bwd_mode(_ptr(dout), _ptr(X), batch, n, d, int(mode), _ptr(dX), _ptr(ws),
                                            ws.numel(), _stream(stream))
    _ok("ctr_dot_interaction_bwd_mode", st)


def ctr_embedding_bag_bwd_update(grad_pooled: torch.Tensor, g_stride_b: int, g_stride_f: int, offsets: torch.Tensor,
                                 num_fields: int, batch: int, pool: int, unique_rows: torch.Tensor,
                                 n_unique: torch.Tensor, run_offsets: torch.Tensor, sorted_bag: torch.Tensor,
                                 n_ids: int, lr: float, table: torch.Tensor, d: int,
                                 grad_unique_out: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    total_rows = table.numel() // d
    st = lib().ctr_embedding_bag_bwd_update(_ptr(grad_pooled), g_stride_b, g_stride_f, _ptr(offsets), num_fields,
                                            batch, pool, _ptr(unique_rows), _ptr(n_unique), _ptr(run_offsets),
                                            _ptr(sorted_bag), n_ids, lr, _ptr(table), DTYPES[table.dtype], d,
                                            total_rows, _ptr(grad_unique_out), _ptr(ws), ws.numel(), _stream(stream))
    _ok("ctr_embedding_bag_bwd_update", st)


BWD_LONG_RUNS, BWD_SHORT_RUNS, BWD_FINISH = 1, 2, 4
BWD_ALL = BWD_SHORT_RUNS | BWD_LONG_RUNS | BWD_FINISH
OPT_SGD, OPT_ADAGRAD, OPT_ROWWISE_ADAGRAD, OPT_ADAM = 0, 1, 2, 3


class CtrOptimizer(C.Structure):
    """ctr_optimizer of ctr.h."""
    _fields_ = [("kind", C.c_int), ("eps", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float),
                ("step", C.c_int64), ("state0", C.c_void_p), ("state1", C.c_void_p),
                ("stochastic_rounding", C.c_int32), ("sr_seed", C.c_uint64)]


def optimizer(kind: int, eps: float = 1e-8, beta1: float = 0.9, beta2: float = 0.999, step: int = 1,
              state0: Optional[torch.Tensor] = None, state1: Optional[torch.Tensor] = None,
              stochastic_rounding: bool = False, sr_seed: int = 0) -> CtrOptimizer:
    return CtrOptimizer(int(kind), float(eps), float(beta1), float(beta2), int(step),
                        None if state0 is None else _ptr(state0), None if state1 is None else _ptr(state1),
                        1 if stochastic_rounding else 0, int(sr_seed) & ((1 << 64) - 1))


def ctr_embedding_bag_bwd_update_opt(grad_pooled: torch.Tensor, g_stride_b: int, g_stride_f: int,
                                     offsets: torch.Tensor, num_fields: int, batch: int, pool: int,
                                     unique_rows: torch.Tensor, n_unique: torch.Tensor, run_offsets: torch.Tensor,
                                     sorted_bag: torch.Tensor, n_ids: int, lr: float, table: torch.Tensor, d: int,
                                     grad_unique_out: Optional[torch.Tensor], phases: int, opt: CtrOptimizer,
                                     ws: torch.Tensor, stream=None) -> None:
    total_rows = table.numel() // d
    st = lib().ctr_embedding_bag_bwd_update_opt(_ptr(grad_pooled), g_stride_b, g_stride_f, _ptr(offsets), num_fields,
                                                batch, pool, _ptr(unique_rows), _ptr(n_unique), _ptr(run_offsets),
                                                _ptr(sorted_bag), n_ids, lr, _ptr(table), DTYPES[table.dtype], d,
                                                total_rows, _ptr(grad_unique_out), int(phases), C.addressof(opt),
                                                _ptr(ws), ws.numel(), _stream(stream))
    _ok("ctr_embedding_bag_bwd_update_opt", st)


def ctr_embedding_bag_bwd_update_phases(grad_pooled: torch.Tensor, g_stride_b: int, g_stride_f: int,
                                        offsets: torch.Tensor, num_fields: int, batch: int, pool: int,
                                        unique_rows: torch.Tensor, n_unique: torch.Tensor, run_offsets: torch.Tensor,
                                        sorted_bag: torch.Tensor, n_ids: int, lr: float, table: torch.Tensor, d: int,
                                        grad_unique_out: Optional[torch.Tensor], phases: int, ws: torch.Tensor,
                                        stream=None) -> None:
    total_rows = table.numel() // d
    st = lib().ctr_embedding_bag_bwd_update_phases(_ptr(grad_pooled), g_stride_b, g_stride_f, _ptr(offsets),
                                                   num_fields, batch, pool, _ptr(unique_rows), _ptr(n_unique),
                                                   _ptr(run_offsets), _ptr(sorted_bag), n_ids, lr, _ptr(table),
                                                   DTYPES[table.dtype], d, total_rows, _ptr(grad_unique_out),
                                                   int(phases), _ptr(ws), ws.numel(), _stream(stream))
    _ok("ctr_embedding_bag_bwd_update_phases", st)


# ---------------------------------------------------------------------------
# expert layer
# ---------------------------------------------------------------------------
# These calls take their sizes from the tensors' shapes, so the shapes, types and
# layouts are checked here: the library sees only pointers.  Matrices may have a
# row stride; maps, weights, codes and scales are dense.  The checks are written
# for their cost: a call of a small batch is a few microseconds of kernels.
_F = (torch.float32, torch.bfloat16)
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_F32_ONLY = (torch.float32,)


def _here(device: Optional[int], what: str) -> None:
    """Refuse data of another device than the current one, where the call's kernels run."""
    if device is not None and device != torch.cuda.current_device():
        raise ValueError(f"{what} is on cuda:{device}, and the current device is cuda:{torch.cuda.current_device()}")


def _mat(t: torch.Tensor, what: str, dtypes=_F):
    """(rows, columns, row stride) of a CUDA matrix whose rows are contiguous and do not overlap."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes:
        _here(t.get_device(), what)
        shape = t.shape
        if len(shape) == 2:
            rows, cols = shape
            if t.is_contiguous():
                return rows, cols, cols or 1
            ld, step = t.stride()
            if (cols <= 1 or step == 1) and (rows <= 1 or ld >= cols):
                return rows, cols, ld if rows > 1 else max(1, cols)
    raise ValueError(f"{what} must be a CUDA matrix of {' or '.join(str(d) for d in dtypes)} with contiguous rows "
                     f"that do not overlap")


def _dense(t: torch.Tensor, what: str, dtype, shape) -> None:
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda:
        _here(t.get_device(), what)
        return
    raise ValueError(f"{what} must be a contiguous CUDA tensor of {dtype} and shape {tuple(shape)}")


def _room(ws: torch.Tensor):
    """(address, bytes) of a workspace: dense bytes on the current device."""
    if isinstance(ws, torch.Tensor) and ws.is_cuda and ws.dtype is _U8 and ws.is_contiguous():
        _here(ws.get_device(), "ws")
        return ws.data_ptr(), ws.numel()
    raise ValueError("ws must be a contiguous CUDA tensor of torch.uint8")


def _want(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _like(t: torch.Tensor, what: str, rows: int, cols: int, dtype) -> int:
    """Row stride of a matrix of the given shape and type."""
    r, c, ld = _mat(t, what, (dtype,))
    if r != rows or c != cols:
        raise ValueError(f"{what} must be {(rows, cols)}, not {(r, c)}")
    return ld


def ctr_expert_workspace_size() -> int:
    return int(lib().ctr_expert_workspace_size())


def ctr_expert_route_workspace_size(tokens: int, experts: int, k: int) -> int:
    return int(lib().ctr_expert_route_workspace_size(tokens, experts, k))


def ctr_set_route_cluster(on: bool) -> bool:
    """Routing of mid-sized batches as one thread-block cluster (the default) or always as three launches;
    returns the previous setting."""
    return bool(lib().ctr_set_route_cluster(1 if on else 0))


def ctr_expert_route(scores: torch.Tensor, k: int, renormalize: bool, expert: torch.Tensor, weight: torch.Tensor,
                     slot: torch.Tensor, token: torch.Tensor, offsets: torch.Tensor, ws: torch.Tensor,
                     stream=None) -> None:
    """The k best experts of every token (row of scores), their softmax weights, and the order by expert."""
    if stream is None and _took("ctr_expert_route", _usual().expert_route(scores, k, renormalize, expert, weight, slot,
                                                                          token, offsets, ws)):
        return
    T, E, ld = _mat(scores, "scores")
    tk = (T, k)
    _dense(expert, "expert", _I32, tk)
    _dense(weight, "weight", _F32, tk)
    _dense(slot, "slot", _I32, tk)
    _dense(token, "token", _I32, (T * k,))
    _dense(offsets, "offsets", _I32, (E + 1,))
    st = lib().ctr_expert_route(scores.data_ptr(), DTYPES[scores.dtype], T, E, ld, k, 1 if renormalize else 0,
                                expert.data_ptr(), weight.data_ptr(), slot.data_ptr(), token.data_ptr(),
                                offsets.data_ptr(), *_room(ws), _stream(stream))
    if st:
        _ok("ctr_expert_route", st)


def ctr_expert_route_bwd(dweight: torch.Tensor, scores: torch.Tensor, renormalize: bool, expert: torch.Tensor,
                         dscores: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    if stream is None and _took("ctr_expert_route_bwd", _usual().expert_route_bwd(dweight, scores, renormalize,
                expert, dscores, ws)):
        return
    T, E, ld = _mat(scores, "scores")
    _want(isinstance(expert, torch.Tensor) and expert.dim() == 2, "expert must be a matrix")
    k = expert.shape[1]
    _dense(expert, "expert", _I32, (T, k))
    _dense(dweight, "dweight", _F32, (T, k))
    ldd = _like(dscores, "dscores", T, E, scores.dtype)
    st = lib().ctr_expert_route_bwd(dweight.data_ptr(), scores.data_ptr(), DTYPES[scores.dtype], T, E, ld, k,
                                    1 if renormalize else 0, expert.data_ptr(), dscores.data_ptr(), ldd,
                                    *_room(ws), _stream(stream))
    if st:
        _ok("ctr_expert_route_bwd", st)


def _slots(slot: torch.Tensor, T: int) -> int:
    """k of a slot map [T, k]."""
    _want(isinstance(slot, torch.Tensor) and slot.dim() == 2, "slot must be a matrix")
    k = slot.shape[1]
    _dense(slot, "slot", _I32, (T, k))
    return k


def ctr_expert_dispatch(x: torch.Tensor, slot: torch.Tensor, token: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                        stream=None) -> None:
    """Token rows of x into the order by expert: out [T*k, d]."""
    if stream is None and _took("ctr_expert_dispatch", _usual().expert_dispatch(x, slot, token, out, ws)):
        return
    T, d, ld = _mat(x, "x")
    k = _slots(slot, T)
    _dense(token, "token", _I32, (T * k,))
    ldo = _like(out, "out", T * k, d, x.dtype)
    st = lib().ctr_expert_dispatch(x.data_ptr(), DTYPES[x.dtype], T, d, ld, k, slot.data_ptr(), token.data_ptr(),
                                   out.data_ptr(), ldo, *_room(ws), _stream(stream))
    if st:
        _ok("ctr_expert_dispatch", st)


def ctr_expert_combine(rows: torch.Tensor, slot: torch.Tensor, weight: Optional[torch.Tensor], y: torch.Tensor,
                       ws: torch.Tensor, stream=None) -> None:
    """Rows [T*k, d] added back to tokens under the weights (None: all 1, the gradient of the dispatch)."""
    if stream is None and _took("ctr_expert_combine", _usual().expert_combine(rows, slot, weight, y, ws)):
        return
    T, d, ldy = _mat(y, "y")
    k = _slots(slot, T)
    ldr = _like(rows, "rows", T * k, d, y.dtype)
    if weight is not None:
        _dense(weight, "weight", _F32, (T, k))
    st = lib().ctr_expert_combine(rows.data_ptr(), DTYPES[y.dtype], T, d, ldr, k, slot.data_ptr(), _ptr(weight),
                                  y.data_ptr(), ldy, *_room(ws), _stream(stream))
    if st:
        _ok("ctr_expert_combine", st)


def ctr_expert_combine_bwd(dy: torch.Tensor, rows: torch.Tensor, slot: torch.Tensor, weight: torch.Tensor,
                           token: torch.Tensor, drows: torch.Tensor, dweight: torch.Tensor, ws: torch.Tensor,
                           stream=None) -> None:
    if stream is None and _took("ctr_expert_combine_bwd", _usual().expert_combine_bwd(dy, rows, slot, weight, token,
                drows, dweight, ws)):
        return
    T, d, ldy = _mat(dy, "dy")
    k = _slots(slot, T)
    ldr = _like(rows, "rows", T * k, d, dy.dtype)
    ldd = _like(drows, "drows", T * k, d, dy.dtype)
    _dense(weight, "weight", _F32, (T, k))
    _dense(dweight, "dweight", _F32, (T, k))
    _dense(token, "token", _I32, (T * k,))
    st = lib().ctr_expert_combine_bwd(dy.data_ptr(), DTYPES[dy.dtype], T, d, ldy, k, rows.data_ptr(), ldr,
                                      slot.data_ptr(), weight.data_ptr(), token.data_ptr(), drows.data_ptr(), ldd,
                                      dweight.data_ptr(), *_room(ws), _stream(stream))
    if st:
        _ok("ctr_expert_combine_bwd", st)


# -- 8-bit products -----------------------------------------------------------
FP8_COLS_BY_COLUMN, FP8_COLS_BY_BLOCK = 0, 1


def fp8_blocks(n: int) -> int:
    """Blocks of 128 that n elements take."""
    return -(-int(n) // 128)


def fp8_padded(n: int) -> int:
    """n rounded up to whole blocks: the row length of codes."""
    return 128 * fp8_blocks(n)


def fp8_padded_rows(rows: int, groups: int) -> int:
    """Row length of the column codes of `rows` rows in `groups` groups."""
    return int(lib().ctr_fp8_padded_rows(rows, groups))


def ctr_fp8_matmul_workspace_size(rows: int, groups: int, n: int, k: int) -> int:
    return int(lib().ctr_fp8_matmul_workspace_size(rows, groups, n, k))


def _codes_of(q: torch.Tensor, row_index: Optional[torch.Tensor], n: int, cols: int) -> int:
    """Rows of the row codes q of a matrix [n, cols], through a map or without."""
    _want(isinstance(q, torch.Tensor) and q.dim() == 2, "q must be a matrix")
    rows = q.shape[0]
    _dense(q, "q", _U8, (rows, (cols + 127) // 128 * 128))
    if row_index is not None:
        _dense(row_index, "row_index", _I32, (rows,))
    elif rows > n:
        raise ValueError("without row_index, q may not have more rows than x")
    return rows


def ctr_fp8_quantize_rows(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, ws: torch.Tensor,
                          row_index: Optional[torch.Tensor] = None, stream=None) -> None:
    """Row codes q [rows, padded cols] and scales [blocks, rows] of x, or of its rows row_index."""
    if stream is None and _took("ctr_fp8_quantize_rows", _usual().fp8_quantize_rows(x, q, scale, ws, row_index)):
        return
    n, cols, ld = _mat(x, "x")
    rows = _codes_of(q, row_index, n, cols)
    lds = _like(scale, "scale", (cols + 127) // 128, rows, _F32)
    st = lib().ctr_fp8_quantize_rows(x.data_ptr(), DTYPES[x.dtype], n, rows, cols, ld, _ptr(row_index), q.data_ptr(),
                                     scale.data_ptr(), lds, *_room(ws), _stream(stream))
    if st:
        _ok("ctr_fp8_quantize_rows", st)


def ctr_fp8_quantize_rows_cols(x: torch.Tensor, offsets: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                               qc: torch.Tensor, scale_c: torch.Tensor, cols_by: int, ws: torch.Tensor,
                               row_index: Optional[torch.Tensor] = None, stream=None) -> None:
    """Row codes as above, and the column codes qc [cols, padded rows] of the grouped rows, in one read of x."""
    if stream is None and _took("ctr_fp8_quantize_rows_cols", _usual().fp8_quantize_rows_cols(x, offsets, q, scale,
                qc, scale_c, cols_by, ws, row_index)):
        return
    n, cols, ld = _mat(x, "x")
    rows = _codes_of(q, row_index, n, cols)
    _want(isinstance(offsets, torch.Tensor) and offsets.numel() >= 2, "offsets must have at least two entries")
    groups = offsets.numel() - 1
    _dense(offsets, "offsets", _I32, (groups + 1,))
    padded = fp8_padded_rows(rows, groups)
    lds = _like(scale, "scale", (cols + 127) // 128, rows, _F32)
    _dense(qc, "qc", _U8, (cols, padded))
    _dense(scale_c, "scale_c", _F32, (padded // 128, cols) if cols_by == FP8_COLS_BY_COLUMN
           else ((cols + 127) // 128, padded // 128))
    st = lib().ctr_fp8_quantize_rows_cols(x.data_ptr(), DTYPES[x.dtype], n, rows, cols, ld, _ptr(row_index),
                                          offsets.data_ptr(), groups, cols_by, q.data_ptr(), scale.data_ptr(), lds,
                                          qc.data_ptr(), scale_c.data_ptr(), *_room(ws),
                                          _stream(stream))
    if st:
        _ok("ctr_fp8_quantize_rows_cols", st)


def ctr_fp8_quantize_blocks(w: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, ws: torch.Tensor,
                            qt: Optional[torch.Tensor] = None, scale_t: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """Block codes of w [groups, n, k], and of its transpose where qt and scale_t are given."""
    if stream is None and _took("ctr_fp8_quantize_blocks", _usual().fp8_quantize_blocks(w, q, scale, ws, qt, scale_t)):
        return
    _want(isinstance(w, torch.Tensor) and w.dim() == 3 and w.dtype in DTYPES, "w must be [groups, n, k] fp32 or bf16")
    G, n, k = w.shape
    _dense(w, "w", w.dtype, (G, n, k))
    _dense(q, "q", torch.uint8, (G, n, fp8_padded(k)))
    _dense(scale, "scale", torch.float32, (G, fp8_blocks(n), fp8_blocks(k)))
    if qt is not None or scale_t is not None:
        _want(qt is not None and scale_t is not None, "qt and scale_t go together")
        _dense(qt, "qt", torch.uint8, (G, k, fp8_padded(n)))
        _dense(scale_t, "scale_t", torch.float32, (G, fp8_blocks(k), fp8_blocks(n)))
    st = lib().ctr_fp8_quantize_blocks(_ptr(w), DTYPES[w.dtype], G, n, k, _ptr(q), _ptr(scale), _ptr(qt),
                                       _ptr(scale_t), *_room(ws), _stream(stream))
    _ok("ctr_fp8_quantize_blocks", st)


def ctr_fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                   offsets: Optional[torch.Tensor], out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """out[r] = W_g a_r for the rows of each group, from row codes a [rows, P(k)] and block codes b [groups, n, P(k)]."""
    if stream is None and _took("ctr_fp8_matmul", _usual().fp8_matmul(a, a_scale, b, b_scale, offsets, out, ws)):
        return
    rows, n, ldo = _mat(out, "out")
    _want(isinstance(b, torch.Tensor) and b.dim() == 3, "b must be [groups, n, padded k]")
    G, bn, kp = b.shape
    _want(bn == n, "out must have a column for each row of b")
    _want(kp % 128 == 0 and kp > 0, "codes must have whole blocks of 128")
    _dense(a, "a", _U8, (rows, kp))
    _dense(b, "b", _U8, (G, n, kp))
    lds = _like(a_scale, "a_scale", kp // 128, rows, _F32)
    _dense(b_scale, "b_scale", _F32, (G, (n + 127) // 128, kp // 128))
    if offsets is not None:
        _dense(offsets, "offsets", _I32, (G + 1,))
    st = lib().ctr_fp8_matmul(a.data_ptr(), a_scale.data_ptr(), lds, b.data_ptr(), b_scale.data_ptr(), _ptr(offsets),
                              rows, G, n, kp, out.data_ptr(), DTYPES[out.dtype], ldo, *_room(ws),
                              _stream(stream))
    if st:
        _ok("ctr_fp8_matmul", st)


def ctr_fp8_matmul_wgrad(d: torch.Tensor, d_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                         offsets: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, rows: Optional[int] = None,
                         stream=None) -> None:
    """out[g] = d_g^T x_g [n, k] from column codes of d (by column) and of x (by block).

    `rows` is the row count the codes were made for (it fixes their padding); by
    default the largest that has the codes' padded length."""
    if stream is None and _took("ctr_fp8_matmul_wgrad", _usual().fp8_matmul_wgrad(d, d_scale, x, x_scale, offsets,
                out, ws, rows)):
        return
    _want(isinstance(out, torch.Tensor) and out.dim() == 3 and out.dtype in DTYPES, "out must be [groups, n, k]")
    G, n, k = out.shape
    _dense(out, "out", out.dtype, (G, n, k))
    _want(isinstance(d, torch.Tensor) and d.dim() == 2, "d must be a matrix")
    padded = d.shape[1]
    if rows is None:
        rows = _rows_of_padding(padded, G)
    _want(fp8_padded_rows(rows, G) == padded, f"codes of {rows} rows in {G} groups are {fp8_padded_rows(rows, G)} long")
    _dense(d, "d", torch.uint8, (n, padded))
    _dense(x, "x", torch.uint8, (k, padded))
    _dense(d_scale, "d_scale", torch.float32, (padded // 128, n))
    _dense(x_scale, "x_scale", torch.float32, (fp8_blocks(k), padded // 128))
    _dense(offsets, "offsets", torch.int32, (G + 1,))
    st = lib().ctr_fp8_matmul_wgrad(_ptr(d), _ptr(d_scale), _ptr(x), _ptr(x_scale), _ptr(offsets), rows, G, n, k,
                                    _ptr(out), DTYPES[out.dtype], *_room(ws), _stream(stream))
    _ok("ctr_fp8_matmul_wgrad", st)


def _rows_of_padding(padded: int, groups: int) -> int:
    """The most rows whose column codes are `padded` long: ctr_fp8_padded_rows is 128 max(1, min((rows + 127
    groups) / 128, rows))."""
    tiles = padded // 128
    return max(tiles, (tiles + 1) * 128 - 1 - 127 * groups)


# -- gradient clipping ----------------------------------------------------------
class GradList:
    """Host arrays of ctr_clip_grads for a list of tensors (built once, kept alive with them)."""

    def __init__(self, grads, outs):
        n = len(grads)
        self.n, self.grads, self.outs = n, list(grads), None if outs is None else list(outs)
        self.device = self.grads[0].get_device() if n else None
        self.ptrs = (C.c_void_p * max(1, n))(*[t.data_ptr() for t in grads])
        self.out_ptrs = None if outs is None else (C.c_void_p * max(1, n))(*[t.data_ptr() for t in outs])
        self.dtypes = (C.c_int32 * max(1, n))(*[DTYPES[t.dtype] for t in grads])
        self.counts = (C.c_int64 * max(1, n))(*[t.numel() for t in grads])
        self.addresses = tuple(None if a is None else C.addressof(a)
                               for a in (self.ptrs, self.out_ptrs, self.dtypes, self.counts))


def grad_list(grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None) -> GradList:
    """A list for ctr_clip_grads: dense fp32 or bf16 CUDA tensors, and where the clipped ones go
    (`grads` itself for in place; None for the norm alone)."""
    devices = set()
    for t in list(grads) + list(outs or []):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in DTYPES or not t.is_contiguous():
            raise ValueError("gradients must be contiguous fp32 or bf16 CUDA tensors")
        devices.add(t.get_device())
    _want(len(devices) <= 1, "gradients must be on one device")
    if outs is not None:
        _want(len(outs) == len(grads), "outs must be as many as grads")
        for g, o in zip(grads, outs):
            _want(g.dtype == o.dtype and g.numel() == o.numel(), "outs must have the types and sizes of grads")
    return GradList(grads, outs)


def ctr_clip_grads_workspace_size() -> int:
    return int(lib().ctr_clip_grads_workspace_size())


def ctr_clip_grads(grads: GradList, max_norm: float, norm: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """The global norm of a grad_list into norm (fp32 [1]), and its outs = grads * min(1, max_norm / norm)."""
    if stream is None and _took("ctr_clip_grads", _usual().clip_grads(*grads.addresses, grads.n, grads.device, max_norm,
                                                                      norm, ws)):
        return
    _here(grads.device, "the list of gradients")
    _dense(norm, "norm", torch.float32, (1,))
    st = lib().ctr_clip_grads(*grads.addresses, grads.n, max_norm,
                              norm.data_ptr(), *_room(ws), _stream(stream))
    if st:
        _ok("ctr_clip_grads", st)


# ---------------------------------------------------------------------------
# layers around the experts
# ---------------------------------------------------------------------------
MAX_NORM_WIDTH = 16384


def _like_or_none(t: Optional[torch.Tensor], what: str, rows: int, cols: int, dtype):
    """(address, row stride) of an optional matrix of the given shape and type."""
    return (None, 0) if t is None else (t.data_ptr() if isinstance(t, torch.Tensor) else None,
                                        _like(t, what, rows, cols, dtype))


def _dense_or_none(t: Optional[torch.Tensor], what: str, dtype, shape):
    """Address of an optional dense tensor."""
    if t is None:
        return None
    _dense(t, what, dtype, shape)
    return t.data_ptr()


MAX_GROUPS = 32
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


def ctr_expert_route_balanced(scores: torch.Tensor, k: int, score: int, bias: Optional[torch.Tensor], groups: int,
                              group_k: int, renormalize: bool, factor: float, expert: torch.Tensor,
                              weight: torch.Tensor, slot: torch.Tensor, token: torch.Tensor, offsets: torch.Tensor,
                              ws: torch.Tensor, stream=None) -> None:
    """ctr_expert_route by the largest score function + bias within the best groups of experts."""
    if stream is None and _took("ctr_expert_route_balanced", _usual().expert_route_balanced(
            scores, k, score, bias, groups, group_k, renormalize, factor, expert, weight, slot, token, offsets, ws)):
        return
    T, E, ld = _mat(scores, "scores")
    pb = _dense_or_none(bias, "bias", _F32, (E,))
    tk = (T, k)
    _dense(expert, "expert", _I32, tk)
    _dense(weight, "weight", _F32, tk)
    _dense(slot, "slot", _I32, tk)
    _dense(token, "token", _I32, (T * k,))
    _dense(offsets, "offsets", _I32, (E + 1,))
    _ok("ctr_expert_route_balanced", lib().ctr_expert_route_balanced(
        scores.data_ptr(), DTYPES[scores.dtype], T, E, ld, k, score, pb, groups, group_k, 1 if renormalize else 0, factor,
        expert.data_ptr(), weight.data_ptr(), slot.data_ptr(), token.data_ptr(), offsets.data_ptr(), *_room(ws),
        _stream(stream)))


def ctr_expert_route_balanced_bwd(dweight: torch.Tensor, scores: torch.Tensor, score: int, renormalize: bool,
                                  factor: float, expert: torch.Tensor, dscores: torch.Tensor, ws: torch.Tensor,
                                  stream=None) -> None:
    if stream is None and _took("ctr_expert_route_balanced_bwd", _usual().expert_route_balanced_bwd(
            dweight, scores, score, renormalize, factor, expert, dscores, ws)):
        return
    T, E, ld = _mat(scores, "scores")
    _want(isinstance(expert, torch.Tensor) and expert.dim() == 2, "expert must be a matrix")
    k = expert.shape[1]
    _dense(expert, "expert", _I32, (T, k))
    _dense(dweight, "dweight", _F32, (T, k))
    ldd = _like(dscores, "dscores", T, E, scores.dtype)
    _ok("ctr_expert_route_balanced_bwd", lib().ctr_expert_route_balanced_bwd(
        dweight.data_ptr(), scores.data_ptr(), DTYPES[scores.dtype], T, E, ld, k, score, 1 if renormalize else 0, factor,
        expert.data_ptr(), dscores.data_ptr(), ldd, *_room(ws), _stream(stream)))


ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_SIGMOID = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "sigmoid": ACT_SIGMOID}


def ctr_dense_workspace_size(rows: int, n: int, k: int, dtype: torch.dtype, train: bool = False,
                             packed: Optional[bool] = None) -> int:
    """Workspace of a dense layer's calls.  packed: rows of some matrix do not start at multiples of 16 bytes (by
    default, whether those of dense bf16 matrices with n or k columns do not)."""
    if packed is None:
        packed = n % 8 != 0 or k % 8 != 0
    return int(lib().ctr_dense_workspace_size(rows, n, k, DTYPES[dtype], 1 if train else 0, 1 if packed else 0))


def ctr_dense(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor], act: int, residual: Optional[torch.Tensor],
              y: torch.Tensor, pre: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    """y = act(x w^T + bias) + residual; pre gets what the activation is of."""
    if stream is None and _took("ctr_dense", _usual().dense(x, w, bias, act, residual, y, pre, ws)):
        return
    rows, k, ldx = _mat(x, "x")
    n, wk, ldw = _mat(w, "w", (x.dtype,))
    _want(wk == k, "w must have as many columns as x")
    pb = _dense_or_none(bias, "bias", x.dtype, (n,))
    pr, ldr = _like_or_none(residual, "residual", rows, n, x.dtype)
    ldy = _like(y, "y", rows, n, x.dtype)
    pp, ldp = _like_or_none(pre, "pre", rows, n, x.dtype)
    _ok("ctr_dense", lib().ctr_dense(x.data_ptr(), DTYPES[x.dtype], rows, k, ldx, w.data_ptr(), n, ldw, pb, act, pr, ldr,
                                     y.data_ptr(), ldy, pp, ldp, *_room(ws), _stream(stream)))


def ctr_dense_bwd(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, pre: Optional[torch.Tensor], act: int,
                  dx: Optional[torch.Tensor], dw: Optional[torch.Tensor], dbias: Optional[torch.Tensor],
                  ws: torch.Tensor, stream=None) -> None:
    """Gradients of x, w and bias, each where it is given; the residual's is dy."""
    if stream is None and _took("ctr_dense_bwd", _usual().dense_bwd(dy, x, w, pre, act, dx, dw, dbias, ws)):
        return
    rows, n, ld_dy = _mat(dy, "dy")
    xr, k, ldx = _mat(x, "x", (dy.dtype,))
    _want(xr == rows, "x must have as many rows as dy")
    ldw = _like(w, "w", n, k, dy.dtype)
    _want(act == ACT_NONE or pre is not None, "an activation's gradient needs pre")
    pp, ldp = _like_or_none(pre, "pre", rows, n, dy.dtype)
    px, ld_dx = _like_or_none(dx, "dx", rows, k, dy.dtype)
    some = dw if dw is not None else dbias
    grad = some.dtype if isinstance(some, torch.Tensor) else dy.dtype
    _want(grad in (torch.float32, dy.dtype), "dw and dbias must be fp32 or of dy's type")
    pw, ld_dw = _like_or_none(dw, "dw", n, k, grad)
    pb = _dense_or_none(dbias, "dbias", grad, (n,))
    _ok("ctr_dense_bwd", lib().ctr_dense_bwd(dy.data_ptr(), DTYPES[dy.dtype], rows, n, ld_dy, x.data_ptr(), k, ldx,
                                             w.data_ptr(), ldw, pp, ldp, act, px, ld_dx, DTYPES[grad], pw, ld_dw, pb,
                                             *_room(ws), _stream(stream)))


def ctr_rms_norm_workspace_size(rows: int, d: int) -> int:
    return int(lib().ctr_rms_norm_workspace_size(rows, d))


def ctr_rms_norm(x: torch.Tensor, residual: Optional[torch.Tensor], gamma: Optional[torch.Tensor], eps: float,
                 s: Optional[torch.Tensor], y: Optional[torch.Tensor], q: Optional[torch.Tensor],
                 scale: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    """s = x + residual, and its norm times gamma as values y or as row codes q with their scales, or both."""
    if stream is None and _took("ctr_rms_norm", _usual().rms_norm(x, residual, gamma, eps, s, y, q, scale, ws)):
        return
    rows, d, ldx = _mat(x, "x")
    pr, ldr = _like_or_none(residual, "residual", rows, d, x.dtype)
    pg = _dense_or_none(gamma, "gamma", _F32, (d,))
    ps, lds = _like_or_none(s, "s", rows, d, x.dtype)
    py, ldy = _like_or_none(y, "y", rows, d, x.dtype)
    _want((q is None) == (scale is None), "q and scale go together")
    pq = _dense_or_none(q, "q", _U8, (rows, fp8_padded(d)))
    pc, ldc = _like_or_none(scale, "scale", fp8_blocks(d), rows, _F32)
    _ok("ctr_rms_norm", lib().ctr_rms_norm(x.data_ptr(), DTYPES[x.dtype], rows, d, ldx, pr, ldr, pg, eps, ps, lds, py,
                                           ldy, pq, pc, ldc, *_room(ws), _stream(stream)))


def ctr_rms_norm_bwd(dy: torch.Tensor, ds: Optional[torch.Tensor], s: torch.Tensor, gamma: Optional[torch.Tensor],
                     eps: float, dx: torch.Tensor, dgamma: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    """dx = ds + the norm's gradient by dy, and gamma's; s is what the forward wrote (x without a residual)."""
    if stream is None and _took("ctr_rms_norm_bwd", _usual().rms_norm_bwd(dy, ds, s, gamma, eps, dx, dgamma, ws)):
        return
    rows, d, ld_dy = _mat(dy, "dy")
    pd, ldd = _like_or_none(ds, "ds", rows, d, dy.dtype)
    ld_s = _like(s, "s", rows, d, dy.dtype)
    pg = _dense_or_none(gamma, "gamma", _F32, (d,))
    ld_dx = _like(dx, "dx", rows, d, dy.dtype)
    po = _dense_or_none(dgamma, "dgamma", _F32, (d,))
    _ok("ctr_rms_norm_bwd", lib().ctr_rms_norm_bwd(dy.data_ptr(), DTYPES[dy.dtype], rows, d, ld_dy, pd, ldd, s.data_ptr(),
                                                   ld_s, pg, eps, dx.data_ptr(), ld_dx, po, *_room(ws),
                                                   _stream(stream)))
