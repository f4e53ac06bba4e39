"""Python binding of libvsa.so (include/vsa.h).

Argument marshalling only: every step of the attention path runs in the
library's CUDA kernels. PyTorch provides device memory and streams. The
functions named like the C entry points (``vsa_build_block_map``,
``vsa_mask_to_index``, ``vsa_fwd``, ``vsa_bwd``, ...) take torch tensors
and pass their device pointers; ``Plan`` wraps a problem's descriptor,
workspace and index buffers for convenient use. There is no fallback: a
missing library raises.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import math
import os
import weakref
from typing import Optional

import torch

from . import build as _build

LAYOUTS = {"bhsd": 0, "bshd": 1, "tnd": 2}
DTYPES = {torch.bfloat16: 0, torch.float16: 1}

STATUS = {0: "VSA_OK", 1: "VSA_ERR_NULL", 2: "VSA_ERR_SHAPE", 3: "VSA_ERR_DTYPE", 4: "VSA_ERR_LAYOUT",
          5: "VSA_ERR_UNSUPPORTED", 6: "VSA_ERR_MISSING_SEQLENS", 7: "VSA_ERR_WORKSPACE",
          8: "VSA_ERR_CUDA", 9: "VSA_ERR_DEVICE", 10: "VSA_ERR_SCRATCH"}

EXPORTS = ("vsa_workspace_size", "vsa_build_block_map", "vsa_build_block_map_static", "vsa_mask_to_index",
           "vsa_fwd", "vsa_bwd",
           "vsa_status_string", "vsa_last_cuda_error", "vsa_device_status", "vsa_profile_enable", "vsa_profile_count",
           "vsa_profile_name", "vsa_profile_ms", "vsa_profile_reset", "vsa_launch_count",
           "vsa_tile_3d_count", "vsa_tile_3d", "vsa_untile_3d", "vsa_gate_grad",
           "vsa_mask_to_index_blocks", "vsa_fwd_blocks", "vsa_bwd_blocks", "vsa_check_wait_timeout",
           "vsa_train_step_host_size", "vsa_train_step_host", "vsa_fwd_step_host", "vsa_step_host_status",
           "vsa_check_inputs", "vsa_head_slice", "vsa_fwd_reuse", "vsa_bwd_reuse",
           "vsa_paged_workspace_size", "vsa_paged_append", "vsa_page_select", "vsa_paged_attn",
           "vsa_paged8_append", "vsa_paged8_attn", "vsa_paged_read", "vsa_paged_weigh_workspace_size",
           "vsa_paged_attn_weigh", "vsa_page_evict", "vsa_rope_init", "vsa_rope_apply", "vsa_rope_table")

REUSE_QK_MEANS, REUSE_V_MEANS = 1, 2  # vsa_fwd_reuse / vsa_bwd_reuse mask bits


class VsaError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        msg = f"{fn} failed: {STATUS.get(code, code)} ({_lib.vsa_status_string(code).decode()})"
        if code == 8:
            msg += f": {_lib.vsa_last_cuda_error().decode()}"
        super().__init__(msg)


class VsaDesc(C.Structure):
    _fields_ = [("layout", C.c_int32), ("dtype", C.c_int32), ("B", C.c_int32), ("Hq", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("Sq", C.c_int32), ("Skv", C.c_int32),
                ("tile_q", C.c_int32), ("tile_kv", C.c_int32), ("nQ", C.c_int32), ("nKV", C.c_int32),
                ("cu_seqlens_q", C.c_void_p), ("cu_seqlens_kv", C.c_void_p), ("scale", C.c_float)]


class PagedDesc(C.Structure):
    _fields_ = [("layout", C.c_int32), ("dtype", C.c_int32), ("B", C.c_int32), ("Hq", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("page", C.c_int32), ("num_pages", C.c_int32),
                ("max_pages", C.c_int32), ("page_stride", C.c_int64), ("page_table", C.c_void_p),
                ("seq_lens", C.c_void_p), ("scale", C.c_float)]


class RopeDesc(C.Structure):
    _fields_ = [("n_axes", C.c_int32), ("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("axis", C.c_uint8 * 64),
                ("turn", C.c_uint64 * 64)]


class RopeTensor(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("heads", C.c_int32), ("x_batch", C.c_int64),
                ("x_token", C.c_int64), ("x_head", C.c_int64), ("y_batch", C.c_int64), ("y_token", C.c_int64),
                ("y_head", C.c_int64)]


_lib = None
P = C.c_void_p


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libvsa.so (built in-tree by __graft_entry__.build()); raise if absent."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libvsa.so is not built ({path}); run __graft_entry__.build()")
        L = C.CDLL(path)
        L.vsa_workspace_size.restype = C.c_size_t
        L.vsa_workspace_size.argtypes = [C.POINTER(VsaDesc), C.c_int]
        L.vsa_build_block_map.restype = C.c_int
        L.vsa_build_block_map.argtypes = [C.POINTER(VsaDesc), P, P, P, P, C.c_int, C.c_int, P, P, P, C.c_int,
                                          P, P, P, C.c_size_t, P]
        L.vsa_build_block_map_static.restype = C.c_int
        L.vsa_build_block_map_static.argtypes = [C.POINTER(VsaDesc), P, P, P, P, C.c_int, C.c_int, P, P, P,
                                                 C.c_int, P, P, P]
        L.vsa_mask_to_index.restype = C.c_int
        L.vsa_mask_to_index.argtypes = [C.POINTER(VsaDesc), P, P, P, C.c_int, P, P, C.c_int, P, P, P]
        L.vsa_fwd.restype = C.c_int
        L.vsa_fwd.argtypes = [C.POINTER(VsaDesc), P, P, P, P, P, C.c_int, P, P, P, P, P, P, P, C.c_size_t, P]
        L.vsa_bwd.restype = C.c_int
        L.vsa_bwd.argtypes = [C.POINTER(VsaDesc), P, P, P, P, P, P, P, P, C.c_int, P, P, P, P, P, P, P, P, P,
                              C.c_size_t, P]
        L.vsa_fwd_reuse.restype = C.c_int
        L.vsa_fwd_reuse.argtypes = [C.POINTER(VsaDesc), P, P, P, P, P, C.c_int, P, P, P, P, P, P, C.c_int, P,
                                    C.c_size_t, P]
        L.vsa_bwd_reuse.restype = C.c_int
        L.vsa_bwd_reuse.argtypes = [C.POINTER(VsaDesc), P, P, P, P, P, P, P, P, C.c_int, P, P, P, P, P, P, P, P,
                                    C.c_int, P, C.c_size_t, P]
        L.vsa_status_string.restype = C.c_char_p
        L.vsa_status_string.argtypes = [C.c_int]
        L.vsa_last_cuda_error.restype = C.c_char_p
        L.vsa_device_status.restype = C.c_int
        L.vsa_device_status.argtypes = [P, P, C.POINTER(C.c_int32)]
        L.vsa_profile_enable.argtypes = [C.c_int]
        L.vsa_profile_count.restype = C.c_int
        L.vsa_profile_name.restype = C.c_char_p
        L.vsa_profile_name.argtypes = [C.c_int]
        L.vsa_profile_ms.restype = C.c_float
        L.vsa_profile_ms.argtypes = [C.c_int]
        L.vsa_launch_count.restype = C.c_longlong
        L.vsa_check_wait_timeout.restype = C.c_int
        L.vsa_check_wait_timeout.argtypes = [P, C.c_ulonglong, P, P]
        L.vsa_mask_to_index_blocks.restype = C.c_int
        L.vsa_mask_to_index_blocks.argtypes = [C.POINTER(VsaDesc), C.c_int, C.c_int, P, P, P, C.c_int, P, P, P, P,
                                               C.c_int, P, P, P, P]
        L.vsa_fwd_blocks.restype = C.c_int
        L.vsa_fwd_blocks.argtypes = [C.POINTER(VsaDesc), C.c_int, P, P, P, P, P, P, C.c_int, P, P, P, P, P,
                                     C.c_size_t, P]
        L.vsa_bwd_blocks.restype = C.c_int
        L.vsa_bwd_blocks.argtypes = [C.POINTER(VsaDesc), C.c_int, P, P, P, P, P, P, P, P, P, C.c_int, P, P, P, P,
                                     P, P, P, P, P, C.c_size_t, P]
        L.vsa_gate_grad.restype = C.c_int
        L.vsa_gate_grad.argtypes = [C.POINTER(VsaDesc), P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.vsa_tile_3d_count.restype = C.c_int
        L.vsa_tile_3d_count.argtypes = [C.c_int] * 6
        L.vsa_tile_3d.restype = C.c_int
        L.vsa_tile_3d.argtypes = [C.c_int] * 8 + [P, P, P, P]
        L.vsa_untile_3d.restype = C.c_int
        L.vsa_untile_3d.argtypes = [C.c_int] * 8 + [P, P, P]
        L.vsa_train_step_host_size.restype = C.c_size_t
        L.vsa_train_step_host_size.argtypes = [C.POINTER(VsaDesc), C.c_int, C.c_int, C.c_int]
        L.vsa_train_step_host.restype = C.c_int
        L.vsa_train_step_host.argtypes = [C.POINTER(VsaDesc), C.c_int, P, P, P, P, P, P, P, C.c_int, P, P, P, P, P,
                                          P, C.c_size_t, P]
        L.vsa_step_host_status.restype = C.c_int
        L.vsa_step_host_status.argtypes = [C.POINTER(VsaDesc), C.c_int, C.c_int, C.c_int, P, P, C.POINTER(C.c_int32)]
        L.vsa_check_inputs.restype = C.c_int
        L.vsa_check_inputs.argtypes = [C.POINTER(VsaDesc), P, P, P, P, C.c_int, P, P, P, C.c_size_t, P,
                                       C.POINTER(C.c_int32)]
        L.vsa_head_slice.restype = C.c_int
        L.vsa_head_slice.argtypes = [C.POINTER(VsaDesc), C.c_int, C.c_int, C.POINTER(VsaDesc), C.POINTER(C.c_int32),
                                     C.POINTER(C.c_int32)]
        L.vsa_fwd_step_host.restype = C.c_int
        L.vsa_fwd_step_host.argtypes = [C.POINTER(VsaDesc), C.c_int, P, P, P, P, P, P, C.c_int, P, P, P, C.c_size_t,
                                        P]
        i64 = C.c_int64
        L.vsa_paged_workspace_size.restype = C.c_size_t
        L.vsa_paged_workspace_size.argtypes = [C.POINTER(PagedDesc)]
        L.vsa_paged_append.restype = C.c_int
        L.vsa_paged_append.argtypes = [C.POINTER(PagedDesc), C.c_int, P, i64, P, i64, P, i64, P, P, P, P, P, C.c_int,
                                       C.c_int, C.c_int, P, P, P, P]
        L.vsa_page_select.restype = C.c_int
        L.vsa_page_select.argtypes = [C.POINTER(PagedDesc), P, i64, P, C.c_int, C.c_int, C.c_int, P, P, P, C.c_size_t,
                                      P]
        L.vsa_paged_attn.restype = C.c_int
        L.vsa_paged_attn.argtypes = [C.POINTER(PagedDesc), P, i64, P, P, P, P, C.c_int, P, P, P, C.c_size_t, P]
        L.vsa_paged8_append.restype = C.c_int
        L.vsa_paged8_append.argtypes = [C.POINTER(PagedDesc), C.c_int, P, i64, P, i64, P, i64, P, P, P, P, P, C.c_int,
                                        C.c_int, C.c_int, P, P, P, P, P, P]
        L.vsa_paged8_attn.restype = C.c_int
        L.vsa_paged8_attn.argtypes = [C.POINTER(PagedDesc), P, i64, P, P, P, P, P, P, C.c_int, P, P, P, C.c_size_t, P]
        L.vsa_paged_read.restype = C.c_int
        L.vsa_paged_read.argtypes = [C.POINTER(PagedDesc), C.c_int, P, P, P, P, P, P, P, P]
        L.vsa_paged_weigh_workspace_size.restype = C.c_size_t
        L.vsa_paged_weigh_workspace_size.argtypes = [C.POINTER(PagedDesc)]
        L.vsa_paged_attn_weigh.restype = C.c_int
        L.vsa_paged_attn_weigh.argtypes = [C.POINTER(PagedDesc), P, i64, P, P, P, P, P, P, C.c_int, P, P, P, P, C.c_float,
                                           P, C.c_size_t, P]
        L.vsa_page_evict.restype = C.c_int
        L.vsa_page_evict.argtypes = [C.POINTER(PagedDesc), P, C.c_int, C.c_int, C.c_int, P, P, P, P, P, P, C.c_size_t, P]
        L.vsa_rope_init.restype = C.c_int
        L.vsa_rope_init.argtypes = [C.POINTER(RopeDesc), C.c_int, C.c_int, C.c_int, P, P]
        L.vsa_rope_apply.restype = C.c_int
        L.vsa_rope_apply.argtypes = [C.POINTER(RopeDesc), C.c_int, C.c_int, C.c_int, C.c_int, C.POINTER(RopeTensor),
                                     C.c_int, P, i64, i64, C.c_int, P]
        L.vsa_rope_table.restype = C.c_int
        L.vsa_rope_table.argtypes = [C.POINTER(RopeDesc), C.c_int, P, i64, P, P, P]
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _check(fn, code):
    if code != 0:
        raise VsaError(fn, code)


# ------------------------------------------------------------- raw entry points

def vsa_workspace_size(desc: VsaDesc, with_gate: bool) -> int:
    return int(lib().vsa_workspace_size(C.byref(desc), int(bool(with_gate))))


def vsa_build_block_map(desc, q, k, q_var, kv_var, topk, need_bwd_index, block_map, q_idx, q_cnt, idx_cap,
                        kv_ptr, kv_qidx, workspace, stream=None):
    _check("vsa_build_block_map", lib().vsa_build_block_map(
        C.byref(desc), _p(q), _p(k), _p(q_var), _p(kv_var), int(topk), int(bool(need_bwd_index)),
        _p(block_map), _p(q_idx), _p(q_cnt), int(idx_cap), _p(kv_ptr), _p(kv_qidx), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def vsa_build_block_map_static(desc, q, k, q_var, kv_var, topk, need_bwd_index, block_map, q_idx, q_cnt,
                               idx_cap, kv_ptr, kv_qidx, stream=None):
    """vsa_build_block_map without a workspace: for callers that cannot
    allocate device memory (the scratch is a fixed array in the library)."""
    _check("vsa_build_block_map_static", lib().vsa_build_block_map_static(
        C.byref(desc), _p(q), _p(k), _p(q_var), _p(kv_var), int(topk), int(bool(need_bwd_index)),
        _p(block_map), _p(q_idx), _p(q_cnt), int(idx_cap), _p(kv_ptr), _p(kv_qidx), _stream(stream)))


def vsa_mask_to_index(desc, block_map, q_var, kv_var, need_bwd_index, q_idx, q_cnt, idx_cap, kv_ptr, kv_qidx,
                      stream=None):
    _check("vsa_mask_to_index", lib().vsa_mask_to_index(
        C.byref(desc), _p(block_map), _p(q_var), _p(kv_var), int(bool(need_bwd_index)), _p(q_idx), _p(q_cnt),
        int(idx_cap), _p(kv_ptr), _p(kv_qidx), _stream(stream)))


def vsa_fwd(desc, q, k, v, q_idx, q_cnt, idx_cap, q_var, kv_var, gate, out, lse, o_sparse, workspace,
            stream=None, reuse=0):
    """vsa_fwd (reuse = 0) or vsa_fwd_reuse (reuse: REUSE_* bits)."""
    args = (C.byref(desc), _p(q), _p(k), _p(v), _p(q_idx), _p(q_cnt), int(idx_cap), _p(q_var), _p(kv_var),
            _p(gate), _p(out), _p(lse), _p(o_sparse))
    tail = (_p(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if reuse:
        _check("vsa_fwd_reuse", lib().vsa_fwd_reuse(*args, int(reuse), *tail))
    else:
        _check("vsa_fwd", lib().vsa_fwd(*args, *tail))


def vsa_bwd(desc, dO, q, k, v, o_sparse, lse, q_idx, q_cnt, idx_cap, kv_ptr, kv_qidx, q_var, kv_var, gate,
            dq, dk, dv, workspace, stream=None, reuse=0):
    """vsa_bwd (reuse = 0) or vsa_bwd_reuse (reuse: REUSE_* bits)."""
    args = (C.byref(desc), _p(dO), _p(q), _p(k), _p(v), _p(o_sparse), _p(lse), _p(q_idx), _p(q_cnt),
            int(idx_cap), _p(kv_ptr), _p(kv_qidx), _p(q_var), _p(kv_var), _p(gate), _p(dq), _p(dk), _p(dv))
    tail = (_p(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if reuse:
        _check("vsa_bwd_reuse", lib().vsa_bwd_reuse(*args, int(reuse), *tail))
    else:
        _check("vsa_bwd", lib().vsa_bwd(*args, *tail))


def vsa_gate_grad(desc, dO, q, k, v, q_var, kv_var, dgate, workspace, stream=None):
    _check("vsa_gate_grad", lib().vsa_gate_grad(
        C.byref(desc), _p(dO), _p(q), _p(k), _p(v), _p(q_var), _p(kv_var), _p(dgate), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def vsa_check_inputs(desc, q_var, kv_var, q_idx, q_cnt, idx_cap, kv_ptr, kv_qidx, workspace, stream=None):
    """Opt-in validation of the device-resident arguments (synchronises).
    Returns (status, code): status 0 = all in range, 2 = a check failed
    (code names it), 9 = the status word already held another failure."""
    code = C.c_int32(0)
    st = lib().vsa_check_inputs(C.byref(desc), _p(q_var), _p(kv_var), _p(q_idx), _p(q_cnt), int(idx_cap),
                                _p(kv_ptr), _p(kv_qidx), _p(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream), C.byref(code))
    if st not in (0, 2, 9):
        raise VsaError("vsa_check_inputs", st)
    return int(st), int(code.value)


def vsa_head_slice(desc, groups, g):
    """Slice g of a problem's heads cut into `groups` (GQA groups whole):
    returns (slice descriptor, first query head, first key/value head)."""
    out, q0, kv0 = VsaDesc(), C.c_int32(0), C.c_int32(0)
    _check("vsa_head_slice", lib().vsa_head_slice(C.byref(desc), int(groups), int(g), C.byref(out), C.byref(q0),
                                                  C.byref(kv0)))
    return out, int(q0.value), int(kv0.value)


def vsa_device_status(workspace, stream=None) -> int:
    code = C.c_int32(0)
    lib().vsa_device_status(_p(workspace), _stream(stream), C.byref(code))
    return int(code.value)


def vsa_launch_count() -> int:
    return int(lib().vsa_launch_count())


class profile:
    """Context manager collecting per-kernel CUDA-event times (ms)."""

    def __enter__(self):
        L = lib()
        L.vsa_profile_reset()
        L.vsa_profile_enable(1)
        self.records = []
        return self

    def __exit__(self, *exc):
        L = lib()
        L.vsa_profile_enable(0)
        self.records = [(L.vsa_profile_name(i).decode(), float(L.vsa_profile_ms(i)))
                        for i in range(L.vsa_profile_count())]
        L.vsa_profile_reset()
        return False


# ----------------------------------------------------------------------- Plan

def describe(layout, dtype, B, Hq, Hkv, D, Sq, Skv, tile_q, tile_kv, nQ, nKV, cu_seqlens_q=None, cu_seqlens_kv=None,
             scale=0.0) -> VsaDesc:
    """A vsa_desc: layout "bhsd" | "bshd" | "tnd", dtype torch.bfloat16 |
    torch.float16, sizes as in include/vsa.h (TND offsets: int32 device
    tensors)."""
    return VsaDesc(LAYOUTS[layout], DTYPES[dtype], B, Hq, Hkv, D, Sq, Skv, tile_q, tile_kv, nQ, nKV,
                   _p(cu_seqlens_q), _p(cu_seqlens_kv), float(scale))


class Plan:
    """Descriptor, workspace and index buffers of one problem.

    layout: "bhsd" | "bshd" | "tnd"; sizes as in vsa_desc. For TND pass
    cu_seqlens_q / cu_seqlens_kv (int32 device tensors, [B+1]) and
    max_seqlen_q / max_seqlen_kv (host ints) instead of Sq / Skv per batch.

    With a gate, the plan's methods keep the tile means in its workspace
    between calls (vsa_fwd_reuse / vsa_bwd_reuse). It tracks what its own
    calls pooled and reuses means only for the same tensor objects whose
    torch version counter has not moved. Two things it cannot see must be
    followed by build_block_map before the next gated forward or backward:
    a module-level call that writes plan.workspace with other tensors, and
    a write to q, k or v that bypasses the version counter (through a raw
    pointer or .data).
    """

    def __init__(self, layout, dtype, B, Hq, Hkv, D, tile_q, tile_kv, nQ, nKV, Sq, Skv, idx_cap, gate=False,
                 cu_seqlens_q=None, cu_seqlens_kv=None, q_var=None, kv_var=None, scale=0.0, device="cuda"):
        self.layout, self.dtype = layout, dtype
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, D
        self.tile_q, self.tile_kv, self.nQ, self.nKV = tile_q, tile_kv, nQ, nKV
        self.Sq, self.Skv, self.idx_cap, self.gate = Sq, Skv, idx_cap, gate
        self.cu_q, self.cu_kv = cu_seqlens_q, cu_seqlens_kv
        self.q_var, self.kv_var = q_var, kv_var
        self.device = torch.device(device)
        self.desc = describe(layout, dtype, B, Hq, Hkv, D, Sq, Skv, tile_q, tile_kv, nQ, nKV, cu_seqlens_q,
                             cu_seqlens_kv, scale)
        ws = vsa_workspace_size(self.desc, gate)
        if ws == 0:
            raise ValueError("invalid problem description")
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=self.device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.block_map = torch.zeros((B, Hq, nQ, nKV), dtype=torch.uint8, device=self.device)
        self.q_idx = torch.empty((B, Hq, nQ, idx_cap), **i32)
        self.q_cnt = torch.empty((B, Hq, nQ), **i32)
        self.kv_ptr = torch.empty((B, Hq, nKV + 1), **i32)
        self.kv_qidx = torch.empty((B, Hq, nQ * idx_cap), **i32)
        # Tile means the workspace holds: {"qk": key of (q, k), "v": key of v}
        # as left by the last call that pooled them. A later gated call
        # passes the matching reuse bit only for the same tensor objects,
        # unmodified since: torch bumps a tensor's version counter on every
        # in-place write, through any view of it.
        self._means = {}

    @staticmethod
    def _key(*ts):
        return tuple((weakref.ref(t), t._version) for t in ts)

    def _holds(self, which, *ts):
        key = self._means.get(which)
        return key is not None and len(key) == len(ts) and all(
            r() is t and ver == t._version for (r, ver), t in zip(key, ts))

    def _reuse(self, q, k, v):
        return (REUSE_QK_MEANS if self._holds("qk", q, k) else 0) | (REUSE_V_MEANS if self._holds("v", v) else 0)

    def _pooled(self, q=None, k=None, v=None):
        if q is not None:
            self._means["qk"] = self._key(q, k)
        if v is not None:
            self._means["v"] = self._key(v)

    def lse_shape(self):
        return (self.Hq, self.Sq) if self.layout == "tnd" else (self.B, self.Hq, self.Sq)

    def build_block_map(self, q, k, topk, need_bwd_index=True, stream=None):
        self._means.clear()  # a step starts here: only the means this call pools are kept
        vsa_build_block_map(self.desc, q, k, self.q_var, self.kv_var, topk, need_bwd_index, self.block_map,
                            self.q_idx, self.q_cnt, self.idx_cap, self.kv_ptr if need_bwd_index else None,
                            self.kv_qidx if need_bwd_index else None, self.workspace, stream)
        self._pooled(q, k)

    def mask_to_index(self, block_map, need_bwd_index=True, stream=None):
        self.block_map = block_map
        vsa_mask_to_index(self.desc, block_map, self.q_var, self.kv_var, need_bwd_index, self.q_idx, self.q_cnt,
                          self.idx_cap, self.kv_ptr if need_bwd_index else None,
                          self.kv_qidx if need_bwd_index else None, stream)

    def forward(self, q, k, v, gate=None, out=None, lse=None, o_sparse=None, stream=None):
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty(self.lse_shape(), dtype=torch.float32, device=q.device) if lse is None else lse
        if gate is not None and o_sparse is None:
            o_sparse = torch.empty_like(q)
        reuse = self._reuse(q, k, v) if gate is not None else 0
        if gate is not None:
            self._means.clear()
        vsa_fwd(self.desc, q, k, v, self.q_idx, self.q_cnt, self.idx_cap, self.q_var, self.kv_var, gate, out, lse,
                o_sparse, self.workspace, stream, reuse=reuse)
        if gate is not None:
            self._pooled(q, k, v)
        return out, lse, (o_sparse if o_sparse is not None else out)

    def backward(self, dO, q, k, v, o_sparse, lse, gate=None, dq=None, dk=None, dv=None, stream=None):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        reuse = self._reuse(q, k, v) if gate is not None else 0
        if gate is not None:
            self._means.clear()
        vsa_bwd(self.desc, dO, q, k, v, o_sparse, lse, self.q_idx, self.q_cnt, self.idx_cap, self.kv_ptr,
                self.kv_qidx, self.q_var, self.kv_var, gate, dq, dk, dv, self.workspace, stream, reuse=reuse)
        if gate is not None:
            self._pooled(q, k, v)
        return dq, dk, dv

    def mask_to_index_blocks(self, block_q, block_mask, need_bwd_index=True, stream=None):
        """Index from a query-block mask [B, Hq, nQb, nKV] (block_q rows per
        block); keeps the per-entry block bits for forward_blocks /
        backward_blocks."""
        self.block_q = block_q
        i32 = dict(dtype=torch.int32, device=self.device)
        self.q_sub = torch.empty_like(self.q_idx)
        self.kv_qsub = torch.empty_like(self.kv_qidx)
        _check("vsa_mask_to_index_blocks", lib().vsa_mask_to_index_blocks(
            C.byref(self.desc), int(block_q), int(block_mask.shape[2]), _p(block_mask), _p(self.q_var),
            _p(self.kv_var), int(bool(need_bwd_index)), _p(self.block_map), _p(self.q_idx), _p(self.q_cnt),
            _p(self.q_sub), int(self.idx_cap), _p(self.kv_ptr if need_bwd_index else None),
            _p(self.kv_qidx if need_bwd_index else None), _p(self.kv_qsub if need_bwd_index else None),
            _stream(stream)))

    def forward_blocks(self, q, k, v, out=None, lse=None, stream=None):
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty(self.lse_shape(), dtype=torch.float32, device=q.device) if lse is None else lse
        _check("vsa_fwd_blocks", lib().vsa_fwd_blocks(
            C.byref(self.desc), int(self.block_q), _p(q), _p(k), _p(v), _p(self.q_idx), _p(self.q_cnt),
            _p(self.q_sub), int(self.idx_cap), _p(self.q_var), _p(self.kv_var), _p(out), _p(lse),
            _p(self.workspace), self.workspace.numel() * self.workspace.element_size(), _stream(stream)))
        return out, lse

    def backward_blocks(self, dO, q, k, v, out, lse, dq=None, dk=None, dv=None, stream=None):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        _check("vsa_bwd_blocks", lib().vsa_bwd_blocks(
            C.byref(self.desc), int(self.block_q), _p(dO), _p(q), _p(k), _p(v), _p(out), _p(lse), _p(self.q_idx),
            _p(self.q_cnt), _p(self.q_sub), int(self.idx_cap), _p(self.kv_ptr), _p(self.kv_qidx), _p(self.kv_qsub),
            _p(self.q_var), _p(self.kv_var), _p(dq), _p(dk), _p(dv), _p(self.workspace),
            self.workspace.numel() * self.workspace.element_size(), _stream(stream)))
        return dq, dk, dv

    def gate_grad(self, dO, q, k, v, dgate=None, stream=None):
        """dgate = dO (*) c (the plan must have been made with gate=True)."""
        dgate = torch.empty_like(dO) if dgate is None else dgate
        self._means.clear()
        vsa_gate_grad(self.desc, dO, q, k, v, self.q_var, self.kv_var, dgate, self.workspace, stream)
        self._pooled(q, k, v)
        return dgate

    def check_inputs(self, with_index=True, with_bwd_index=True, stream=None):
        """vsa_check_inputs on this plan's tile fills / offsets and (when
        asked) its index buffers; returns (status, code)."""
        return vsa_check_inputs(self.desc, self.q_var, self.kv_var, self.q_idx if with_index else None,
                                self.q_cnt if with_index else None, self.idx_cap,
                                self.kv_ptr if with_bwd_index else None, self.kv_qidx if with_bwd_index else None,
                                self.workspace, stream)

    def device_status(self, stream=None) -> int:
        return vsa_device_status(self.workspace, stream)

    def _staging(self, groups, topk, gated):
        """Zeroed device staging memory for the host-buffer steps (kept and
        reused; its status words start at 0)."""
        need = int(lib().vsa_train_step_host_size(C.byref(self.desc), int(groups), int(topk), int(gated)))
        if need == 0:
            raise ValueError("invalid descriptor, groups or topk for the host-buffer step")
        buf = getattr(self, "_host_step_buf", None)
        if buf is None or buf.numel() < need:
            buf = self._host_step_buf = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self._host_step_args = (int(groups), int(topk), int(gated))
        return buf, need

    def host_step_status(self, stream=None) -> int:
        """vsa_step_host_status for the last host-buffer step: synchronises
        and returns the first failure code of its staging slots (0 = none)."""
        groups, topk, gated = self._host_step_args
        code = C.c_int32(0)
        rc = lib().vsa_step_host_status(C.byref(self.desc), groups, topk, gated, _p(self._host_step_buf),
                                        _stream(stream), C.byref(code))
        if rc not in (0, 9):
            raise VsaError("vsa_step_host_status", rc)
        return int(code.value)

    def train_step_host(self, q, k, v, dO, topk, groups, gate=None, out=None, lse=None, dq=None, dk=None,
                        dv=None, stream=None):
        """vsa_train_step_host: one step (block map, forward, backward; with
        a gate also the gated compression branch) from host tensors (pin
        them for overlap), heads in `groups` slices whose copies overlap the
        kernels. Outputs are host tensors (allocated pinned when not given);
        `stream` is left ordered after the last copy back, so synchronise it
        before reading them. Returns (out, lse, dq, dk, dv); out / lse only
        if passed in."""
        buf, need = self._staging(groups, topk, gate is not None)
        dq = torch.empty(q.shape, dtype=q.dtype, pin_memory=True) if dq is None else dq
        dk = torch.empty(k.shape, dtype=k.dtype, pin_memory=True) if dk is None else dk
        dv = torch.empty(v.shape, dtype=v.dtype, pin_memory=True) if dv is None else dv
        for t in (q, k, v, dO, gate, out, lse, dq, dk, dv):
            if t is not None and (t.is_cuda or not t.is_contiguous()):
                raise ValueError("vsa_train_step_host takes contiguous host tensors")
        _check("vsa_train_step_host", lib().vsa_train_step_host(
            C.byref(self.desc), int(groups), _p(q), _p(k), _p(v), _p(dO), _p(gate), _p(self.q_var), _p(self.kv_var),
            int(topk), _p(out), _p(lse), _p(dq), _p(dk), _p(dv), _p(buf), need, _stream(stream)))
        return out, lse, dq, dk, dv

    def fwd_step_host(self, q, k, v, topk, groups, gate=None, out=None, lse=None, stream=None):
        """vsa_fwd_step_host: block map and forward from host tensors, head
        slices overlapped with the copies; returns host (out, lse) (out
        allocated pinned when not given; lse only if passed in)."""
        buf, need = self._staging(groups, topk, gate is not None)
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True) if out is None else out
        for t in (q, k, v, gate, out, lse):
            if t is not None and (t.is_cuda or not t.is_contiguous()):
                raise ValueError("vsa_fwd_step_host takes contiguous host tensors")
        _check("vsa_fwd_step_host", lib().vsa_fwd_step_host(
            C.byref(self.desc), int(groups), _p(q), _p(k), _p(v), _p(gate), _p(self.q_var), _p(self.kv_var),
            int(topk), _p(out), _p(lse), _p(buf), need, _stream(stream)))
        return out, lse


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)


# ------------------------------------------------------------- 3D video tiling

def vsa_tile_3d_count(T, H, W, tile=(4, 8, 8)):
    return int(lib().vsa_tile_3d_count(T, H, W, *tile))


def tile_3d(latent: torch.Tensor, tile=(4, 8, 8), out=None, tile_var=None, stream=None):
    """latent [B, T, H, W, heads, D] (or [..., row] with any trailing shape)
    -> (tiled [B, nTiles * prod(tile), heads, D], tile_var [nTiles] int32)."""
    if not latent.is_contiguous():
        raise ValueError("tile_3d: latent must be contiguous")
    B, T, H, W = latent.shape[:4]
    rest = tuple(latent.shape[4:])
    n = vsa_tile_3d_count(T, H, W, tile)
    slots = n * tile[0] * tile[1] * tile[2]
    row_bytes = latent[0, 0, 0, 0].numel() * latent.element_size()
    if out is None:
        out = torch.empty((B, slots) + rest, dtype=latent.dtype, device=latent.device)
    if tile_var is None:
        tile_var = torch.empty(n, dtype=torch.int32, device=latent.device)
    _check("vsa_tile_3d", lib().vsa_tile_3d(B, T, H, W, row_bytes, *tile, _p(latent), _p(out),
                                            _p(tile_var), _stream(stream)))
    return out, tile_var


def untile_3d(tiled: torch.Tensor, grid, tile=(4, 8, 8), out=None, stream=None):
    """tiled [B, nTiles * prod(tile), ...] -> latent [B, T, H, W, ...] for grid = (T, H, W)."""
    if not tiled.is_contiguous():
        raise ValueError("untile_3d: tiled must be contiguous")
    T, H, W = grid
    B = tiled.shape[0]
    rest = tuple(tiled.shape[2:])
    row_bytes = tiled[0, 0].numel() * tiled.element_size()
    if out is None:
        out = torch.empty((B, T, H, W) + rest, dtype=tiled.dtype, device=tiled.device)
    _check("vsa_untile_3d", lib().vsa_untile_3d(B, T, H, W, row_bytes, *tile, _p(tiled), _p(out),
                                                _stream(stream)))
    return out


# ---------------------------------------------- rotary positions, several axes

class AxialRope:
    """Rotary positions with several axes (include/vsa.h): queries and keys of
    image and video tokens, turned by their frame, row and column.

    dims: rotated dims of each axis (even; together a multiple of 16, up to
    128). The head's pairs, (2i, 2i + 1) when interleaved, else (i, i +
    rot_dim / 2), go to the axes in this order; pair j of an axis of n dims
    turns by base ** (-2 j / n) * scale radians per step of the axis (scale: a
    number, or one per axis, e.g. the ratio of two frame rates). freqs: the
    radians per step of every pair instead, at most 1024 each; axes: the axis
    of every pair, instead of the order of dims.

    The calls run on the device of their tensors, with the rules for streams of
    the rest of this module. They record no gradient (tensors that require one
    are refused while gradients are recorded): backward() gives it.
    """

    def __init__(self, dims, base=10000.0, scale=1.0, interleaved=False, freqs=None, axes=None):
        dims = [int(n) for n in dims]
        if not 1 <= len(dims) <= 4 or any(n < 0 or n % 2 for n in dims):
            raise ValueError(f"dims: even numbers for 1 to 4 axes, not {dims}")
        self.dims, self.rot_dim, self.interleaved = tuple(dims), sum(dims), bool(interleaved)
        pairs = self.rot_dim // 2
        if self.rot_dim % 16 or not 0 < self.rot_dim <= 128:
            raise ValueError(f"dims: their sum must be a multiple of 16 up to 128, not {self.rot_dim}")
        scales = [float(scale)] * len(dims) if isinstance(scale, (int, float)) else [float(x) for x in scale]
        if len(scales) != len(dims):
            raise ValueError("scale: a number, or one for each axis")
        if freqs is None:
            if not base > 0:
                raise ValueError(f"base: must be positive, not {base}")
            freqs = [float(base) ** (-2.0 * j / n) * x for n, x in zip(dims, scales) for j in range(n // 2)]
        elif any(x != 1.0 for x in scales):
            raise ValueError("scale: freqs hold it already")
        if axes is None:
            axes = [a for a, n in enumerate(dims) for _ in range(n // 2)]
        freqs, axes = [float(f) for f in freqs], [int(a) for a in axes]
        if len(freqs) != pairs or len(axes) != pairs:
            raise ValueError(f"freqs, axes: one for each of the {pairs} pairs")
        if not all(abs(f) <= 1024 for f in freqs) or not all(0 <= a < len(dims) for a in axes):
            raise ValueError("freqs: at most 1024 radians per step; axes: those of dims")
        self.freqs, self.axes = tuple(freqs), tuple(axes)
        self.desc = RopeDesc()
        L = lib()
        _check("vsa_rope_init", L.vsa_rope_init(C.byref(self.desc), len(dims), self.rot_dim, int(self.interleaved),
                                                (C.c_int32 * pairs)(*axes), (C.c_double * pairs)(*freqs)))
        entry = lambda f: C.cast(f, C.c_void_p).value  # noqa: E731
        self._calls = _paged_binding().Rope(C.addressof(self.desc), entry(L.vsa_rope_apply), entry(L.vsa_rope_table),
                                            _check)

    def _apply(self, q, k, positions, layout, q_out, k_out, stream, inverse):
        if layout not in LAYOUTS:
            raise ValueError(f"layout: bshd, bhsd or tnd, not {layout}")
        if stream is not None:
            if torch.is_tensor(q) and stream.device != q.device:
                raise ValueError(f"stream: expected one of {q.device}, got {stream.device}")
            with torch.cuda.stream(stream):
                return self._calls.apply(q, k, positions, LAYOUTS[layout], q_out, k_out, inverse)
        return self._calls.apply(q, k, positions, LAYOUTS[layout], q_out, k_out, inverse)

    def forward(self, q, k=None, positions=None, layout="bshd", q_out=None, k_out=None, stream=None):
        """vsa_rope_apply: q and k (or q alone) of one set of tokens, "bshd"
        [B, S, H, 128], "bhsd" [B, H, S, 128] or "tnd" [T, H, 128], rotated by
        positions int32 [S, axes] or [B, S, axes] ([T, axes]). Any strides
        that are multiples of 8 with dense last dimensions, so that q and k may
        be parts of a projection's output. q_out, k_out may be q and k; those
        not given are dense. Returns (q, k), or q without k."""
        return self._apply(q, k, positions, layout, q_out, k_out, stream, False)

    def backward(self, dq, dk=None, positions=None, layout="bshd", q_out=None, k_out=None, stream=None):
        """The gradients with respect to forward's inputs from those with
        respect to its outputs: the rotation by the opposite angles."""
        return self._apply(dq, dk, positions, layout, q_out, k_out, stream, True)

    def table(self, positions, cos=None, sin=None, stream=None):
        """vsa_rope_table: (cos, sin), fp32 [T, rot_dim / 2], of positions int32
        [T, axes]: what PagedCache.append takes, with the row of each token in
        its own positions argument (torch.arange(T) where each has its own)."""
        if stream is not None:
            if torch.is_tensor(positions) and stream.device != positions.device:
                raise ValueError(f"stream: expected one of {positions.device}, got {stream.device}")
            with torch.cuda.stream(stream):
                return self._calls.table(positions, cos, sin)
        return self._calls.table(positions, cos, sin)


def tile_positions(T, H, W, tile=(4, 8, 8), device="cuda"):
    """Positions int32 [slots, 3] (frame, row, column) of the tokens that
    tile_3d lays out from a T x H x W latent; zeros in padding slots."""
    at = torch.zeros((1, T, H, W, 4), dtype=torch.int32)
    for axis, n in enumerate((T, H, W)):
        at[..., axis] = torch.arange(n, dtype=torch.int32).view([-1 if a == axis else 1 for a in range(3)])
    at = at.to(device)
    with torch.cuda.device(at.device):
        return tile_3d(at, tile)[0][0, :, :3]


def check_wait_timeout(workspace: torch.Tensor, limit_ns: int = 50_000_000, stream=None) -> int:
    """Run the bounded-wait failure check; returns the device's completed flag
    (0: the wait timed out as it should)."""
    done = torch.full((1,), -1, dtype=torch.int32, device=workspace.device)
    _check("vsa_check_wait_timeout", lib().vsa_check_wait_timeout(_p(workspace), int(limit_ns), _p(done),
                                                                    _stream(stream)))
    return int(done.item())


# ---------------------------------------------------------------- paged cache

_binding = None


def _paged_binding():
    """The extension module behind PagedCache's calls; raise if absent."""
    global _binding
    if _binding is None:
        path = _build.binding()
        if not os.path.exists(path):
            raise RuntimeError(f"the paged cache's binding is not built ({path}); run __graft_entry__.build()")
        spec = importlib.util.spec_from_file_location("paged_binding", path)
        _binding = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_binding)
    return _binding


class PagedCache:
    """One layer's paged key/value cache (the conventions of the paged calls
    in include/vsa.h): appending, page selection, one-token attention, reading
    back, page weights and eviction. The calls give no gradients; tensors that
    require one are refused while gradients are recorded.

    layout: "bshd" (pages [page, Hkv, D]) | "bhsd" (pages [Hkv, page, D]).
    k, v: [num_pages, ...page] tensors of dtype, dense inside a page (halves
    of one buffer are fine); k_mean: fp32 [num_pages, Hkv, D], or False for a
    cache whose pages are never selected. Those not given are allocated
    unless allocate is False (a cache that only selects or evicts needs no k and v).
    kv_dtype: torch.float8_e4m3fn for a cache in 8 bits, whose k and v are of that
    type and have a scale per block of 16 tokens and head, k_scale and v_scale:
    fp32 [num_pages, Hkv, page / 16]; None: dtype.
    weigh: whether the workspace allocated here is large enough for attend with
    page weights (``vsa_paged_weigh_workspace_size`` bytes; one passed in decides by
    its size).
    page_table: int32 [B, max_pages]; seq_lens: int32 [B], the tokens in the
    cache with those of the current step counted in. Both belong to the
    caller, are read by every call when it runs on the device and may be
    shared by all layers (allocated as zeros if not given). Tensors that a
    call writes may not overlap its others. workspace: at
    least ``vsa_paged_workspace_size`` bytes, 256-byte aligned, may be shared by
    caches whose calls run one after another on a stream: the layers of a
    model pass on the first one's, of up to 21 MB and the scores, instead of
    allocating one each. As in the rest of this module, tensors used on a
    stream other than the one they were allocated on, a cache's own among
    them, are kept alive by the caller until that stream is done with them.
    """

    def __init__(self, layout, dtype, B, Hq, Hkv, D, page, num_pages, max_pages, k=None, v=None, k_mean=None,
                 page_table=None, seq_lens=None, scale=0.0, workspace=None, allocate=True, device="cuda",
                 kv_dtype=None, k_scale=None, v_scale=None, weigh=False):
        if layout not in ("bshd", "bhsd"):
            raise ValueError(f"a page's layout is bshd or bhsd, not {layout}")
        if dtype not in DTYPES:
            raise ValueError("the cache holds bf16 or fp16")
        kv_dtype = dtype if kv_dtype is None else kv_dtype
        if kv_dtype not in (dtype, torch.float8_e4m3fn):
            raise ValueError(f"kv_dtype: {dtype} or torch.float8_e4m3fn, not {kv_dtype}")
        eight = kv_dtype == torch.float8_e4m3fn
        for name, n in dict(B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, num_pages=num_pages, max_pages=max_pages).items():
            if not 0 < n < 1 << 31:  # ctypes keeps the low 32 bits of others
                raise ValueError(f"{name}: {n} is out of range")
        given = [t for t in (k, v, k_mean, page_table, seq_lens, workspace, k_scale, v_scale) if torch.is_tensor(t)]
        self.device = given[0].device if given else torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.layout, self.dtype, self.kv_dtype = layout, dtype, kv_dtype
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, D
        self.page, self.num_pages, self.max_pages = page, num_pages, max_pages
        shape = (num_pages, page, Hkv, D) if layout == "bshd" else (num_pages, Hkv, page, D)
        if k is None and v is None and allocate:
            k, v = (torch.zeros(shape, dtype=kv_dtype, device=self.device) for _ in range(2))
        blocks = (num_pages, Hkv, max(1, page // 16))
        if not eight and (k_scale is not None or v_scale is not None):
            raise ValueError("k_scale and v_scale belong to a cache of 8 bits")
        if eight and k is not None:
            if k_scale is None and v_scale is None:
                if any(t is k for t in given):  # its bytes stand for nothing without them
                    raise ValueError("give k_scale and v_scale with k and v")
                k_scale, v_scale = (torch.ones(blocks, device=self.device) for _ in range(2))
            if k_scale is None or v_scale is None:
                raise ValueError("give both k_scale and v_scale, or neither")
        elif eight and (k_scale is not None or v_scale is not None):
            raise ValueError("k_scale and v_scale without k and v")
        if k_mean is None and allocate:
            k_mean = torch.zeros((num_pages, Hkv, D), dtype=torch.float32, device=self.device)
        elif k_mean is False:
            k_mean = None
        i32 = dict(dtype=torch.int32, device=self.device)
        page_table = torch.zeros((B, max_pages), **i32) if page_table is None else page_table
        seq_lens = torch.zeros(B, **i32) if seq_lens is None else seq_lens
        inner = (Hkv * D, D, 1) if layout == "bshd" else (page * D, D, 1)
        stride = 0
        for name, t in (("k", k), ("v", v)):
            if t is None:
                continue
            self._is(name, t, shape, kv_dtype)
            if any(n > 1 and a != b for n, a, b in zip(shape[1:], t.stride()[1:], inner)):
                raise ValueError(f"{name}: a page must be dense")
            if num_pages > 1 and t.stride(0) < page * Hkv * D:
                raise ValueError(f"{name}: pages must not share memory")
            if num_pages > 1 and stride not in (0, t.stride(0)):
                raise ValueError("k and v must have the same page stride")
            stride = t.stride(0) if num_pages > 1 else 0
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        for name, t, shp, dt in (("k_mean", k_mean, (num_pages, Hkv, D), torch.float32),
                                 ("page_table", page_table, (B, max_pages), torch.int32),
                                 ("seq_lens", seq_lens, (B,), torch.int32),
                                 ("k_scale", k_scale, blocks, torch.float32),
                                 ("v_scale", v_scale, blocks, torch.float32)):
            if t is not None:
                self._is(name, t, shp, dt)
                if not t.is_contiguous():
                    raise ValueError(f"{name}: must be contiguous")
        self._tensors = (k, v, k_mean, page_table, seq_lens, k_scale, v_scale)
        self.desc = PagedDesc(LAYOUTS[layout], DTYPES[dtype], B, Hq, Hkv, D, page, num_pages, max_pages, stride,
                              page_table.data_ptr(), seq_lens.data_ptr(), float(scale))
        need = int(lib().vsa_paged_workspace_size(C.byref(self.desc)))
        if need == 0 or (eight and stride % 16):
            raise ValueError("invalid paged-cache description")
        weigh_need = int(lib().vsa_paged_weigh_workspace_size(C.byref(self.desc)))
        if weigh:
            need = weigh_need
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        elif (workspace.device != self.device or not workspace.is_contiguous()
              or workspace.numel() * workspace.element_size() < need):
            raise ValueError(f"workspace: at least {need} contiguous bytes on {self.device} are needed")
        self._workspace = workspace
        # every call passes these addresses on: the tensors behind them are read-only attributes
        at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        entry = lambda f: C.cast(f, C.c_void_p).value  # noqa: E731
        L = lib()
        self._calls = _paged_binding().Calls(
            C.addressof(self.desc), self.device.index if self.device.type == "cuda" else -1, eight, at(k), at(v),
            at(k_scale), at(v_scale), at(k_mean), at(workspace), int(lib().vsa_paged_workspace_size(C.byref(self.desc))),
            weigh_need if workspace.numel() * workspace.element_size() >= weigh_need else 0,
            tuple(entry(f) for f in (L.vsa_paged_append, L.vsa_page_select, L.vsa_paged_attn, L.vsa_paged8_append,
                                     L.vsa_paged8_attn, L.vsa_paged_read, L.vsa_paged_attn_weigh, L.vsa_page_evict)),
            _check)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_mean = property(lambda self: self._tensors[2])
    page_table = property(lambda self: self._tensors[3])
    seq_lens = property(lambda self: self._tensors[4])
    k_scale = property(lambda self: self._tensors[5])
    v_scale = property(lambda self: self._tensors[6])
    workspace = property(lambda self: self._workspace)

    def _is(self, name, t, shape, dtype):
        if t.dtype != dtype or t.device != self.device or t.shape != shape:
            raise ValueError(f"{name}: expected {dtype} {list(shape)} on {self.device}, "
                             f"got {t.dtype} {list(t.shape)} on {t.device}")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name}: the paged calls give no gradient; detach it, or make the cache under "
                             "torch.no_grad()")

    def _on(self, stream):
        """Makes `stream` current, for a call and the outputs it allocates."""
        if stream.device != self.device:
            raise ValueError(f"stream: expected one of {self.device}, got {stream.device}")
        return torch.cuda.stream(stream)

    def append(self, k, v, q=None, cu_seqlens=None, cos=None, sin=None, positions=None, interleaved=False, q_out=None,
               stream=None):
        """vsa_paged_append: k, v [T, Hkv, D] (and q [T, Hq, D]) of the new
        tokens, which seq_lens already counts; cu_seqlens int32 [B+1], None
        for one token per sequence. cos, sin: fp32 [rows, rot_dim / 2], None
        for no rotation. Returns the rotated q (None without q); the rows of
        tokens without a place (of an unused sequence, or behind the last one)
        are not written: zeros only where the q_out given held them."""
        if stream is not None:
            with self._on(stream):
                return self._calls.append(k, v, q, cu_seqlens, cos, sin, positions, interleaved, q_out)
        return self._calls.append(k, v, q, cu_seqlens, cos, sin, positions, interleaved, q_out)

    def select(self, q, topk, keep_first=0, keep_last=1, page_idx=None, page_cnt=None, stream=None):
        """vsa_page_select: the pages that q [B, Hq, D] attends to, as
        (page_idx int32 [B, Hkv, topk], page_cnt int32 [B, Hkv]): one list for
        the query heads of a group, by the sum of their queries."""
        if stream is not None:
            with self._on(stream):
                return self._calls.select(q, topk, keep_first, keep_last, page_idx, page_cnt)
        return self._calls.select(q, topk, keep_first, keep_last, page_idx, page_cnt)

    def attend(self, q, pages=None, out=None, lse=None, stream=None, page_weight=None, weight_out=None, decay=1.0):
        """vsa_paged_attn (vsa_paged8_attn): q [B, Hq, D] over the whole cache, or
        over the pages = (page_idx, page_cnt) that select returned. Returns (out
        [B, Hq, D], lse fp32 [B, Hq]). With page_weight fp32 [B, Hkv, max_pages]
        (vsa_paged_attn_weigh) the attention weight that each page receives is
        added to it, in place or into weight_out, what it held multiplied by
        decay: what evict goes by."""
        if stream is not None:
            with self._on(stream):
                return self._calls.attend(q, pages, out, lse, page_weight, weight_out, decay)
        return self._calls.attend(q, pages, out, lse, page_weight, weight_out, decay)

    def read(self, tokens, cu_seqlens=None, k_out=None, v_out=None, stream=None):
        """vsa_paged_read: (k, v), each [tokens, Hkv, D] in dtype, of the newest
        tokens of each sequence: cu_seqlens [B+1] as in append, one each without
        it. A cache in 8 bits gives the values it stands for."""
        if stream is not None:
            with self._on(stream):
                return self._calls.read(tokens, cu_seqlens, k_out, v_out)
        return self._calls.read(tokens, cu_seqlens, k_out, v_out)

    def evict(self, page_weight, keep, keep_first=0, keep_last=1, freed=None, freed_cnt=None, out=None, stream=None):
        """vsa_page_evict: cuts sequences of more than keep pages to those with the
        largest page_weight fp32 [B, Hkv, max_pages] and the first keep_first and
        last keep_last. The table, the lengths and page_weight change in place, or
        are left and written to out = (page_table, seq_lens, page_weight).
        Returns (freed int32 [B, max(1, max_pages - keep)], freed_cnt int32 [B]):
        the pages that went. Layers that share a table evict once, by one
        page_weight that each layer's attend was given (decay in the first one's
        alone). Later appends give positions: lengths no longer are."""
        if stream is not None:
            with self._on(stream):
                return self._calls.evict(page_weight, keep, keep_first, keep_last, freed, freed_cnt, out)
        return self._calls.evict(page_weight, keep, keep_first, keep_last, freed, freed_cnt, out)
