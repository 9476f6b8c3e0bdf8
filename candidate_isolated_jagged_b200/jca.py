"""Thin ctypes binding over libjca.so (the C ABI declared in include/jca.h).

Argument marshalling only: tensors are passed as device pointers with their sizes, the stream is
torch's current CUDA stream, and every step of the computation runs in the library's kernels.
PyTorch allocates the outputs, the workspace and the status word. There is no CPU fallback: when
the library is missing, ``lib()`` raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libjca.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "jca.h")

_lib = None

c_i32, c_i64, c_f32, c_sz, c_vp = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t,
                                   ctypes.c_void_p)

_SIGNATURES = {
    "jca_status_string": (ctypes.c_char_p, [c_i32]),
    "jca_offsets_from_lengths": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "jca_build_segment_ids": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i64, c_i64, c_i32, c_vp, c_vp,
                                      c_vp]),
    "jca_bounds_from_segment_ids": (c_i32, [c_vp, c_vp, c_i64, c_i64, c_i32, c_vp, c_vp, c_vp,
                                            c_vp, c_vp, c_vp]),
    "jca_build_work_queue": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_i32,
                                     c_vp, c_i64, c_vp, c_vp, c_vp]),
    "jca_max_work_items": (c_i64, [c_i64, c_i64, c_i32]),
    "jca_workspace_bytes": (c_sz, [c_i64, c_i64, c_i32, c_i32]),
    "jagged_cand_attn_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_i64, c_i64,
                                     c_i32, c_i32, c_f32, c_i32, c_vp, c_sz, c_vp, c_vp]),
    "cand_only_attn_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32,
                                   c_i64, c_i64, c_i64, c_i32, c_i32, c_f32, c_i32, c_vp, c_sz,
                                   c_vp, c_vp]),
    "jagged_cand_attn_plan": (c_i32, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i32, c_i32, c_i32, c_vp,
                                      c_sz, c_vp, c_vp]),
    "jagged_cand_attn_run": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_i64, c_i64, c_i32,
                                     c_i32, c_f32, c_vp, c_sz, c_vp, c_vp]),
    "cand_only_attn_plan": (c_i32, [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_i32, c_i32,
                                    c_vp, c_sz, c_vp, c_vp]),
    "cand_only_attn_run": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i64, c_i64,
                                   c_i64, c_i32, c_i32, c_f32, c_vp, c_sz, c_vp, c_vp]),
    "jca_rope_positions": (c_i32, [c_vp, c_vp, c_i64, c_i64, c_i64, c_i32, c_vp, c_vp, c_vp]),
    "jca_apply_rope": (c_i32, [c_vp, c_vp, c_vp, c_i64, c_i32, c_i32, c_f32, c_vp]),
    "jagged_cand_attn_fwd_lse": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                         c_i64, c_i64, c_i32, c_i32, c_f32, c_i32, c_vp, c_sz,
                                         c_vp, c_vp]),
    "jca_bwd_workspace_bytes": (c_sz, [c_i64, c_i64, c_i32, c_i32]),
    "jagged_causal_attn_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_i64, c_i64, c_i32,
                                       c_i32, c_f32, c_i32, c_vp, c_sz, c_vp, c_vp]),
    "ug_masked_cross_attn_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i64, c_i32,
                                         c_i32, c_i32, c_i32, c_i32, c_i32, c_f32, c_vp, c_vp]),
    "jagged_cand_attn_bwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp,
                                     c_i32, c_vp, c_vp, c_vp, c_i64, c_i64, c_i32, c_i32, c_f32,
                                     c_i32, c_vp, c_sz, c_vp, c_vp]),
    "jca_rope_attn_workspace_bytes": (c_sz, [c_i64, c_i64, c_i32, c_i32]),
    "jagged_cand_attn_rope_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_i64,
                                          c_i64, c_i32, c_i32, c_f32, c_i64, c_f32, c_i32, c_vp,
                                          c_sz, c_vp, c_vp]),
    "jca_seqpack_workspace_bytes": (c_sz, [c_i64, c_i64, c_i64, c_i32, c_i32]),
    "jca_seqpack_bwd_workspace_bytes": (c_sz, [c_i64, c_i64, c_i64, c_i32, c_i32]),
    "jagged_cand_attn_seqpack_fwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                             c_i64, c_i64, c_i64, c_i32, c_i32, c_f32, c_i32, c_vp,
                                             c_sz, c_vp, c_vp]),
    "jagged_cand_attn_seqpack_bwd": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                             c_vp, c_i32, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64,
                                             c_i32, c_i32, c_f32, c_i32, c_vp, c_sz, c_vp, c_vp]),
    "jca_stack_workspace_bytes": (c_sz, [c_i64, c_i64, c_i64, c_i64, c_i32, c_i32]),
    "jca_stack_fwd": (c_i32, [c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64,
                              c_i64, c_i32, c_i32, c_f32, c_i64, c_f32, c_i32, c_vp, c_sz, c_vp,
                              c_vp]),
    "jca_rope_axes_fwd": (c_i32, [c_vp] * 6 + [c_i32, c_i32, c_i64, c_i32, c_i32, c_i32] +
                          [c_i64] * 4 + [c_f32, c_i32, c_i32, c_vp]),
    "jca_rope_axes_bwd": (c_i32, [c_vp] * 6 + [c_i32, c_i32, c_i64, c_i32, c_i32, c_i32] +
                          [c_i64] * 4 + [c_f32, c_i32, c_i32, c_vp]),
    "jca_window_workspace_bytes": (c_sz, [c_i64, c_i64, c_i32, c_i32, c_i32, c_i32]),
    "jca_window_bwd_workspace_bytes": (c_sz, [c_i64, c_i64, c_i32, c_i32, c_i32, c_i32]),
    "jca_window_bwd_workspace_bytes_for": (c_sz, [c_i64, c_i64, c_i32, c_i32, c_i32, c_i32, c_i64]),
    "jagged_window_attn_fwd": (c_i32, [c_vp] * 7 + [c_i64, c_i64, c_i32, c_i32, c_i32, c_i64, c_i32,
                                                    c_i64, c_i64, c_i64, c_f32, c_i32, c_vp, c_sz,
                                                    c_vp, c_vp]),
    "jagged_window_attn_bwd": (c_i32, [c_vp] * 11 + [c_i64, c_i64, c_i32, c_i32, c_i32, c_i64,
                                                     c_i32, c_i64, c_i64, c_i64, c_f32, c_i32,
                                                     c_vp, c_sz, c_vp, c_vp]),
    "jagged_window_decode_fwd": (c_i32, [c_vp] * 8 + [c_i64, c_i64, c_i32, c_i32, c_i32, c_i64,
                                                      c_i64, c_i64, c_i64, c_i64, c_f32, c_i32,
                                                      c_vp, c_vp]),
    "cand_tree_attn_fwd": (c_i32, [c_vp] * 10 + [c_i64, c_i64, c_i64, c_i32, c_i32, c_i32, c_i32,
                                                 c_i64, c_i64, c_i64, c_f32, c_i32, c_vp, c_vp]),
    "jca_noalloc_scratch_bytes": (c_sz, []),
    "jca_noalloc_prepare": (c_i32, []),
    "jca_user_tile_cost": (c_i64, [c_i64, c_i64]),
    "jca_selftest_wait_timeout": (c_i32, [c_vp, c_vp]),
    "jca_shard_users": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "jagged_cand_attn_fwd_noalloc": (c_i32, [c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp,
                                             c_i64, c_i64, c_i32, c_i32, c_f32, c_i32, c_vp,
                                             c_vp]),
}


class JcaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {status_string(code)} (code {code})")


def lib(path: Optional[str] = None):
    """Load libjca.so (once). Raises when it is missing: there is no fallback."""
    global _lib
    if path is not None:
        return _load(path)
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def _load(path: str):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           f"`python -m candidate_isolated_jagged_b200.build`")
    L = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def header_functions(path: str = HEADER_PATH):
    """Names of the functions declared in include/jca.h."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*([a-z_0-9]+)\s*\(", text,
                                 flags=re.M)))


def status_string(code: int) -> str:
    return lib().jca_status_string(int(code)).decode()


# ------------------------------------------------------------------------------------------------
# Marshalling helpers
# ------------------------------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _idx_bits(t: torch.Tensor) -> int:
    if t.dtype == torch.int32:
        return 32
    if t.dtype == torch.int64:
        return 64
    raise TypeError(f"index tensors must be int32 or int64, got {t.dtype}")


def _check(code: int, where: str) -> int:
    if code < 0:
        raise JcaError(code, where)
    return code


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_status(status: torch.Tensor, where: str = "device") -> None:
    """Read the device status word (synchronises) and raise on a recorded data error."""
    code = int(status.item())
    if code != 0:
        raise JcaError(code, where)


# ------------------------------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ------------------------------------------------------------------------------------------------

def jca_offsets_from_lengths(lengths: torch.Tensor, offsets: torch.Tensor, status: torch.Tensor,
                             stream=None) -> int:
    return _check(lib().jca_offsets_from_lengths(_ptr(lengths), _ptr(offsets), lengths.numel(),
                                                 _idx_bits(lengths), _ptr(status), _stream(stream)),
                  "jca_offsets_from_lengths")


def jca_build_segment_ids(offsets, candidate_start, valid_mask, attend_padded_history: bool,
                          seg: torch.Tensor, status: torch.Tensor, stream=None) -> int:
    B = offsets.numel() - 1
    return _check(lib().jca_build_segment_ids(
        _ptr(offsets), _ptr(candidate_start), _ptr(valid_mask), int(bool(attend_padded_history)),
        B, seg.numel(), _idx_bits(offsets), _ptr(seg), _ptr(status), _stream(stream)),
        "jca_build_segment_ids")


def jca_bounds_from_segment_ids(seg, offsets, hist_lo, hist_hi, cand_lo, cand_hi, status,
                                stream=None) -> int:
    B = offsets.numel() - 1
    return _check(lib().jca_bounds_from_segment_ids(
        _ptr(seg), _ptr(offsets), B, seg.numel(), _idx_bits(offsets), _ptr(hist_lo), _ptr(hist_hi),
        _ptr(cand_lo), _ptr(cand_hi), _ptr(status), _stream(stream)), "jca_bounds_from_segment_ids")


def jca_build_work_queue(q_offsets, kv_lo, kv_hi, kv_count, q_rows: int, kv_rows: int, H: int,
                         items: torch.Tensor, n_items: torch.Tensor, status, stream=None) -> int:
    B = q_offsets.numel() - 1
    return _check(lib().jca_build_work_queue(
        _ptr(q_offsets), _ptr(kv_lo), _ptr(kv_hi), _ptr(kv_count), B, int(q_rows), int(kv_rows),
        int(H), _idx_bits(q_offsets), _ptr(items), items.numel() // 4, _ptr(n_items), _ptr(status),
        _stream(stream)), "jca_build_work_queue")


def jca_max_work_items(B: int, rows: int, H: int) -> int:
    return int(lib().jca_max_work_items(int(B), int(rows), int(H)))


def jca_workspace_bytes(B: int, rows: int, H: int, d_head: int) -> int:
    return int(lib().jca_workspace_bytes(int(B), int(rows), int(H), int(d_head)))


def jagged_cand_attn_fwd(q, k, v, out, offsets, candidate_start=None, seg=None, scale: float = 0.0,
                         workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> int:
    T, H, d = q.shape
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_workspace_bytes(B, T, H, d), dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(offsets), _ptr(candidate_start),
        _ptr(seg), B, T, H, d, float(scale), _idx_bits(offsets), _ptr(workspace),
        workspace.numel(), _ptr(status), _stream(stream)), "jagged_cand_attn_fwd")


def cand_only_attn_fwd(cand_q, own_k, own_v, cand_offsets, hist_k, hist_v, hist_offsets, out,
                       hist_seg=None, scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> int:
    Nc, H, d = cand_q.shape
    Th = hist_k.shape[0]
    B = cand_offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_workspace_bytes(B, Nc, H, d), dtype=torch.uint8,
                                device=cand_q.device)
    if status is None:
        status = new_status(cand_q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().cand_only_attn_fwd(
        _ptr(cand_q), _ptr(own_k), _ptr(own_v), _ptr(cand_offsets), _ptr(hist_k), _ptr(hist_v),
        _ptr(hist_offsets), _ptr(hist_seg), _ptr(out), out_fp32, B, Nc, Th, H, d, float(scale),
        _idx_bits(cand_offsets), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)), "cand_only_attn_fwd")


def jagged_cand_attn_plan(offsets, candidate_start, seg, T: int, H: int, d_head: int,
                          workspace: torch.Tensor, status: torch.Tensor, stream=None) -> int:
    B = offsets.numel() - 1
    return _check(lib().jagged_cand_attn_plan(
        _ptr(offsets), _ptr(candidate_start), _ptr(seg), B, int(T), int(H), int(d_head),
        _idx_bits(offsets), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
        "jagged_cand_attn_plan")


def jagged_cand_attn_run(q, k, v, out, seg, B: int, workspace: torch.Tensor, status: torch.Tensor,
                         scale: float = 0.0, stream=None) -> int:
    T, H, d = q.shape
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_run(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(seg), int(B), T, H, d, float(scale),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)), "jagged_cand_attn_run")


def cand_only_attn_plan(cand_offsets, hist_offsets, hist_seg, Nc: int, Th: int, H: int, d_head: int,
                        workspace: torch.Tensor, status: torch.Tensor, stream=None) -> int:
    B = cand_offsets.numel() - 1
    return _check(lib().cand_only_attn_plan(
        _ptr(cand_offsets), _ptr(hist_offsets), _ptr(hist_seg), B, int(Nc), int(Th), int(H),
        int(d_head), _idx_bits(cand_offsets), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)), "cand_only_attn_plan")


def cand_only_attn_run(cand_q, own_k, own_v, hist_k, hist_v, hist_seg, out, B: int,
                       workspace: torch.Tensor, status: torch.Tensor, scale: float = 0.0,
                       stream=None) -> int:
    Nc, H, d = cand_q.shape
    Th = hist_k.shape[0]
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().cand_only_attn_run(
        _ptr(cand_q), _ptr(own_k), _ptr(own_v), _ptr(hist_k), _ptr(hist_v), _ptr(hist_seg),
        _ptr(out), out_fp32, int(B), Nc, Th, H, d, float(scale), _ptr(workspace),
        workspace.numel(), _ptr(status), _stream(stream)), "cand_only_attn_run")


def jca_noalloc_prepare() -> int:
    """Caches the static scratch array's device address for the current device (call it before
    capturing a stream that will hold jagged_cand_attn_fwd_noalloc)."""
    return _check(lib().jca_noalloc_prepare(), "jca_noalloc_prepare")


def jagged_cand_attn_fwd_noalloc(q, k, v, out, offsets, candidate_start=None, seg=None,
                                 scale: float = 0.0, status: Optional[torch.Tensor] = None,
                                 stream=None) -> int:
    """jagged_cand_attn_fwd for callers that cannot allocate device memory at call time: the
    library uses its own fixed 8 MiB static scratch array instead of a caller workspace (see
    include/jca.h for the size limit and the sharing rules). The caller passes the int32 status
    word too (device memory it owns), so that nothing here allocates either; only the C call is
    allocation-free when called some other way."""
    T, H, d = q.shape
    B = offsets.numel() - 1
    if status is None:
        raise ValueError("jagged_cand_attn_fwd_noalloc needs a caller-owned status tensor "
                         "(new_status() once, outside the allocation-free region)")
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(offsets), _ptr(candidate_start),
        _ptr(seg), B, T, H, d, float(scale), _idx_bits(offsets), _ptr(status), _stream(stream)),
        "jagged_cand_attn_fwd_noalloc")


def jca_selftest_wait_timeout(status, stream=None) -> int:
    """One block that runs the library's bounded pipeline wait on a barrier nothing completes:
    *status becomes JCA_STATUS_TIMEOUT (16) after about 2 s, and the context stays usable."""
    return _check(lib().jca_selftest_wait_timeout(_ptr(status), _stream(stream)),
                  "jca_selftest_wait_timeout")


def shard_users(row_lengths, n_keys, n_shards: int):
    """Host-side LPT split of a batch's users over n_shards GPUs (jca_shard_users).

    row_lengths, n_keys: per-user rows and segment-1 keys (array-likes of int). Returns
    (shard [B] int32, load [n_shards] int64) as numpy arrays."""
    import numpy as np
    rl = np.ascontiguousarray(np.asarray(row_lengths, dtype=np.int64))
    nk = np.ascontiguousarray(np.asarray(n_keys, dtype=np.int64))
    if rl.shape != nk.shape or rl.ndim != 1:
        raise ValueError("row_lengths and n_keys must be 1-D arrays of the same length")
    shard = np.empty(rl.shape[0], dtype=np.int32)
    load = np.empty(int(n_shards), dtype=np.int64)
    _check(lib().jca_shard_users(rl.ctypes.data if rl.size else None,
                                 nk.ctypes.data if nk.size else None, rl.shape[0], int(n_shards),
                                 shard.ctypes.data if shard.size else None, load.ctypes.data),
           "jca_shard_users")
    return shard, load


def user_tile_cost(row_length: int, n_keys: int) -> int:
    """Tile cost of one user (jca_user_tile_cost)."""
    return int(lib().jca_user_tile_cost(int(row_length), int(n_keys)))


def jca_rope_positions(seg, offsets, positions, history_end: int, status, stream=None) -> int:
    """Right-anchored positions (int32 [T]) of the tokens of a segment-ID array."""
    B = offsets.numel() - 1
    T = seg.numel()
    return _check(lib().jca_rope_positions(_ptr(seg), _ptr(offsets), B, T, int(history_end),
                                           _idx_bits(offsets), _ptr(positions), _ptr(status),
                                           _stream(stream)), "jca_rope_positions")


def jca_apply_rope(x, out, positions, base: float = 10000.0, stream=None) -> int:
    """Rotate the rows of a [T, H, d] bf16 tensor by their positions (out may be x)."""
    T, H, d = x.shape
    return _check(lib().jca_apply_rope(_ptr(x), _ptr(out), _ptr(positions), T, H, d, float(base),
                                       _stream(stream)), "jca_apply_rope")


def jagged_cand_attn_fwd_lse(q, k, v, out, lse, offsets, candidate_start=None, seg=None,
                             scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None) -> int:
    """jagged_cand_attn_fwd that also writes lse [T, H] fp32 (log of each row's softmax
    denominator; -inf for padding rows)."""
    T, H, d = q.shape
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_workspace_bytes(B, T, H, d), dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_fwd_lse(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(lse), _ptr(offsets),
        _ptr(candidate_start), _ptr(seg), B, T, H, d, float(scale), _idx_bits(offsets),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
        "jagged_cand_attn_fwd_lse")


def jagged_causal_attn_fwd(q, k, v, out, offsets, scale: float = 0.0,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Per-user causal attention over packed sequences (row i sees rows j <= i of its user)."""
    T, H, d = q.shape
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_workspace_bytes(B, T, H, d), dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_causal_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(offsets), B, T, H, d, float(scale),
        _idx_bits(offsets), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
        "jagged_causal_attn_fwd")


def ug_masked_cross_attn_fwd(q, k, v, out, c_u: int, n_u: int, residual=None,
                             scale: float = 0.0, status: Optional[torch.Tensor] = None,
                             stream=None) -> int:
    """UG-Sep's masked cross-attention: q [B, T_out, H, d], k and v [B, T_in, H, d] (bf16); the
    first c_u outputs read only the first n_u inputs. out [B, T_out, H, d] (bf16 or fp32) gets
    residual + R when a residual is given."""
    B, T_out, H, d = q.shape
    T_in = k.shape[1]
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().ug_masked_cross_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(residual), _ptr(out),
        out_fp32, B, T_out, T_in, int(c_u), int(n_u), H, d, float(scale), _ptr(status),
        _stream(stream)), "ug_masked_cross_attn_fwd")


def jca_bwd_workspace_bytes(B: int, T: int, H: int, d_head: int) -> int:
    return int(lib().jca_bwd_workspace_bytes(int(B), int(T), int(H), int(d_head)))


def jagged_cand_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, offsets, candidate_start=None,
                         seg=None, scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Gradients dq, dk, dv ([T, H, d], bf16 or fp32 as the tensors given) of the jagged
    candidate-isolated attention for the upstream gradient dout."""
    T, H, d = q.shape
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_bwd_workspace_bytes(B, T, H, d), dtype=torch.uint8,
                                device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    grad_fp32 = 1 if dq.dtype == torch.float32 else 0
    assert dk.dtype == dq.dtype and dv.dtype == dq.dtype
    return _check(lib().jagged_cand_attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
        _ptr(dv), grad_fp32, _ptr(offsets), _ptr(candidate_start), _ptr(seg), B, T, H, d,
        float(scale), _idx_bits(offsets), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)), "jagged_cand_attn_bwd")


def jca_rope_attn_workspace_bytes(B: int, T: int, H: int, d_head: int) -> int:
    return int(lib().jca_rope_attn_workspace_bytes(int(B), int(T), int(H), int(d_head)))


def jagged_cand_attn_rope_fwd(q, k, v, out, offsets, candidate_start=None, seg=None,
                              history_end: int = 0, rope_base: float = 10000.0, scale: float = 0.0,
                              workspace: Optional[torch.Tensor] = None,
                              status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Jagged candidate-isolated attention with right-anchored RoPE rotated inside the kernel
    (q and k unrotated, left unchanged)."""
    T, H, d = q.shape
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(max(1, jca_rope_attn_workspace_bytes(B, T, H, d)),
                                dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_rope_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(offsets), _ptr(candidate_start),
        _ptr(seg), B, T, H, d, float(scale), int(history_end), float(rope_base),
        _idx_bits(offsets), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
        "jagged_cand_attn_rope_fwd")


def jca_seqpack_workspace_bytes(B: int, Th: int, Nc: int, H: int, d_head: int) -> int:
    return int(lib().jca_seqpack_workspace_bytes(int(B), int(Th), int(Nc), int(H), int(d_head)))


def jca_seqpack_bwd_workspace_bytes(B: int, Th: int, Nc: int, H: int, d_head: int) -> int:
    return int(lib().jca_seqpack_bwd_workspace_bytes(int(B), int(Th), int(Nc), int(H),
                                                     int(d_head)))


def jagged_cand_attn_seqpack_fwd(q, k, v, out, hist_offsets, cand_offsets, seg=None, lse=None,
                                 scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                                 status: Optional[torch.Tensor] = None, stream=None,
                                 Th: Optional[int] = None) -> int:
    """Forward over the candidate-packed matrix [history runs | candidate runs] (rows [0, Th)
    split at hist_offsets, rows [Th, T) split at cand_offsets); lse [T, H] fp32 optional.
    Th (history rows) is read back from hist_offsets when not given."""
    T, H, d = q.shape
    B = hist_offsets.numel() - 1
    Th = _seqpack_th(hist_offsets) if Th is None else int(Th)
    Nc = T - Th
    if workspace is None:
        workspace = torch.empty(max(1, jca_seqpack_workspace_bytes(B, Th, Nc, H, d)),
                                dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    return _check(lib().jagged_cand_attn_seqpack_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(lse), _ptr(hist_offsets),
        _ptr(cand_offsets), _ptr(seg), B, Th, Nc, H, d, float(scale), _idx_bits(hist_offsets),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)),
        "jagged_cand_attn_seqpack_fwd")


def jagged_cand_attn_seqpack_bwd(q, k, v, out, dout, lse, dq, dk, dv, hist_offsets, cand_offsets,
                                 seg=None, scale: float = 0.0,
                                 workspace: Optional[torch.Tensor] = None,
                                 status: Optional[torch.Tensor] = None, stream=None,
                                 Th: Optional[int] = None) -> int:
    """Gradients dq, dk, dv over the candidate-packed matrix (see jagged_cand_attn_seqpack_fwd)."""
    T, H, d = q.shape
    B = hist_offsets.numel() - 1
    Th = _seqpack_th(hist_offsets) if Th is None else int(Th)
    Nc = T - Th
    if workspace is None:
        workspace = torch.empty(max(1, jca_seqpack_bwd_workspace_bytes(B, Th, Nc, H, d)),
                                dtype=torch.uint8, device=q.device)
    if status is None:
        status = new_status(q.device)
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    grad_fp32 = 1 if dq.dtype == torch.float32 else 0
    assert dk.dtype == dq.dtype and dv.dtype == dq.dtype
    return _check(lib().jagged_cand_attn_seqpack_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), out_fp32, _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
        _ptr(dv), grad_fp32, _ptr(hist_offsets), _ptr(cand_offsets), _ptr(seg), B, Th, Nc, H, d,
        float(scale), _idx_bits(hist_offsets), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)), "jagged_cand_attn_seqpack_bwd")


def _seqpack_th(hist_offsets) -> int:
    """Th = hist_offsets[B], read back to the host (the caller's layout; a device read)."""
    return int(hist_offsets[-1].item())


def jca_stack_workspace_bytes(B: int, T: int, Nc: int, Th: int, H: int, d_head: int) -> int:
    return int(lib().jca_stack_workspace_bytes(int(B), int(T), int(Nc), int(Th), int(H),
                                               int(d_head)))


def jca_stack_fwd(x, x_out, weights, n_cand_only: int, offsets, candidate_start=None, seg=None,
                  Nc: int = 0, Th: int = 0, H: int = 1, scale: float = 0.0,
                  history_end: Optional[int] = None, rope_base: float = 10000.0,
                  workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None) -> int:
    """Layer stack with candidate-only tail layers: x [T, D] bf16 -> x_out [T, D] bf16 through
    weights [n_layers, 4, D, D] bf16 (Wq, Wk, Wv, Wo per layer, x @ W). Nc / Th: total candidate and
    history tokens. history_end None turns RoPE off."""
    T, D = x.shape
    n_layers = weights.shape[0] if weights.dim() == 4 else 0
    d = D // int(H)
    B = offsets.numel() - 1
    if workspace is None:
        workspace = torch.empty(jca_stack_workspace_bytes(B, T, Nc, Th, H, d), dtype=torch.uint8,
                                device=x.device)
    if status is None:
        status = new_status(x.device)
    return _check(lib().jca_stack_fwd(
        _ptr(x), _ptr(x_out), _ptr(weights), int(n_layers), int(n_cand_only), _ptr(offsets),
        _ptr(candidate_start), _ptr(seg), B, T, int(Nc), int(Th), int(H), d, float(scale),
        -1 if history_end is None else int(history_end), float(rope_base), _idx_bits(offsets),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)), "jca_stack_fwd")


# Rotary positions with several axes, windowed attention, and attention over a cache. These check
# shapes, types, devices and strides here, run on the tensors' own device (its current stream,
# unless a stream is given) and accept rows that are apart (slices of a fused projection).

_ROPE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _bad_rows(name: str, t: torch.Tensor, shape, dtype, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _rows(name: str, t: torch.Tensor, rows: int, heads: int, d: int, dtype, device) -> int:
    """Checks a [rows, heads, d] tensor with packed heads; returns its row stride in elements."""
    if t.dtype != dtype or t.shape != (rows, heads, d) or t.device != device:
        _bad_rows(name, t, (rows, heads, d), dtype, device)
    if rows == 0:
        return heads * d
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a row must be packed")
    return s0 if rows > 1 else heads * d


def _packed(name: str, t: torch.Tensor, rows: int, heads: int, d: int, dtype, device) -> None:
    if t.dtype != dtype or t.shape != (rows, heads, d) or t.device != device:
        _bad_rows(name, t, (rows, heads, d), dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _vector(name: str, t: Optional[torch.Tensor], n: int, dtype, device) -> None:
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements, got {list(t.shape)}")


def _heads(name: str, t: torch.Tensor):
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions, got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.shape


def _on(stream, device):
    """Context in which a call's own scratch is made: on the call's stream, so that its first fill
    comes before the kernels and its memory is not handed out again before they are done."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _status_on(status: Optional[torch.Tensor], device, stream) -> torch.Tensor:
    if status is None:
        with _on(stream, device):
            return new_status(device)
    _vector("status", status, 1, torch.int32, device)
    return status


# The current stream's handle of a device; torch.cuda.current_stream(i).cuda_stream builds two Python
# objects for the same number, 6 us where the small calls here take 4 us on the GPU.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn: str, device, stream, *args) -> int:
    """The C entry point `fn` with `device` current, on its current stream unless one is given."""
    f = getattr(_lib or lib(), fn)
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    if stream is None:
        handle = _raw_stream(device.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    code = f(*args, handle)
    return code if code >= 0 else _check(code, fn)


def _clip(x: int, bits: int) -> int:
    """x, or the nearest integer of that many bits: ctypes would drop the upper ones."""
    top = 2 ** (bits - 1)
    return max(-top, min(int(x), top - 1))


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=64, typed=True)   # typed: 8.0 is not taken for an 8 seen before
def _section_array(*sections):
    # ctypes refuses what is no integer.
    return (c_i32 * len(sections))(*(_clip(x, 32) if isinstance(x, int) else x for x in sections))


def _sections(sections):
    return _section_array(*sections)


def _rope_axes(fn, q, k, q_out, k_out, positions, sections, base, per_axis, stream) -> int:
    T, H, d = _heads("q", q)
    dev, dtype = q.device, q.dtype
    if dtype not in _ROPE_TYPES:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dtype}")
    qs, qo = _rows("q", q, T, H, d, dtype, dev), _rows("q_out", q_out, T, H, d, dtype, dev)
    Hkv, ks, ko = 0, 0, 0
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is not None:
        Hkv = _heads("k", k)[1]
        ks, ko = _rows("k", k, T, Hkv, d, dtype, dev), _rows("k_out", k_out, T, Hkv, d, dtype, dev)
    n_axes = len(sections)
    if positions.dim() == 1:
        positions = positions[:, None]
    if positions.shape != (T, n_axes) or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous [{T}, {n_axes}], got "
                         f"{list(positions.shape)}")
    if positions.device != dev:
        raise ValueError(f"positions is on {positions.device}, not on {dev}")
    sec = _sections(sections)
    return _call(fn, dev, stream, _at(q), _at(k), _at(q_out), _at(k_out), _at(positions), sec,
                 n_axes, int(bool(per_axis)), T, H, Hkv, d, qs, ks, qo, ko, float(base),
                 _ROPE_TYPES[dtype], _idx_bits(positions))


def jca_rope_axes_fwd(q, k, q_out, k_out, positions, sections, base: float = 10000.0,
                      per_axis: bool = False, stream=None) -> int:
    """Rotates q [T, H, d] and k [T, Hkv, d] (k may be None) by several axes of positions
    [T, n_axes] (int32 or int64): the first sections[0] pairs (j, j + d/2) of every head by axis 0,
    the next sections[1] by axis 1, ...; the rest stays. Frequencies run over the head, or over
    each axis' own pairs with per_axis. bf16, fp16 or fp32; outputs may be the inputs."""
    return _rope_axes("jca_rope_axes_fwd", q, k, q_out, k_out, positions, sections, base, per_axis,
                      stream)


def jca_rope_axes_bwd(dq_out, dk_out, dq, dk, positions, sections, base: float = 10000.0,
                      per_axis: bool = False, stream=None) -> int:
    """Gradient of jca_rope_axes_fwd: dq, dk from the gradients of its outputs."""
    return _rope_axes("jca_rope_axes_bwd", dq_out, dk_out, dq, dk, positions, sections, base,
                      per_axis, stream)


def _window_sizes(B, T, H, Hkv, d_head, n_sinks):
    return (_clip(B, 64), _clip(T, 64), *(_clip(x, 32) for x in (H, Hkv, d_head, n_sinks)))


def jca_window_workspace_bytes(B: int, T: int, H: int, Hkv: int, d_head: int, n_sinks: int) -> int:
    return int(lib().jca_window_workspace_bytes(*_window_sizes(B, T, H, Hkv, d_head, n_sinks)))


def jca_window_bwd_workspace_bytes(B: int, T: int, H: int, Hkv: int, d_head: int, n_sinks: int,
                                   window: int = 1) -> int:
    """Enough for `window` and every longer one; without it for all of them. Many users with many
    first tokens need far less under a window that few of them exceed."""
    return int(lib().jca_window_bwd_workspace_bytes_for(
        *_window_sizes(B, T, H, Hkv, d_head, n_sinks), _clip(window, 64)))


def _window_scratch(workspace, status, nbytes, dev, stream):
    if workspace is None:
        with _on(stream, dev):
            workspace = torch.empty(nbytes(), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    return workspace, _status_on(status, dev, stream)


def jagged_window_attn_fwd(q, k, v, out, offsets, window: int, n_sinks: int = 0, valid=None,
                           lse=None, scale: float = 0.0,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Per-user causal attention with a sliding window and the first n_sinks tokens of every row
    visible: q [T, H, d], k and v [T, Hkv, d] bf16, out [T, H, d] bf16; valid [T] uint8 (1 = real
    token) and lse [T, H] fp32 are optional."""
    T, H, d = _heads("q", q)
    Hkv, dev, t16 = _heads("k", k)[1], q.device, torch.bfloat16
    B = offsets.numel() - 1
    qs, ks = _rows("q", q, T, H, d, t16, dev), _rows("k", k, T, Hkv, d, t16, dev)
    vs = _rows("v", v, T, Hkv, d, t16, dev)
    _packed("out", out, T, H, d, t16, dev)
    _vector("offsets", offsets, B + 1, offsets.dtype, dev)
    _vector("valid", valid, T, torch.uint8, dev)
    _vector("lse", lse, T * H, torch.float32, dev)
    workspace, status = _window_scratch(
        workspace, status, lambda: jca_window_workspace_bytes(
            B, T, H, Hkv, d, n_sinks), dev, stream)
    return _call("jagged_window_attn_fwd", dev, stream, _at(q), _at(k), _at(v), _at(out), _at(lse),
                 _at(offsets), _at(valid), B, T, H, Hkv, d, _clip(window, 64), _clip(n_sinks, 32), qs,
                 ks, vs, float(scale), _idx_bits(offsets), _at(workspace),
                 workspace.numel() * workspace.element_size(), _at(status))


def jagged_window_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, offsets, window: int,
                           n_sinks: int = 0, valid=None, scale: float = 0.0,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Gradients dq [T, H, d], dk and dv [T, Hkv, d] (bf16) of jagged_window_attn_fwd for the
    upstream gradient dout; out and lse are the forward's."""
    T, H, d = _heads("q", q)
    Hkv, dev, t16 = _heads("k", k)[1], q.device, torch.bfloat16
    B = offsets.numel() - 1
    qs, ks = _rows("q", q, T, H, d, t16, dev), _rows("k", k, T, Hkv, d, t16, dev)
    vs = _rows("v", v, T, Hkv, d, t16, dev)
    for name, x, n in (("out", out, H), ("dout", dout, H), ("dq", dq, H), ("dk", dk, Hkv),
                       ("dv", dv, Hkv)):
        _packed(name, x, T, n, d, t16, dev)
    _vector("offsets", offsets, B + 1, offsets.dtype, dev)
    _vector("valid", valid, T, torch.uint8, dev)
    _vector("lse", lse, T * H, torch.float32, dev)
    workspace, status = _window_scratch(
        workspace, status, lambda: jca_window_bwd_workspace_bytes(
            B, T, H, Hkv, d, n_sinks, window), dev, stream)
    return _call("jagged_window_attn_bwd", dev, stream, _at(q), _at(k), _at(v), _at(out), _at(dout),
                 _at(lse), _at(dq), _at(dk), _at(dv), _at(offsets), _at(valid), B, T, H, Hkv, d,
                 _clip(window, 64), _clip(n_sinks, 32), qs, ks, vs, float(scale), _idx_bits(offsets),
                 _at(workspace), workspace.numel() * workspace.element_size(), _at(status))


def jagged_window_decode_fwd(q, k_new, v_new, k_cache, v_cache, out, cache_offsets, cache_len,
                             window: int, n_sinks: int = 0, scale: float = 0.0,
                             status: Optional[torch.Tensor] = None, stream=None) -> int:
    """One new token per user over a cache: q [B, H, d], k_new and v_new [B, Hkv, d] are written
    behind the cache_len[b] tokens of user b's region [cache_offsets[b], cache_offsets[b+1]) of
    k_cache, v_cache [R, Hkv, d], and attended with them under jagged_window_attn_fwd's mask.
    cache_len[b] = -1 marks an empty slot."""
    B, H, d = _heads("q", q)
    Hkv, dev, t16 = _heads("k_new", k_new)[1], q.device, torch.bfloat16
    R = _heads("k_cache", k_cache)[0]
    qs, ks = _rows("q", q, B, H, d, t16, dev), _rows("k_new", k_new, B, Hkv, d, t16, dev)
    vs = _rows("v_new", v_new, B, Hkv, d, t16, dev)
    _packed("k_cache", k_cache, R, Hkv, d, t16, dev)
    _packed("v_cache", v_cache, R, Hkv, d, t16, dev)
    _packed("out", out, B, H, d, t16, dev)
    _vector("cache_offsets", cache_offsets, B + 1, cache_offsets.dtype, dev)
    _vector("cache_len", cache_len, B, cache_offsets.dtype, dev)
    status = _status_on(status, dev, stream)
    return _call("jagged_window_decode_fwd", dev, stream, _at(q), _at(k_new), _at(v_new),
                 _at(k_cache), _at(v_cache), _at(out), _at(cache_offsets), _at(cache_len), B, R, H,
                 Hkv, d, _clip(window, 64), _clip(n_sinks, 64), qs, ks, vs, float(scale),
                 _idx_bits(cache_offsets), _at(status))


def cand_tree_attn_fwd(cand_q, own_k, own_v, cand_offsets, parent, hist_k, hist_v, hist_offsets,
                       out, max_cand: int, hist_len=None, scale: float = 0.0,
                       status: Optional[torch.Tensor] = None, stream=None) -> int:
    """Trees of drafted candidate tokens over cached histories: cand_q [Nc, H, d], own_k and own_v
    [Nc, Hkv, d]; parent [Nc] int32 is the parent's index in the user's run or -1. Each token sees
    its user's history (the first hist_len[b] rows of region [hist_offsets[b], hist_offsets[b+1])
    of hist_k, hist_v [R, Hkv, d]), its ancestors and itself. No run is longer than max_cand."""
    N, H, d = _heads("cand_q", cand_q)
    Hkv, dev, t16 = _heads("own_k", own_k)[1], cand_q.device, torch.bfloat16
    R = _heads("hist_k", hist_k)[0]
    B = cand_offsets.numel() - 1
    qs, ks = _rows("cand_q", cand_q, N, H, d, t16, dev), _rows("own_k", own_k, N, Hkv, d, t16, dev)
    vs = _rows("own_v", own_v, N, Hkv, d, t16, dev)
    _packed("hist_k", hist_k, R, Hkv, d, t16, dev)
    _packed("hist_v", hist_v, R, Hkv, d, t16, dev)
    _packed("out", out, N, H, d, t16, dev)
    _vector("cand_offsets", cand_offsets, B + 1, cand_offsets.dtype, dev)
    _vector("hist_offsets", hist_offsets, B + 1, cand_offsets.dtype, dev)
    _vector("hist_len", hist_len, B, cand_offsets.dtype, dev)
    _vector("parent", parent, N, torch.int32, dev)
    status = _status_on(status, dev, stream)
    return _call("cand_tree_attn_fwd", dev, stream, _at(cand_q), _at(own_k), _at(own_v),
                 _at(cand_offsets), _at(parent), _at(hist_k), _at(hist_v), _at(hist_offsets),
                 _at(hist_len), _at(out), B, N, R, H, Hkv, d, _clip(max_cand, 32), qs, ks, vs,
                 float(scale), _idx_bits(cand_offsets), _at(status))


def jca_noalloc_scratch_bytes() -> int:
    return int(lib().jca_noalloc_scratch_bytes())


def jca_status_string(code: int) -> str:
    return status_string(code)


# ------------------------------------------------------------------------------------------------
# Convenience: allocate outputs with torch, call, check the status word
# ------------------------------------------------------------------------------------------------

def attention(q, k, v, offsets, candidate_start=None, seg=None, out_fp32: bool = False,
              scale: float = 0.0, check: bool = True) -> torch.Tensor:
    out = torch.empty(q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
    status = new_status(q.device)
    jagged_cand_attn_fwd(q, k, v, out, offsets, candidate_start, seg, scale, status=status)
    if check:
        check_status(status, "jagged_cand_attn_fwd")
    return out


def cand_only(cand_q, own_k, own_v, cand_offsets, hist_k, hist_v, hist_offsets, hist_seg=None,
              out_fp32: bool = False, scale: float = 0.0, check: bool = True) -> torch.Tensor:
    out = torch.empty(cand_q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                      device=cand_q.device)
    status = new_status(cand_q.device)
    cand_only_attn_fwd(cand_q, own_k, own_v, cand_offsets, hist_k, hist_v, hist_offsets, out,
                       hist_seg, scale, status=status)
    if check:
        check_status(status, "cand_only_attn_fwd")
    return out
