"""GB300 (sm_103a) DSA candidate-block selection.

A thin binding over ``libdsa_cb.so`` (C ABI declared in ``include/dsa_cb.h``,
``include/dsa_dcp_attn.h``, ``include/dsa_attention.h`` and
``include/dsa_cache.h``):
argument marshalling only. Every step of the computation runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback, and every call
raises if the library is missing or a call fails.

Functions carry the C ABI's names:

* ``dsa_block_scores`` -- per-block windowed maxima (candidate_blocks.py diff,
  ``_block_scores``).
* ``dsa_select_candidate_blocks`` -- ranked top-k block ids, -1 padded
  (``select_candidate_blocks`` without a DCP group).
* ``dsa_select_candidate_blocks_sharded`` -- the DCP form with the ranks'
  local logits held as a leading ``[D, rows, local_width]`` axis.
* ``dsa_mask_candidate_logits[_sharded]`` -- the masking pass after
  selection: -inf outside each row's window and candidate blocks.
* ``dsa_correct_attn_out`` / ``dsa_merge_attn_out`` -- the DCP partial-
  attention LSE correction (sglang ``dcp/kernels.py``, ``correct_attn_out``;
  C ABI in ``include/dsa_dcp_attn.h``) and the sum over shards after it.
* ``dsa_prompt_attention`` / ``dsa_shared_prefix_attention`` -- attention over
  packed prompts, and of single tokens on a paged cache whose first pages a
  batch shares; both give the base-2 LSE that the merge takes, with bf16
  outputs as they are and fp16 ones widened to fp32
  (``include/dsa_attention.h``).
* ``dsa_cache_fork`` / ``dsa_cache_free`` / ``dsa_cache_compact`` -- the pages
  of such a cache (``include/dsa_cache.h``).

Tensors are PyTorch CUDA tensors (PyTorch supplies device memory and the
current stream) or pinned host tensors, which the kernels read and write in
place through ``dsa_mapped_host_pointer`` (across NVLink-C2C on Grace
systems). Logits may be float32 or bfloat16 (the ``*_bf16`` C entry points);
scores follow the logits' dtype. The attention and cache operators take CUDA
tensors only. ``select_candidate_blocks[_sharded]_host``
take host tensors and wait for the ids: pinned inputs are read in place
(only the in-window logits cross the link), other host tensors are copied to
the device first.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

__all__ = [
    "DsaError",
    "library",
    "library_path",
    "dsa_block_scores",
    "dsa_select_candidate_blocks",
    "dsa_select_candidate_blocks_sharded",
    "dsa_mask_candidate_logits",
    "dsa_mask_candidate_logits_sharded",
    "dsa_correct_attn_out",
    "dsa_merge_attn_out",
    "dsa_prompt_attention",
    "dsa_shared_prefix_attention",
    "dsa_cache_fork",
    "dsa_cache_free",
    "dsa_cache_compact",
    "FORK_OK",
    "FORK_NO_PAGE",
    "FORK_REFUSED",
    "select_candidate_blocks_host",
    "select_candidate_blocks_sharded_host",
    "prompt_workspace_bytes",
    "shared_prefix_workspace_bytes",
    "cache_workspace_bytes",
    "release_workspaces",
    "max_select_blocks",
    "mapped_host_pointer",
    "set_launch_override",
    "pipeline_error",
    "attention_error",
    "EXPORTED_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "_build", "libdsa_cb.so")

EXPORTED_SYMBOLS = (
    "dsa_status_string",
    "dsa_select_max_blocks",
    "dsa_select_max_shards",
    "dsa_select_workspace_bytes",
    "dsa_block_scores",
    "dsa_select_candidate_blocks",
    "dsa_select_candidate_blocks_sharded",
    "dsa_mask_candidate_logits",
    "dsa_mask_candidate_logits_sharded",
    "dsa_select_candidate_blocks_sharded_static",
    "dsa_mapped_host_pointer",
    "dsa_stream_id",
    "dsa_attn_max_shards",
    "dsa_correct_attn_out",
    "dsa_merge_attn_out",
    "dsa_block_scores_bf16",
    "dsa_select_candidate_blocks_bf16",
    "dsa_select_candidate_blocks_sharded_bf16",
    "dsa_mask_candidate_logits_bf16",
    "dsa_mask_candidate_logits_sharded_bf16",
    "dsa_select_candidate_blocks_sharded_starts",
    "dsa_select_candidate_blocks_sharded_starts_bf16",
    "dsa_mask_candidate_logits_sharded_starts",
    "dsa_mask_candidate_logits_sharded_starts_bf16",
    "dsa_select_set_launch_override",
    "dsa_pipeline_error",
    "dsa_prompt_workspace_bytes",
    "dsa_prompt_attention",
    "dsa_shared_prefix_workspace_bytes",
    "dsa_shared_prefix_attention",
    "dsa_attention_error",
    "dsa_cache_workspace_bytes",
    "dsa_cache_fork",
    "dsa_cache_free",
    "dsa_cache_compact",
)

# Knobs of dsa_select_set_launch_override (include/dsa_cb.h).
LAUNCH_KNOBS = {"split": 1, "threads": 2, "warp_rows": 3, "warp_order": 4, "pipeline": 5,
                "pipe_split": 6, "pipe_stages": 7, "pipe_stage_kb": 8, "pipe_sched": 9,
                "pipe_warps": 10, "pipe_ctas": 11, "pipe_stage_owner": 12, "pipe_order": 13,
                "rank_cta": 14}

_lib = None


class DsaError(RuntimeError):
    """A library call returned a status other than DSA_OK."""

    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {text} (status {status})")
        self.status = status


def library():
    """Load libdsa_cb.so (build it with ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"libdsa_cb.so is not built ({library_path}); "
                           "run __graft_entry__.build() first")
    lib = ctypes.CDLL(library_path)
    i64, i32, p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    lib.dsa_status_string.argtypes = [ctypes.c_int]
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_select_max_blocks.argtypes = []
    lib.dsa_select_max_blocks.restype = i32
    lib.dsa_select_max_shards.argtypes = []
    lib.dsa_select_max_shards.restype = i32
    lib.dsa_select_workspace_bytes.argtypes = [i64, i64]
    lib.dsa_select_workspace_bytes.restype = ctypes.c_size_t
    lib.dsa_pipeline_error.argtypes = [ctypes.c_int]
    lib.dsa_pipeline_error.restype = ctypes.c_int
    lib.dsa_select_set_launch_override.argtypes = [i32, i32]
    lib.dsa_select_set_launch_override.restype = ctypes.c_int
    lib.dsa_block_scores.argtypes = [p, i64, i64, i64, p, p, i32, i32, i32, p, i64, p]
    sz = ctypes.c_size_t
    lib.dsa_select_candidate_blocks.argtypes = [p, i64, i64, i64, p, p, i32, i32, i32, i32,
                                                p, i64, p, i64, p, sz, p]
    lib.dsa_select_candidate_blocks_sharded.argtypes = [p, i32, i64, i64, i64, i64, p, i32, i32,
                                                        i32, i32, p, i64, p, i64, p, sz, p]
    lib.dsa_mask_candidate_logits.argtypes = [p, i64, i64, i64, p, p, p, i32, i64, i32, i32, p]
    lib.dsa_mask_candidate_logits_sharded.argtypes = [p, i32, i64, i64, i64, i64, p, i32, i32, p,
                                                      i32, i64, p]
    lib.dsa_mapped_host_pointer.argtypes = [p, ctypes.POINTER(ctypes.c_void_p)]
    lib.dsa_mapped_host_pointer.restype = ctypes.c_int
    lib.dsa_stream_id.argtypes = [p]
    lib.dsa_stream_id.restype = ctypes.c_uint64
    lib.dsa_attn_max_shards.argtypes = []
    lib.dsa_attn_max_shards.restype = i32
    lib.dsa_correct_attn_out.argtypes = [p, i32, i64, i64, i64, i64, i64, i64, p, i32, i64, i64,
                                         i64, i32, p, i64, i64, i64, p, i64, i64, p]
    lib.dsa_merge_attn_out.argtypes = [p, i32, i32, i64, i64, i64, i64, i64, i64, i64, p, i64,
                                       i64, i64, p, i64, i64, i64, p, i64, i64, p]
    lib.dsa_select_candidate_blocks_sharded_starts.argtypes = [
        p, i32, i64, i64, i64, i64, p, p, i32, i32, i32, i32, p, i64, p, i64, p, sz, p]
    lib.dsa_mask_candidate_logits_sharded_starts.argtypes = [p, i32, i64, i64, i64, i64, p, p,
                                                             i32, i32, p, i32, i64, p]
    f32 = ctypes.c_float
    lib.dsa_prompt_attention.argtypes = [p, p, p, i32, i64, i64, i32, i32, i32, i64, i64, i64,
                                         i64, i64, i64, p, p, i32, i32, f32, p, i64, i64, p, i64,
                                         i64, p, sz, p]
    lib.dsa_prompt_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i32]
    lib.dsa_prompt_workspace_bytes.restype = sz
    lib.dsa_shared_prefix_workspace_bytes.argtypes = [i64, i32, i32, i32, i64, i64, i32]
    lib.dsa_shared_prefix_workspace_bytes.restype = sz
    lib.dsa_shared_prefix_attention.argtypes = [p, p, p, i32, i64, i32, i32, i32, i64, i32, i64,
                                                i64, i64, i64, i64, i64, i64, i64, p, i64, p, i64,
                                                i64, p, f32, p, i64, i64, p, i64, i64, p, sz, p]
    lib.dsa_attention_error.argtypes = [ctypes.c_int]
    lib.dsa_attention_error.restype = ctypes.c_int
    lib.dsa_cache_workspace_bytes.argtypes = [i64, i64]
    lib.dsa_cache_workspace_bytes.restype = sz
    lib.dsa_cache_fork.argtypes = [p, i64, i64, i64, i64, i32, i64, p, p, i64, i64, i64, p, p, p,
                                   i64, p, p, sz, p]
    lib.dsa_cache_free.argtypes = [p, i64, p, i64, i64, i64, p, p, i64, p]
    lib.dsa_cache_compact.argtypes = [p, i64, i64, i64, i64, i32, i64, p, p, i64, i64, i64, p, p,
                                      p, sz, p]
    for f in (lib.dsa_prompt_attention, lib.dsa_shared_prefix_attention, lib.dsa_cache_fork,
              lib.dsa_cache_free, lib.dsa_cache_compact):
        f.restype = ctypes.c_int
    for name in ("dsa_block_scores", "dsa_select_candidate_blocks",
                 "dsa_select_candidate_blocks_sharded", "dsa_mask_candidate_logits",
                 "dsa_mask_candidate_logits_sharded", "dsa_select_candidate_blocks_sharded_starts",
                 "dsa_mask_candidate_logits_sharded_starts"):
        getattr(lib, name + "_bf16").argtypes = getattr(lib, name).argtypes
    for f in (lib.dsa_block_scores, lib.dsa_select_candidate_blocks,
              lib.dsa_select_candidate_blocks_sharded, lib.dsa_mask_candidate_logits,
              lib.dsa_mask_candidate_logits_sharded, lib.dsa_correct_attn_out,
              lib.dsa_merge_attn_out, lib.dsa_block_scores_bf16,
              lib.dsa_select_candidate_blocks_bf16, lib.dsa_select_candidate_blocks_sharded_bf16,
              lib.dsa_mask_candidate_logits_bf16, lib.dsa_mask_candidate_logits_sharded_bf16,
              lib.dsa_select_candidate_blocks_sharded_starts,
              lib.dsa_select_candidate_blocks_sharded_starts_bf16,
              lib.dsa_mask_candidate_logits_sharded_starts,
              lib.dsa_mask_candidate_logits_sharded_starts_bf16):
        f.restype = ctypes.c_int
    _lib = lib
    return lib


def set_launch_override(knob: str, value: int) -> None:
    """Pin one launch-shape choice of the selecting calls for this process
    (value 0 hands it back to the launcher); for tests and tuning sweeps."""
    _check("dsa_select_set_launch_override",
           library().dsa_select_set_launch_override(LAUNCH_KNOBS[knob], int(value)))


def pipeline_error(clear: bool = False) -> int:
    """The pipelined kernels' give-up flag (0: none of their waits ever gave
    up); see dsa_pipeline_error."""
    return int(library().dsa_pipeline_error(1 if clear else 0))


def attention_error(clear: bool = False) -> int:
    """The attention kernels' give-up flag (0: none of their waits ever gave
    up), read behind all work of the current device; see dsa_attention_error."""
    return int(library().dsa_attention_error(1 if clear else 0))


def _check(fn: str, status: int):
    if status != 0:
        raise DsaError(fn, status, library().dsa_status_string(status).decode())


def max_select_blocks() -> int:
    return int(library().dsa_select_max_blocks())


def _torch():
    import torch
    return torch


def workspace_bytes(rows: int, nblocks: int) -> int:
    """Bytes of workspace that let a selecting call split rows over CTAs."""
    return int(library().dsa_select_workspace_bytes(rows, nblocks))


_ws_cache = {}


def _workspace(workspace, rows: int, nblocks: int, device, stream_handle):
    """(pointer, bytes) of the workspace for one call.

    ``workspace`` may be a CUDA tensor (zero-filled before its first use,
    written by nothing but these calls, and not shared by calls that can
    overlap), ``False`` (no workspace: one CTA per row) or ``None``: a
    zero-filled workspace cached per (device, stream) and grown when a call
    needs more."""
    torch = _torch()
    if workspace is False:
        return None, 0
    if workspace is not None:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a CUDA tensor")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    need = workspace_bytes(rows, nblocks)
    key = (device.index if device.index is not None else torch.cuda.current_device(),
           stream_handle)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.zeros(need, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf.data_ptr(), buf.numel()


def _stream_handle(stream) -> Optional[int]:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream or None


def mapped_host_pointer(t) -> int:
    """Device address of a pinned (page-locked) host tensor's data, under
    which kernels read and write it in place (``dsa_mapped_host_pointer``)."""
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a pinned host tensor")
    dev = ctypes.c_void_p()
    _check("dsa_mapped_host_pointer", library().dsa_mapped_host_pointer(t.data_ptr(),
                                                                         ctypes.byref(dev)))
    return dev.value


def _dev_ptr(t, dtype, name, *, allow_none=False):
    """Device address of a CUDA tensor, or of a pinned host tensor (read and
    written in place across the host link)."""
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        if not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or a pinned host tensor")
        return (mapped_host_pointer(t) if t.numel() else None) or None
    return t.data_ptr() or None


def _empty_beside(shape, dtype, t):
    """An output tensor where input ``t`` lives: on its CUDA device, or in
    pinned host memory for a host input."""
    torch = _torch()
    if t.is_cuda:
        return torch.empty(shape, dtype=dtype, device=t.device)
    return torch.empty(shape, dtype=dtype, pin_memory=True)


def _cuda_device(t):
    """The device a call on tensor ``t`` runs on: its own, or the current
    CUDA device for a pinned host tensor."""
    torch = _torch()
    return t.device if t.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _logits_kind(t, name="logits"):
    """(dtype, C-ABI name suffix) of a logits tensor: fp32 or bf16."""
    torch = _torch()
    if t.dtype == torch.float32:
        return torch.float32, ""
    if t.dtype == torch.bfloat16:
        return torch.bfloat16, "_bf16"
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _row_major(t, name):
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return t.stride(-2) if t.dim() >= 2 else t.shape[-1]


def dsa_block_scores(logits, row_ks, row_ke, block_size: int, row_repeat: int = 1,
                     pin_newest: bool = True, scores_out=None, stream=None):
    """Block scores ``[rows, ceil(width / block_size)]`` in the logits' dtype
    (fp32 or bf16; returned)."""
    torch = _torch()
    dt, sfx = _logits_kind(logits)
    rows, width = logits.shape
    nb = -(-width // block_size) if block_size > 0 else 0
    if scores_out is None:
        scores_out = _empty_beside((rows, nb), dt, logits)
    st = getattr(library(), "dsa_block_scores" + sfx)(
        _dev_ptr(logits, dt, "logits"), rows, width, _row_major(logits, "logits"),
        _dev_ptr(row_ks, torch.int32, "row_ks", allow_none=True),
        _dev_ptr(row_ke, torch.int32, "row_ke"), block_size, row_repeat, int(bool(pin_newest)),
        _dev_ptr(scores_out, dt, "scores_out"),
        _row_major(scores_out, "scores_out") if scores_out.numel() else nb,
        _stream_handle(stream))
    _check("dsa_block_scores" + sfx, st)
    return scores_out


def dsa_select_candidate_blocks(logits, row_ks, row_ke, topk_blocks: int, block_size: int,
                                out, row_repeat: int = 1, pin_newest: bool = True,
                                scores_out=None, stream=None, workspace=None):
    """Write ranked candidate block ids (-1 padded) into ``out`` [rows, >=topk]
    int32; optionally the block scores into ``scores_out`` (the logits'
    dtype). Logits are fp32 or bf16. ``workspace``: see ``_workspace``."""
    torch = _torch()
    dt, sfx = _logits_kind(logits)
    rows, width = logits.shape
    nb = -(-width // block_size) if block_size > 0 else 0
    handle = _stream_handle(stream)
    ws_ptr, ws_bytes = _workspace(workspace, rows, nb, _cuda_device(logits), handle)
    st = getattr(library(), "dsa_select_candidate_blocks" + sfx)(
        _dev_ptr(logits, dt, "logits"), rows, width, _row_major(logits, "logits"),
        _dev_ptr(row_ks, torch.int32, "row_ks", allow_none=True),
        _dev_ptr(row_ke, torch.int32, "row_ke"), topk_blocks, block_size, row_repeat,
        int(bool(pin_newest)), _dev_ptr(out, torch.int32, "out"),
        _row_major(out, "out") if out.dim() == 2 else topk_blocks,
        _dev_ptr(scores_out, dt, "scores_out", allow_none=True),
        _row_major(scores_out, "scores_out") if scores_out is not None else 0,
        ws_ptr, ws_bytes, handle)
    _check("dsa_select_candidate_blocks" + sfx, st)
    return out


def dsa_select_candidate_blocks_sharded(logits, global_row_ke, global_block_size: int,
                                        max_global_blocks: int, topk_blocks: int, out,
                                        row_repeat: int = 1, scores_out=None, stream=None,
                                        workspace=None, global_row_ks=None):
    """DCP form: ``logits`` is ``[D, rows, local_width]`` (unit stride in the last
    dimension); writes ranked global block ids into ``out``. ``global_row_ks``
    (optional) gives global window starts (the ``_starts`` C entry point).
    ``workspace``: see ``_workspace``."""
    torch = _torch()
    dt, sfx = _logits_kind(logits)
    shards, rows, lw = logits.shape
    handle = _stream_handle(stream)
    ws_ptr, ws_bytes = _workspace(workspace, rows, max(int(max_global_blocks), 1),
                                  _cuda_device(logits), handle)
    if logits.stride(2) != 1:
        raise ValueError("logits must have unit stride in its last dimension")
    name = "dsa_select_candidate_blocks_sharded" + ("_starts" if global_row_ks is not None
                                                    else "") + sfx
    starts = (_dev_ptr(global_row_ks, torch.int32, "global_row_ks"),) \
        if global_row_ks is not None else ()
    st = getattr(library(), name)(
        _dev_ptr(logits, dt, "logits"), shards, rows, lw, logits.stride(1),
        logits.stride(0), *starts, _dev_ptr(global_row_ke, torch.int32, "global_row_ke"),
        global_block_size, max_global_blocks, row_repeat, topk_blocks,
        _dev_ptr(out, torch.int32, "out"), _row_major(out, "out") if out.dim() == 2 else topk_blocks,
        _dev_ptr(scores_out, dt, "scores_out", allow_none=True),
        _row_major(scores_out, "scores_out") if scores_out is not None else 0,
        ws_ptr, ws_bytes, handle)
    _check(name, st)
    return out


def dsa_mask_candidate_logits(logits, row_ks, row_ke, candidates, block_size: int,
                              row_repeat: int = 1, stream=None):
    """In place: -inf for every logit outside its row's window or outside the
    row's candidate blocks (``candidates`` [rows, topk] int32, -1 = empty)."""
    torch = _torch()
    dt, sfx = _logits_kind(logits)
    rows, width = logits.shape
    topk = candidates.shape[1] if candidates is not None else 0
    st = getattr(library(), "dsa_mask_candidate_logits" + sfx)(
        _dev_ptr(logits, dt, "logits"), rows, width, _row_major(logits, "logits"),
        _dev_ptr(row_ks, torch.int32, "row_ks", allow_none=True),
        _dev_ptr(row_ke, torch.int32, "row_ke"),
        _dev_ptr(candidates, torch.int32, "candidates", allow_none=True), topk,
        _row_major(candidates, "candidates") if candidates is not None else 0, block_size,
        row_repeat, _stream_handle(stream))
    _check("dsa_mask_candidate_logits" + sfx, st)
    return logits


def dsa_mask_candidate_logits_sharded(logits, global_row_ke, global_block_size: int, candidates,
                                      row_repeat: int = 1, stream=None, global_row_ks=None):
    """DCP form of ``dsa_mask_candidate_logits`` on ``[D, rows, local_width]``;
    ``global_row_ks`` (optional) gives global window starts."""
    torch = _torch()
    dt, sfx = _logits_kind(logits)
    shards, rows, lw = logits.shape
    if logits.stride(2) != 1:
        raise ValueError("logits must have unit stride in its last dimension")
    topk = candidates.shape[1] if candidates is not None else 0
    name = "dsa_mask_candidate_logits_sharded" + ("_starts" if global_row_ks is not None
                                                  else "") + sfx
    starts = (_dev_ptr(global_row_ks, torch.int32, "global_row_ks"),) \
        if global_row_ks is not None else ()
    st = getattr(library(), name)(
        _dev_ptr(logits, dt, "logits"), shards, rows, lw, logits.stride(1),
        logits.stride(0), *starts, _dev_ptr(global_row_ke, torch.int32, "global_row_ke"),
        global_block_size, row_repeat,
        _dev_ptr(candidates, torch.int32, "candidates", allow_none=True), topk,
        _row_major(candidates, "candidates") if candidates is not None else 0,
        _stream_handle(stream))
    _check(name, st)
    return logits


DTYPE_F32, DTYPE_BF16 = 0, 1


def _attn_dtype(t, name):
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _attn_ptr(t, name, dtype_code):
    torch = _torch()
    want = torch.float32 if dtype_code == DTYPE_F32 else torch.bfloat16
    return _dev_ptr(t, want, name)


def dsa_correct_attn_out(out, lses, rank: int, new_out=None, lse_out=None, stream=None):
    """DCP LSE correction of shard ``rank``'s partial attention output.

    ``out`` [B, H, Dh] (or [B, 1, H, Dh]) fp32 or bf16; ``lses`` [N, B, H]
    fp32 base-2 LSEs of all shards (a trailing or second size-1 dimension is
    squeezed, as on the page). Writes ``new_out`` [H, B, Dh] (allocated when
    None, same dtype as ``out``) and the combined LSE ``lse_out`` [B, H]
    fp32 (allocated when None); returns both."""
    torch = _torch()
    if out.dim() == 4 and out.shape[1] == 1:
        out = out.squeeze(1)
    if lses.dim() == 4 and lses.shape[-1] == 1:
        lses = lses.squeeze(-1)
    if lses.dim() == 4 and lses.shape[1] == 1:
        lses = lses.squeeze(1)
    if out.dim() != 3 or lses.dim() != 3:
        raise ValueError("expected out [B, H, Dh] and lses [N, B, H]")
    B, H, D = out.shape
    N = lses.shape[0]
    if tuple(lses.shape[1:]) != (B, H):
        raise ValueError(f"lses {tuple(lses.shape)} does not match out {tuple(out.shape)}")
    code = _attn_dtype(out, "out")
    if new_out is None:
        new_out = _empty_beside((H, B, D), out.dtype, out)
    if lse_out is None:
        lse_out = _empty_beside((B, H), torch.float32, out)
    if tuple(new_out.shape) != (H, B, D) or tuple(lse_out.shape) != (B, H):
        raise ValueError("new_out must be [H, B, Dh] and lse_out [B, H]")
    st = library().dsa_correct_attn_out(
        _attn_ptr(out, "out", code), code, B, H, D, *out.stride(),
        _dev_ptr(lses, torch.float32, "lses"), N, *lses.stride(), rank,
        _attn_ptr(new_out, "new_out", code), *new_out.stride(),
        _dev_ptr(lse_out, torch.float32, "lse_out"), *lse_out.stride(), _stream_handle(stream))
    _check("dsa_correct_attn_out", st)
    return new_out, lse_out


def dsa_merge_attn_out(outs, lses, merged=None, lse_out=None, stream=None):
    """Sum over shards of the corrected partial outputs.

    ``outs`` [N, B, H, Dh] fp32 or bf16, ``lses`` [N, B, H] fp32. Writes
    ``merged`` [H, B, Dh] (same dtype as ``outs``) and ``lse_out`` [B, H]
    fp32, allocating them when None; returns both."""
    torch = _torch()
    if outs.dim() != 4 or lses.dim() != 3:
        raise ValueError("expected outs [N, B, H, Dh] and lses [N, B, H]")
    N, B, H, D = outs.shape
    if tuple(lses.shape) != (N, B, H):
        raise ValueError(f"lses {tuple(lses.shape)} does not match outs {tuple(outs.shape)}")
    code = _attn_dtype(outs, "outs")
    if merged is None:
        merged = _empty_beside((H, B, D), outs.dtype, outs)
    if lse_out is None:
        lse_out = _empty_beside((B, H), torch.float32, outs)
    if tuple(merged.shape) != (H, B, D) or tuple(lse_out.shape) != (B, H):
        raise ValueError("merged must be [H, B, Dh] and lse_out [B, H]")
    st = library().dsa_merge_attn_out(
        _attn_ptr(outs, "outs", code), code, N, B, H, D, *outs.stride(),
        _dev_ptr(lses, torch.float32, "lses"), *lses.stride(),
        _attn_ptr(merged, "merged", code), *merged.stride(),
        _dev_ptr(lse_out, torch.float32, "lse_out"), *lse_out.stride(), _stream_handle(stream))
    _check("dsa_merge_attn_out", st)
    return merged, lse_out


DTYPE_F16 = 2


class _Launch:
    """The device of a call's tensors made current and, for a given
    ``stream``, that stream, so that what the call allocates belongs to the
    stream that it runs on."""

    def __init__(self, index, stream):
        torch = _torch()
        self._guards = [torch.cuda.device(index)]
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


def _call(index: int, stream, enqueue, *args):
    """``enqueue(*args, stream handle)`` with device ``index`` and ``stream``
    current; nothing is switched for the usual call, on the current stream of
    the current device."""
    c = _torch()._C
    if stream is None and index == c._cuda_getDevice():
        return enqueue(*args, c._cuda_getCurrentRawStream(index) or None)
    with _Launch(index, stream):
        return enqueue(*args, c._cuda_getCurrentRawStream(index) or None)


def _on_gpu(t, dtype, name, dim, index=None):
    """Address, shape and strides of a CUDA tensor of the given type and rank
    on device ``index``."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {tuple(shape)}")
    if at != index and index is not None:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return t.data_ptr() or None, shape, t.stride()


def _row_strides(shape, strides, name):
    """Strides of all dimensions but the last, which has unit stride. A
    dimension of one element is never stepped over: any stride will do."""
    last = shape[-1]
    if strides[-1] != 1 and last > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    if 1 in shape:
        return tuple(st if n != 1 else last for n, st in zip(shape[:-1], strides[:-1]))
    return strides[:-1]


def _vector(t, name, index):
    """Address and length of a contiguous int32 vector."""
    at = t.get_device()
    if at != index or t.dtype is not _torch().int32 or t.dim() != 1:
        _on_gpu(t, _torch().int32, name, 1, index)
    n = t.shape[0]
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None, n


def _attention_dtype(t, name):
    torch = _torch()
    dt = t.dtype
    if dt is torch.bfloat16:
        return DTYPE_BF16
    if dt is torch.float16:
        return DTYPE_F16
    raise TypeError(f"{name} must be bfloat16 or float16, got {dt}")


def _attention_outputs(q, shape, index, out, lse_out):
    """Output tensors (allocated when None) and their addresses and strides."""
    torch = _torch()
    T, H, D = shape
    device = q.device
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
        o = out.data_ptr(), H * D, D
    else:
        op, oshape, ost = _on_gpu(out, q.dtype, "out", 3, index)
        if oshape != shape:
            raise ValueError(f"out must be {tuple(shape)}, got {tuple(oshape)}")
        o = op, *_row_strides(oshape, ost, "out")
    if lse_out is None:
        lse_out = torch.empty((T, H), dtype=torch.float32, device=device)
        l = lse_out.data_ptr(), H, 1
    else:
        lp, lshape, lst = _on_gpu(lse_out, torch.float32, "lse_out", 2, index)
        if lshape != shape[:2]:
            raise ValueError(f"lse_out must be {tuple(shape[:2])}, got {tuple(lshape)}")
        l = lp, *lst
    return out, lse_out, (*o, *l)


def _scale(scale, dim):
    return (dim ** -0.5 if dim else 1.0) if scale is None else float(scale)


def dsa_prompt_attention(q, k, v, cu_q, cu_k, *, causal: bool = True, scale=None, out=None,
                         lse_out=None, workspace=None, stream=None):
    """Attention over packed prompts with grouped heads.

    ``q`` [Tq, H, D], ``k`` and ``v`` [Tk, Hkv, D] bfloat16 or float16, D a
    multiple of 8 up to 128; sequence i's queries are rows cu_q[i]:cu_q[i+1]
    and its keys rows cu_k[i]:cu_k[i+1] (int32 CUDA tensors of equal length).
    ``causal``: the last query of a sequence sees all of its keys, each
    earlier one a key less. ``scale`` defaults to 1/sqrt(D). Writes ``out``
    [Tq, H, D] and the base-2 log-sum-exp ``lse_out`` [Tq, H] fp32 (allocated
    when None) and returns both; rows that see no key get 0 and -inf, rows of
    no sequence are left as they were. ``workspace``: a CUDA uint8 tensor of
    ``prompt_workspace_bytes(...)`` bytes that no overlapping call uses
    (None: one kept for this thread and stream). Forward only: the outputs carry no autograd
    graph."""
    code = _attention_dtype(q, "q")
    dt, dev = q.dtype, q.get_device()
    qp, qs, qst = _on_gpu(q, dt, "q", 3)
    kp, ks, kst = _on_gpu(k, dt, "k", 3, dev)
    vp, vs, vst = _on_gpu(v, dt, "v", 3, dev)
    if ks != vs or ks[2] != qs[2]:
        raise ValueError(f"q {tuple(qs)}, k {tuple(ks)} and v {tuple(vs)} do not match")
    (cq, nq), (ck, nk) = _vector(cu_q, "cu_q", dev), _vector(cu_k, "cu_k", dev)
    if nq != nk or nq < 1:
        raise ValueError(f"cu_q and cu_k must have one length of at least 1, got {nq} and {nk}")
    T, H, D = qs
    Tk, Hkv, _ = ks
    args = (qp, kp, vp, code, T, Tk, H, Hkv, D, *_row_strides(qs, qst, "q"),
            *_row_strides(ks, kst, "k"), *_row_strides(vs, vst, "v"), cq, ck, nq - 1,
            1 if causal else 0, _scale(scale, D))

    def enqueue(out, lse_out, handle):
        out, lse_out, outs = _attention_outputs(q, qs, dev, out, lse_out)
        held, ws, ws_bytes = _scratch(
            workspace, _need("dsa_prompt_workspace_bytes", dev, T, Tk, H, Hkv, D, nq - 1), q,
            handle)
        st = library().dsa_prompt_attention(*args, *outs, ws, ws_bytes, handle)
        if st:
            _check("dsa_prompt_attention", st)
        return out, lse_out

    return _call(dev, stream, enqueue, out, lse_out)


def prompt_workspace_bytes(total_q: int, total_k: int, heads: int, kv_heads: int, head_dim: int,
                           seqs: int) -> int:
    """Bytes of workspace of a ``dsa_prompt_attention`` call."""
    return library().dsa_prompt_workspace_bytes(total_q, total_k, heads, kv_heads, head_dim, seqs)


def dsa_shared_prefix_attention(q, k_pages, v_pages, tables, lens, prefix_len: int = 0, *,
                                prefix_pages=None, scale=None, out=None, lse_out=None,
                                workspace=None, stream=None):
    """Attention of one query token per sequence on a paged cache, the first
    ``prefix_len`` tokens of which (whole pages) are the same for the batch.

    ``q`` [B, H, D] bfloat16 or float16; ``k_pages`` and ``v_pages`` [N, page,
    Hkv, D]; token t of sequence b lies on page ``tables``[b, t // page]
    (int32 [B, P]); the sequence sees its first ``lens``[b] tokens (int32
    [B]). The prefix is read once, through ``prefix_pages`` (int32, by default
    the first row of ``tables`` that is not an empty slot's, of length 0 and
    with a negative first entry; ``tables[0]`` stands for that too); 0 gives
    plain paged decode attention. Pages
    numbered outside [0, N) are not seen. Writes ``out`` [B, H, D] and the
    base-2 log-sum-exp ``lse_out`` [B, H] fp32 (allocated when None) and
    returns both; a sequence that sees no token gets 0 and -inf.
    ``workspace``: a CUDA uint8 tensor of
    ``shared_prefix_workspace_bytes(...)`` bytes that no overlapping call
    uses (None: one kept for this thread and stream). Forward only, as
    ``dsa_prompt_attention``."""
    torch = _torch()
    code = _attention_dtype(q, "q")
    dt, dev = q.dtype, q.get_device()
    qp, qs, qst = _on_gpu(q, dt, "q", 3)
    B, H, D = qs
    kp, ks, kst = _on_gpu(k_pages, dt, "k_pages", 4, dev)
    vp, vs, vst = _on_gpu(v_pages, dt, "v_pages", 4, dev)
    tp, (Bt, P), tst = _on_gpu(tables, torch.int32, "tables", 2, dev)
    lp, n = _vector(lens, "lens", dev)
    N, page, Hkv, Dk = ks
    if ks != vs or Dk != D:
        raise ValueError(f"q {tuple(q.shape)}, k_pages {tuple(ks)} and v_pages {tuple(vs)} do "
                         "not match")
    if n != B or Bt != B:
        raise ValueError(f"tables {tuple(tables.shape)} and lens {tuple(lens.shape)} do not "
                         f"match q {tuple(q.shape)}")
    if P > 1 and tst[1] != 1:
        raise ValueError("tables must have unit stride in its last dimension")
    prefix_len = int(prefix_len)
    pp = None
    if prefix_len > 0:
        if prefix_pages is None:
            pp = tp
        else:
            pp, n = _vector(prefix_pages, "prefix_pages", dev)
            if page > 0 and n < prefix_len // page:
                raise ValueError(f"prefix_pages holds {n} pages, prefix_len {prefix_len} needs "
                                 f"{prefix_len // page}")
    args = (qp, kp, vp, code, B, H, Hkv, D, N, page, *_row_strides(qs, qst, "q"),
            *_row_strides(ks, kst, "k_pages"), *_row_strides(vs, vst, "v_pages"), pp, prefix_len,
            tp, P, tst[0] if B > 1 else P, lp, _scale(scale, D))

    def enqueue(out, lse_out, handle):
        out, lse_out, outs = _attention_outputs(q, qs, dev, out, lse_out)
        held, ws, ws_bytes = _scratch(
            workspace, _need("dsa_shared_prefix_workspace_bytes", dev, B, H, Hkv, D, prefix_len, P,
                             page), q, handle)
        st = library().dsa_shared_prefix_attention(*args, *outs, ws, ws_bytes, handle)
        if st:
            _check("dsa_shared_prefix_attention", st)
        return out, lse_out

    return _call(dev, stream, enqueue, out, lse_out)


def shared_prefix_workspace_bytes(batch: int, heads: int, kv_heads: int, head_dim: int,
                                  prefix_len: int, max_pages: int, page_size: int) -> int:
    """Bytes of workspace of a ``dsa_shared_prefix_attention`` call."""
    return library().dsa_shared_prefix_workspace_bytes(batch, heads, kv_heads, head_dim,
                                                       prefix_len, max_pages, page_size)


@functools.lru_cache(maxsize=4096)
def _need(name: str, index: int, *sizes) -> int:
    """A workspace's bytes on device ``index`` (the current one)."""
    return getattr(library(), name)(*sizes)


_KEEP_BYTES = 64 << 20
_KEEP_ALL_BYTES = 256 << 20
_scratch_cache = {}  # in the order of their allocation
_scratch_lock = threading.Lock()


def _scratch(workspace, need: int, like, handle):
    """A call's workspace, held until the call is enqueued, with its address
    and bytes: the caller's tensor, or one of its own on ``like``'s device.

    Its own one is kept for the next call of this thread on this stream (the
    stream itself, not its handle, which another one may get), whose calls
    follow each other; larger ones than 64 MiB, and those of a capture (whose
    graph may run beside other calls), come from the allocator of the current
    stream or graph, which hands their memory on only behind this call. So
    does what is let go: the oldest ones over 256 MiB in all."""
    if workspace is None:
        if not need:
            return None, None, 0
        torch = _torch()
        if need > _KEEP_BYTES or torch._C._cuda_isCurrentStreamCapturing():
            workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
            return workspace, workspace.data_ptr(), need
        # the default stream (no handle) is never destroyed
        stream = handle if handle is None else library().dsa_stream_id(handle)
        key = threading.get_ident(), like.get_device(), stream
        kept = _scratch_cache.get(key)
        if kept is None or kept[2] < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
            kept = workspace, workspace.data_ptr(), need
            with _scratch_lock:
                _scratch_cache.pop(key, None)
                _scratch_cache[key] = kept
                over = sum(k[2] for k in _scratch_cache.values()) - _KEEP_ALL_BYTES
                while over > 0:
                    over -= _scratch_cache.pop(next(iter(_scratch_cache)))[2]
        return kept
    if not workspace.is_cuda or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    n = workspace.numel() * workspace.element_size()
    return workspace, workspace.data_ptr() if n else None, n


def release_workspaces() -> None:
    """Let go of the workspaces that attention and cache calls keep (up to 256
    MiB in all); their memory goes back to PyTorch's allocator. Calls under
    way are not disturbed."""
    with _scratch_lock:
        _scratch_cache.clear()


FORK_OK, FORK_NO_PAGE, FORK_REFUSED = 0, 1, 2


def _cache_state(refs, tables, lens):
    """Arguments that describe refs, tables and lens, and their device."""
    tp, (S, P), (ld, one) = _on_gpu(tables, _torch().int32, "tables", 2)
    dev = tables.get_device()
    rp, pages = _vector(refs, "refs", dev)
    if P > 1 and one != 1:
        raise ValueError("tables must have unit stride in its last dimension")
    if S > 1 and ld < P:
        raise ValueError("rows of tables must not overlap")
    lp = None
    if lens is not None:
        lp, n = _vector(lens, "lens", dev)
        if n != S:
            raise ValueError(f"lens holds {n} lengths, tables {S} rows")
    return rp, pages, tp, S, P, ld if S > 1 else P, lp, dev


def _cache_planes(cache, pages, index):
    """Arguments that describe the page contents [planes, N, page, ...]."""
    at = cache.get_device()
    if at < 0:
        raise ValueError("cache must be a CUDA tensor")
    if at != index:
        raise ValueError(f"cache is on {cache.device}, expected cuda:{index}")
    shape, strides, e = cache.shape, cache.stride(), cache.element_size()
    if len(shape) < 3 or shape[1] != pages:
        raise ValueError(f"cache must be [planes, {pages}, page, ...], got {tuple(shape)}")
    inner = 1
    for d in range(len(shape) - 1, 1, -1):
        if shape[d] > 1 and strides[d] != inner:
            raise ValueError("the pages of cache must be contiguous")
        if d > 2:
            inner *= shape[d]
    token, page = inner * e, inner * e * shape[2]
    plane_st = strides[0] * e if shape[0] > 1 else page
    page_st = strides[1] * e if pages > 1 else page
    if plane_st < page or page_st < page:
        raise ValueError("the pages of cache must not overlap")
    return cache.data_ptr() or None, shape[0], plane_st, pages, page_st, shape[2], token


def dsa_cache_fork(cache, refs, tables, lens, parents, children, *, status=None, workspace=None,
                   stream=None):
    """Make slot children[i] a copy of slot parents[i] (int32 CUDA vectors).

    ``cache`` [planes, N, page, ...] of any type (pages contiguous, tokens of
    a multiple of 16 bytes), ``refs`` int32 [N], ``tables`` int32 [S, P],
    ``lens`` int32 [S]. Whole pages are shared; the used tokens of a partly
    filled last page are copied to the lowest free page. Returns ``status``
    int32 (FORK_OK, FORK_NO_PAGE or FORK_REFUSED for each pair), allocated
    when None; the host waits for nothing."""
    torch = _torch()
    rp, pages, tp, S, P, ld, lp, dev = _cache_state(refs, tables, lens)
    planes = _cache_planes(cache, pages, dev)
    (pp, n), (cp, nc) = _vector(parents, "parents", dev), _vector(children, "children", dev)
    if n != nc:
        raise ValueError(f"{n} parents, {nc} children")

    def enqueue(status, handle):
        if status is None:
            status = torch.empty(n, dtype=torch.int32, device=refs.device)
        sp, ns = _vector(status, "status", dev)
        if ns != n:
            raise ValueError(f"status holds {ns} entries, expected {n}")
        held, ws, ws_bytes = _scratch(
            workspace, _need("dsa_cache_workspace_bytes", dev, n, pages) if n else 0, refs, handle)
        st = library().dsa_cache_fork(*planes, rp, tp, S, P, ld, lp, pp, cp, n, sp, ws, ws_bytes,
                                       handle)
        if st:
            _check("dsa_cache_fork", st)
        return status

    return _call(dev, stream, enqueue, status)


def dsa_cache_free(refs, tables, lens, seqs, *, stream=None):
    """Empty the slots named in ``seqs`` (int32 CUDA vector): their pages'
    refs go down by one, their rows become -1 and their lengths 0."""
    rp, pages, tp, S, P, ld, lp, dev = _cache_state(refs, tables, lens)
    sp, n = _vector(seqs, "seqs", dev)
    st = _call(dev, stream, library().dsa_cache_free, rp, pages, tp, S, P, ld, lp, sp, n)
    if st:
        _check("dsa_cache_free", st)


def dsa_cache_compact(cache, refs, tables, *, remap=None, live=None, workspace=None, stream=None):
    """Move the pages in use to the lowest numbers (contents in all planes,
    refs and table entries). Returns ``remap`` int32 [N], the new number of
    each used page (-1 for free ones), and ``live`` int32 [1], how many are in
    use; allocated when None."""
    torch = _torch()
    rp, pages, tp, S, P, ld, _, dev = _cache_state(refs, tables, None)
    planes = _cache_planes(cache, pages, dev)

    def enqueue(remap, live, handle):
        if remap is None:
            remap = torch.empty(pages, dtype=torch.int32, device=refs.device)
        if live is None:
            live = torch.empty(1, dtype=torch.int32, device=refs.device)
        (mp, n), (vp, one) = _vector(remap, "remap", dev), _vector(live, "live", dev)
        if n != pages or one != 1:
            raise ValueError(f"remap must have {pages} entries and live one")
        held, ws, ws_bytes = _scratch(
            workspace, _need("dsa_cache_workspace_bytes", dev, 0, pages), refs, handle)
        st = library().dsa_cache_compact(*planes, rp, tp, S, P, ld, mp, vp, ws, ws_bytes, handle)
        if st:
            _check("dsa_cache_compact", st)
        return remap, live

    return _call(dev, stream, enqueue, remap, live)


def cache_workspace_bytes(pairs: int, num_pages: int) -> int:
    """Bytes of workspace of ``dsa_cache_fork`` (of ``pairs`` pairs) or, with
    0 pairs, of ``dsa_cache_compact``."""
    return library().dsa_cache_workspace_bytes(pairs, num_pages)


def _to_device(host, dev_buf, stream):
    torch = _torch()
    if host is None:
        return None
    if dev_buf is None:
        dev_buf = torch.empty(host.shape, dtype=host.dtype, device="cuda")
    with torch.cuda.stream(stream):
        dev_buf.copy_(host, non_blocking=True)
    return dev_buf


def _all_pinned(*ts) -> bool:
    return all(t is None or (not t.is_cuda and t.is_pinned()) for t in ts)


def select_candidate_blocks_host(logits, row_ks, row_ke, topk_blocks: int, block_size: int,
                                 row_repeat: int = 1, pin_newest: bool = True, *,
                                 out=None, device_buffers: Optional[dict] = None, stream=None,
                                 in_place: bool = True):
    """Host-memory form of ``dsa_select_candidate_blocks``; waits for the
    result and returns the ids in host tensor ``out`` (pinned; allocated when
    None).

    Pinned inputs are read in place (unless ``in_place`` is False): the
    kernel reads only the in-window logits across the host link and writes
    the ids straight into ``out``. Other host tensors are first copied to the
    device whole; ``device_buffers``
    may then hold preallocated device tensors under 'logits', 'row_ks',
    'row_ke', 'out' so that repeated calls allocate nothing. A device
    tensor under 'workspace' is passed on as the call's workspace."""
    torch = _torch()
    stream = torch.cuda.current_stream() if stream is None else stream
    db = device_buffers if device_buffers is not None else {}
    rows = logits.shape[0]
    if out is None:
        out = torch.empty((rows, topk_blocks), dtype=torch.int32, pin_memory=True)
    if in_place and _all_pinned(logits, row_ks, row_ke, out):
        dsa_select_candidate_blocks(logits, row_ks, row_ke, topk_blocks, block_size, out,
                                    row_repeat, pin_newest, stream=stream,
                                    workspace=db.get("workspace"))
        stream.synchronize()
        return out
    d_logits = _to_device(logits, db.get("logits"), stream)
    d_ks = _to_device(row_ks, db.get("row_ks"), stream)
    d_ke = _to_device(row_ke, db.get("row_ke"), stream)
    d_out = db.get("out")
    if d_out is None:
        d_out = torch.empty((rows, topk_blocks), dtype=torch.int32, device="cuda")
    dsa_select_candidate_blocks(d_logits, d_ks, d_ke, topk_blocks, block_size, d_out,
                                row_repeat, pin_newest, stream=stream,
                                workspace=db.get("workspace"))
    with torch.cuda.stream(stream):
        out.copy_(d_out, non_blocking=True)
    stream.synchronize()
    return out


def select_candidate_blocks_sharded_host(logits, global_row_ke, global_block_size: int,
                                         max_global_blocks: int, topk_blocks: int,
                                         row_repeat: int = 1, *, out=None,
                                         device_buffers: Optional[dict] = None, stream=None,
                                         global_row_ks=None, in_place: bool = True):
    """Host-memory form of ``dsa_select_candidate_blocks_sharded`` (see
    ``select_candidate_blocks_host``: pinned inputs are read in place;
    ``device_buffers`` may also hold 'global_row_ke' and 'global_row_ks')."""
    torch = _torch()
    stream = torch.cuda.current_stream() if stream is None else stream
    db = device_buffers if device_buffers is not None else {}
    rows = logits.shape[1]
    if out is None:
        out = torch.empty((rows, topk_blocks), dtype=torch.int32, pin_memory=True)
    if in_place and _all_pinned(logits, global_row_ke, global_row_ks, out):
        dsa_select_candidate_blocks_sharded(logits, global_row_ke, global_block_size,
                                            max_global_blocks, topk_blocks, out, row_repeat,
                                            stream=stream, workspace=db.get("workspace"),
                                            global_row_ks=global_row_ks)
        stream.synchronize()
        return out
    d_logits = _to_device(logits, db.get("logits"), stream)
    d_gke = _to_device(global_row_ke, db.get("global_row_ke"), stream)
    d_gks = _to_device(global_row_ks, db.get("global_row_ks"), stream)
    d_out = db.get("out")
    if d_out is None:
        d_out = torch.empty((rows, topk_blocks), dtype=torch.int32, device="cuda")
    dsa_select_candidate_blocks_sharded(d_logits, d_gke, global_block_size, max_global_blocks,
                                        topk_blocks, d_out, row_repeat, stream=stream,
                                        global_row_ks=d_gks, workspace=db.get("workspace"))
    with torch.cuda.stream(stream):
        out.copy_(d_out, non_blocking=True)
    stream.synchronize()
    return out
