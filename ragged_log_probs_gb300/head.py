"""The operators of a served model's head around the ragged log-probability path: final
norm, vocabulary projection with low-rank adapters, processing of logits.

Signatures and documentation only. The checks and the call are compiled
(``csrc/lp_head_binding.cpp``), since these functions run once a token; every operator runs in
the CUDA kernels of ``liblp_ragged.so`` behind the C ABI of ``include/lp_head.h``, whose
comments define it. Matrices may have any row stride, with their last dimension contiguous.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import torch

from . import _build

__all__ = ["head_workspace_size", "new_head_workspace", "clear_status", "rms_norm", "project", "project_cut",
           "process_logits"]

LP_MAX_HIDDEN = 32768
LP_MAX_RANK = 64


def _declare(lib: ctypes.CDLL) -> None:
    u32, u64, vp, sz, f32 = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    lib.lp_head_workspace_size.argtypes = [u32, u32]
    lib.lp_head_workspace_size.restype = sz
    lib.lp_head_clear_status.argtypes = [vp, vp]
    lib.lp_head_clear_status.restype = ctypes.c_int
    lib.lp_head_norm.argtypes = [vp, vp, vp, u32, u32, u32, u32, u64, u64, vp, u32, f32, vp, u32, u64, vp, vp, u64,
                                 vp, sz, vp]
    lib.lp_head_norm.restype = ctypes.c_int
    lib.lp_head_project.argtypes = [vp, u32, u32, u32, u64, vp, vp, u32, u64, vp, vp, vp, u32, u32, u32, vp, vp, vp,
                                    u32, vp, u32, u64, vp, sz, vp]
    lib.lp_head_project.restype = ctypes.c_int
    lib.lp_head_project_cut.argtypes = [u32] * 7 + [vp] * 3
    lib.lp_head_project_cut.restype = ctypes.c_int
    lib.lp_head_process.argtypes = [vp, u32, u32, u32, u64, vp, u32, vp, vp, u32, vp, vp, vp, vp, vp, vp, vp, u32,
                                    vp, u64, u32, vp, vp, u64, vp, sz, vp]
    lib.lp_head_process.restype = ctypes.c_int
    lib.lp_head_process_workspace_size.argtypes = [u32, u32]
    lib.lp_head_process_workspace_size.restype = sz


def _pkg():
    import ragged_log_probs_gb300 as lp
    return lp


_native = None


def _failed(rc: int, what: str) -> None:
    raise _pkg().LpError(rc, what)


def _load():
    """Load the compiled binding (built with the library); raise if it is missing."""
    global _native
    _pkg().load()
    path = _build.binding_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: run __graft_entry__.build() first")
    spec = importlib.util.spec_from_file_location("lp_head_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.on_failure(_failed)
    _native = module
    return module


def head_workspace_size(T: int = 0, rank: int = 0, requests: int = 0, history: int = 0) -> int:
    """Bytes of scratch that serve every call of up to these sizes: ``project`` with adapters of
    that rank over T rows, ``process_logits`` of that many requests with that many history
    tokens in all (0: only the status word)."""
    lib = _pkg().load()
    n = int(lib.lp_head_workspace_size(T, rank))
    if n == 0:
        raise ValueError(f"rank {rank} exceeds {LP_MAX_RANK}")
    return max(n, int(lib.lp_head_process_workspace_size(requests, history)))


def new_head_workspace(T: int = 0, rank: int = 0, requests: int = 0, history: int = 0, device=None) -> torch.Tensor:
    """A zeroed workspace (uint8) of ``head_workspace_size``. Its status word collects the
    bits of every call that is given it, until ``clear_status``; ``read_status`` reads it."""
    return torch.zeros(head_workspace_size(T, rank, requests, history), dtype=torch.uint8,
                       device=torch.device("cuda") if device is None else device)


def clear_status(workspace: torch.Tensor, stream=None) -> None:
    """Enqueue the clearing of a workspace's status word."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.clear_status(workspace)
    return native.clear_status(workspace)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
             rows: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
             out: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Final norm: ``(x + residual) / rms * weight`` of all rows of ``x`` [T, H], or of those
    that ``rows`` [n] names (the scored positions only).

    ``out`` (or a new tensor of ``out_dtype``, default x's) is of x's type, float32, or
    float8_e4m3fn with one float32 scale a row in ``out_scale``. ``residual_out`` receives
    ``x + residual``. Returns ``out``, or ``(out, out_scale)`` for float8_e4m3fn. With
    ``rows`` a workspace is needed: a row index past T sets LP_ERR_OFFSETS in its status."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):  # (what is allocated here belongs to that stream too)
            return native.rms_norm(x, weight, eps, residual, rows, out_dtype, out, out_scale, residual_out, workspace)
    return native.rms_norm(x, weight, eps, residual, rows, out_dtype, out, out_scale, residual_out, workspace)


def project(x: torch.Tensor, weight: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
            weight_scale: Optional[torch.Tensor] = None, lora_a: Optional[torch.Tensor] = None,
            lora_b: Optional[torch.Tensor] = None, adapter_scale: Optional[torch.Tensor] = None,
            adapter_ids: Optional[torch.Tensor] = None, row_offsets: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, *, workspace: torch.Tensor,
            stream=None) -> torch.Tensor:
    """Logits ``x @ weight.T`` [T, V] of hidden states ``x`` [T, H], plus each request's
    low-rank adapter ``adapter_scale[a] * (x @ lora_a[a].T) @ lora_b[a].T``.

    ``x`` and ``weight`` [V, H] are bfloat16, float16, or float8_e4m3fn with ``x_scale`` [T]
    and ``weight_scale`` [V]. ``lora_a`` [A, rank, H], ``lora_b`` [A, V, rank];
    ``adapter_ids`` [B] int32 names each request's adapter (negative: none), ``row_offsets``
    [B+1] its rows (default: one row a request). Returns ``out`` (new by default, of
    ``out_dtype``, float32 by default). ``workspace``: see ``new_head_workspace(T, rank)``."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.project(x, weight, x_scale, weight_scale, lora_a, lora_b, adapter_scale, adapter_ids,
                                  row_offsets, out, out_dtype, workspace)
    return native.project(x, weight, x_scale, weight_scale, lora_a, lora_b, adapter_scale, adapter_ids, row_offsets,
                          out, out_dtype, workspace)


def project_cut(T: int, H: int, V: int, dtype: torch.dtype, adapters: int = 0, rank: int = 0, sms: int = 0):
    """How ``project`` cuts a product of these sizes on a device of ``sms`` SMs (0: the current
    one's): (CTAs of a tile, rows of ``x`` in a tile, whether blocks of rows with one adapter or
    two are multiplied on the tensor cores)."""
    codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3}
    got = (ctypes.c_uint32 * 3)()
    at = ctypes.addressof(got)
    rc = _pkg().load().lp_head_project_cut(T, H, V, codes.get(dtype, 99), adapters, rank, sms, at, at + 4, at + 8)
    if rc:
        _failed(rc, "lp_head_project_cut")
    return got[0], got[1], bool(got[2])


def process_logits(logits: torch.Tensor, row_offsets: Optional[torch.Tensor] = None,
                   history: Optional[torch.Tensor] = None, history_offsets: Optional[torch.Tensor] = None,
                   prompt_lens: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                   frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                   bias_tokens: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                   bias_offsets: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                   mask_index: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, *,
                   workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and grammar masks on ``logits`` [T, V]; returns
    ``out`` (float32, new by default; float32 logits may be processed in place).

    ``row_offsets`` [B+1] gives each request's rows (default: one row a request). Request
    b's ``history`` is ``history[history_offsets[b]:history_offsets[b+1]]``, its first
    ``prompt_lens[b]`` tokens the prompt. ``bias_*`` are ragged lists too, ids strictly
    ascending in each. ``mask`` [rows, words] int32 has a bit for each token, 1 = allowed;
    ``mask_index`` [T] names each row's mask, negative for none. ``workspace``: see
    ``new_head_workspace(requests=B, history=history.numel())``; errors found on the device set
    bits of its status (``read_status``)."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.process_logits(logits, row_offsets, history, history_offsets, prompt_lens, repetition,
                                         frequency, presence, bias_tokens, bias_values, bias_offsets, mask, mask_index,
                                         out, workspace)
    return native.process_logits(logits, row_offsets, history, history_offsets, prompt_lens, repetition, frequency,
                                 presence, bias_tokens, bias_values, bias_offsets, mask, mask_index, out, workspace)
