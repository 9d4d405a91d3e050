"""The operators of a served model's head around the ragged log-probability path: final
norm, vocabulary projection with low-rank adapters or in microscaled 4-bit floating point,
processing of logits, draw of the next token.

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
           "process_logits", "fp4_scale_bytes", "tile_fp4_scales", "quantize_fp4", "dequantize_fp4", "project_fp4",
           "sample"]

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
    lib.lp_head_sample_workspace_size.argtypes = [u32, u32]
    lib.lp_head_sample_workspace_size.restype = sz
    lib.lp_head_sample.argtypes = [vp, u32, u32, u32, u64, vp, vp, u32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.lp_head_sample.restype = ctypes.c_int
    lib.lp_head_fp4_scale_bytes.argtypes = [u32, u32, u32]
    lib.lp_head_fp4_scale_bytes.restype = sz
    lib.lp_head_quantize4.argtypes = [vp, u32, u32, u32, u64, u32, vp, u64, vp, vp, vp]
    lib.lp_head_quantize4.restype = ctypes.c_int
    lib.lp_head_dequantize4.argtypes = [vp, u64, vp, vp, u32, u32, u32, vp, u32, vp, u32, u64, vp, sz, vp]
    lib.lp_head_dequantize4.restype = ctypes.c_int
    lib.lp_head_project4.argtypes = [vp, u64, vp, vp, u32, u32, u32, vp, u64, vp, vp, u32, vp, u32, u64, vp, sz, vp]
    lib.lp_head_project4.restype = ctypes.c_int
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


def head_workspace_size(T: int = 0, rank: int = 0, requests: int = 0, history: int = 0, draws: int = 0,
                        vocab: int = 0) -> int:
    """Bytes of scratch that serve every call of up to these sizes: ``project`` with adapters of
    that rank over T rows, ``process_logits`` of that many requests with that many history
    tokens in all, ``sample`` of that many rows of logits of that vocabulary (0: only the status
    word)."""
    lib = _pkg().load()
    n = int(lib.lp_head_workspace_size(T, rank))
    if n == 0:
        raise ValueError(f"rank {rank} exceeds {LP_MAX_RANK}")
    return max(n, int(lib.lp_head_process_workspace_size(requests, history)),
               int(lib.lp_head_sample_workspace_size(draws, vocab)))


def new_head_workspace(T: int = 0, rank: int = 0, requests: int = 0, history: int = 0, device=None, draws: int = 0,
                       vocab: int = 0) -> torch.Tensor:
    """A zeroed workspace (uint8) of ``head_workspace_size``. Its status word collects the
    bits of every call that is given it, until ``clear_status``; ``read_status`` reads it."""
    return torch.zeros(head_workspace_size(T, rank, requests, history, draws, vocab), dtype=torch.uint8,
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


def fp4_scale_bytes(rows: int, H: int, block: int = 16) -> int:
    """Bytes of the block scales of ``rows`` 4-bit rows of ``H`` elements, in their tiles."""
    if block not in (16, 32):
        raise ValueError(f"block must be 16 or 32, is {block}")
    return int(_pkg().load().lp_head_fp4_scale_bytes(rows, H, block))


def tile_fp4_scales(scales: torch.Tensor) -> torch.Tensor:
    """Block scales [rows, blocks] (uint8, float8_e4m3fn or float8_e8m0fnu, on any device) laid out in
    tiles of 128 rows by 4 blocks, as the functions below take them; for weights that were
    quantised elsewhere. Done once: a copy of torch's."""
    if scales.dim() != 2 or scales.element_size() != 1:
        raise ValueError("scales must be [rows, blocks] of 8-bit elements")
    rows, n = scales.shape
    rb, cb = -(-rows // 128), -(-n // 4)
    full = torch.zeros(rb * 128, cb * 4, dtype=torch.uint8, device=scales.device)
    full[:rows, :n] = scales.view(torch.uint8)
    return full.view(rb, 4, 32, cb, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def quantize_fp4(x: torch.Tensor, block: int = 16, out: Optional[torch.Tensor] = None,
                 out_scales: Optional[torch.Tensor] = None, out_row_scale: Optional[torch.Tensor] = None, stream=None):
    """Rows of ``x`` [T, H] (float32, bfloat16, float16; H a multiple of 32) in 4 bits, with a scale
    for every block of 16 elements (float8_e4m3fn, and a power of two a row) or of 32 (float8_e8m0fnu).

    Returns ``(codes, scales, row_scale)``: uint8 [T, H / 2], two codes to a byte, the first in the
    low half; the scales' bytes in tiles (``fp4_scale_bytes`` of them); float32 [T], or None for
    blocks of 32."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.quantize_fp4(x, block, out, out_scales, out_row_scale)
    return native.quantize_fp4(x, block, out, out_scales, out_row_scale)


def dequantize_fp4(codes: torch.Tensor, scales: torch.Tensor, row_scale: Optional[torch.Tensor] = None,
                   block: int = 16, rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Values of 4-bit rows (as ``quantize_fp4`` returns them): of all, or of those that ``rows`` [n]
    names, such as the tokens to look up in a 4-bit embedding. ``out`` is float32, bfloat16 (by
    default) or float16. With ``rows`` a workspace is needed: a row past the last sets
    LP_ERR_OFFSETS in its status and gives NaN."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.dequantize_fp4(codes, scales, row_scale, block, rows, out, out_dtype, workspace)
    return native.dequantize_fp4(codes, scales, row_scale, block, rows, out, out_dtype, workspace)


def project_fp4(x: torch.Tensor, x_scales: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                block: int = 16, x_row_scale: Optional[torch.Tensor] = None,
                weight_row_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, *, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Logits [T, V] of 4-bit hidden states ``x`` [T, H / 2] and a 4-bit ``weight`` [V, H / 2], both with
    scales as ``quantize_fp4`` returns them (row scales: None means 1). Returns ``out`` (new by
    default, of ``out_dtype``, float32 by default). ``workspace``: see ``new_head_workspace``."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.project_fp4(x, x_scales, weight, weight_scales, block, x_row_scale, weight_row_scale, out,
                                      out_dtype, workspace)
    return native.project_fp4(x, x_scales, weight, weight_scales, block, x_row_scale, weight_row_scale, out, out_dtype,
                              workspace)


def sample(logits: torch.Tensor, uniform: torch.Tensor, row_offsets: Optional[torch.Tensor] = None,
           temperature: Optional[torch.Tensor] = None, top_k: Optional[torch.Tensor] = None,
           top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, out_logprob: Optional[torch.Tensor] = None, *, workspace: torch.Tensor,
           stream=None) -> torch.Tensor:
    """A token for every row of ``logits`` [T, V] (float32, bfloat16, float16), drawn with the random
    number ``uniform`` [T] (float32, in [0, 1)) from what the row's request leaves of the
    distribution; returns ``out`` (int32 [T], new by default).

    ``temperature``, ``top_p``, ``min_p`` (float32) and ``top_k`` (int32) are [B], ``row_offsets`` [B+1]
    gives each request's rows (default: one row a request). Temperature 0 takes the best token;
    ``top_k`` 0, ``top_p`` 1 and ``min_p`` 0 (the defaults) leave all. The order: the best ``top_k``
    tokens; of these the fewest that hold ``top_p`` of their probability; of these those with at
    least ``min_p`` of the best one's. ``out_logprob`` (float32 [T]) receives the token's logprob in
    what was left. A row without a distribution (nothing but -inf, or a NaN or +inf) gives
    -1 and NaN and sets LP_ERR_LOGITS; ``read_status`` reads the workspace's bits. ``workspace``: see
    ``new_head_workspace(draws=T, vocab=V)``."""
    native = _native or _load()
    if stream is not None:
        with torch.cuda.stream(stream):
            return native.sample(logits, uniform, row_offsets, temperature, top_k, top_p, min_p, out, out_logprob, workspace)
    return native.sample(logits, uniform, row_offsets, temperature, top_k, top_p, min_p, out, out_logprob, workspace)
