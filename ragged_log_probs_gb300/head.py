"""The operators of a served model's head around the ragged log-probability path: final
norm, vocabulary projection with low-rank adapters, processing of logits.

Argument marshalling only, like the package's other calls: every operator runs in the
CUDA kernels of ``liblp_ragged.so`` behind the C ABI of ``include/lp_head.h``, whose
comments define the operators. Matrices may have any row stride, with their last
dimension contiguous.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

__all__ = ["head_workspace_size", "new_head_workspace", "clear_status", "rms_norm", "project", "process_logits"]

LP_MAX_HIDDEN = 32768
LP_MAX_RANK = 64
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3}
_INTS = (torch.int32, torch.uint32)


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
    lib.lp_head_process.argtypes = [vp, u32, u32, u32, u64, vp, u32, vp, vp, u32, vp, vp, vp, vp, vp, vp, vp, u32,
                                    vp, u64, u32, vp, vp, u64, vp, sz, vp]
    lib.lp_head_process.restype = ctypes.c_int
    lib.lp_head_process_workspace_size.argtypes = [u32, u32]
    lib.lp_head_process_workspace_size.restype = sz


def _pkg():
    import ragged_log_probs_gb300 as lp
    return lp


# The calls below are made once a token, and a launch takes under 2 us: the checks are kept to
# one look at each tensor, and what is wrong is worked out only once something is.
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_F32 = (torch.float32,)


def _stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream


def _check_device(t: torch.Tensor, name: str, device: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")


def _refuse_matrix(t, name: str, device: int, shape, dtype) -> None:
    _check_device(t, name, device)
    if t.dim() != 2 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, is {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, is {t.dtype}")
    raise ValueError(f"{name}'s last dimension must be contiguous")


def _matrix(t: torch.Tensor, name: str, device: int, shape, dtype: torch.dtype):
    """Pointer and row stride of a 2-D tensor whose last dimension is contiguous."""
    try:
        if t.get_device() == device and t.shape == shape and t.dtype == dtype:
            s0, s1 = t.stride()
            if s1 == 1 or shape[1] == 1:
                return t.data_ptr(), s0 if shape[0] > 1 else shape[1]
    except (AttributeError, ValueError):
        pass
    _refuse_matrix(t, name, device, shape, dtype)


def _shape2(t: torch.Tensor, name: str, device: int):
    """Shape of a CUDA tensor with two dimensions."""
    try:
        r, c = t.shape
        return r, c
    except (AttributeError, ValueError):
        _check_device(t, name, device)
        raise ValueError(f"{name} must be 2-D, has {t.dim()} dimensions") from None


def _vector(t: Optional[torch.Tensor], name: str, device: int, n: int, dtypes) -> Optional[int]:
    """Pointer of a contiguous 1-D tensor of n elements (None stays None)."""
    if t is None:
        return None
    try:
        if t.get_device() == device and t.shape == (n,) and t.dtype in dtypes and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check_device(t, name, device)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, is {t.dtype}")
    raise ValueError(f"{name} must be contiguous 1-D with {n} elements")


def _scratch(workspace: Optional[torch.Tensor], device: int):
    if workspace is None:
        return None, 0
    try:
        if workspace.get_device() == device and workspace.is_contiguous():
            return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    except AttributeError:
        pass
    _check_device(workspace, "workspace", device)
    raise TypeError("workspace must be a contiguous CUDA tensor (see new_head_workspace)")


def _new(shape, dtype: torch.dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An output, allocated on the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _output(out, shape, dtype, like, stream):
    if out is None:
        return _new(shape, dtype, like, stream)
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, is {out.dtype}")
    return out


def _failed(rc: int, what: str) -> None:
    raise _pkg().LpError(rc, what)


def head_workspace_size(T: int = 0, rank: int = 0, requests: int = 0, history: int = 0) -> int:
    """Bytes of scratch that serve every call of these sizes: ``project`` with adapters of
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
    dev = _device()
    rc = _pkg().load().lp_head_clear_status(_scratch(workspace, dev)[0], _stream(stream, dev))
    if rc:
        _failed(rc, "lp_head_clear_status")


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
    dev = _device()
    T, H = _shape2(x, "x", dev)
    dt = x.dtype
    xp, xs = _matrix(x, "x", dev, (T, H), dt)
    n = T
    rp = ip = kp = sp = None
    rs = ks = 0
    if residual is not None:
        rp, rs = _matrix(residual, "residual", dev, (T, H), dt)
    if rows is not None:
        n = rows.numel()
        ip = _vector(rows, "rows", dev, n, _INTS)
    if out is None or out_dtype is not None:
        out = _output(out, (n, H), dt if out_dtype is None else out_dtype, x, stream)
    odt = out.dtype
    op, os_ = _matrix(out, "out", dev, (n, H), odt)
    if odt == torch.float8_e4m3fn and out_scale is None:
        out_scale = _new((n,), torch.float32, x, stream)
    if out_scale is not None:
        sp = _vector(out_scale, "out_scale", dev, n, _F32)
    if residual_out is not None:
        kp, ks = _matrix(residual_out, "residual_out", dev, (n, H), dt)
    wp = _vector(weight, "weight", dev, H, (dt, torch.float32))
    ws, wn = _scratch(workspace, dev)
    rc = _pkg().load().lp_head_norm(xp, rp, wp, _DTYPES.get(dt, 99), _DTYPES[weight.dtype], T, H, xs, rs, ip, n, eps,
                                    op, _DTYPES.get(odt, 99), os_, sp, kp, ks, ws, wn, _stream(stream, dev))
    if rc:
        _failed(rc, "lp_head_norm")
    return (out, out_scale) if odt == torch.float8_e4m3fn else out


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
    dev = _device()
    T, H = _shape2(x, "x", dev)
    dt = x.dtype
    xp, xs = _matrix(x, "x", dev, (T, H), dt)
    V = _shape2(weight, "weight", dev)[0]
    wp, ws = _matrix(weight, "weight", dev, (V, H), dt)
    ap = bp = ip = rp = sp = None
    A = rank = B = 0
    at = dt
    if lora_a is not None:
        if lora_b is None or adapter_ids is None:
            raise ValueError("lora_a needs lora_b and adapter_ids")
        if lora_a.dim() != 3:
            raise ValueError(f"lora_a must be 3-D, has {lora_a.dim()} dimensions")
        A, rank = lora_a.shape[:2]
        B = T if row_offsets is None else row_offsets.numel() - 1
        at = lora_a.dtype
        for t, name, shape in ((lora_a, "lora_a", (A, rank, H)), (lora_b, "lora_b", (A, V, rank))):
            _check_device(t, name, dev)
            if t.shape != shape or not t.is_contiguous() or t.dtype != at:
                raise ValueError(f"{name} must be contiguous {shape} of {at}, is {tuple(t.shape)} of {t.dtype}")
        ap, bp = lora_a.data_ptr(), lora_b.data_ptr()
        ip = _vector(adapter_ids, "adapter_ids", dev, B, (torch.int32,))
        rp = _vector(row_offsets, "row_offsets", dev, B + 1, _INTS)
        sp = _vector(adapter_scale, "adapter_scale", dev, A, _F32)
    elif lora_b is not None or adapter_ids is not None or adapter_scale is not None:
        raise ValueError("lora_b, adapter_ids and adapter_scale need lora_a")
    if out is None or out_dtype is not None:
        out = _output(out, (T, V), torch.float32 if out_dtype is None else out_dtype, x, stream)
    odt = out.dtype
    op, os_ = _matrix(out, "out", dev, (T, V), odt)
    kp, kn = _scratch(workspace, dev)
    rc = _pkg().load().lp_head_project(
        xp, _DTYPES.get(dt, 99), T, H, xs, _vector(x_scale, "x_scale", dev, T, _F32), wp, V, ws,
        _vector(weight_scale, "weight_scale", dev, V, _F32), ap, bp, _DTYPES.get(at, 99), A, rank, sp, ip, rp, B, op,
        _DTYPES.get(odt, 99), os_, kp, kn, _stream(stream, dev))
    if rc:
        _failed(rc, "lp_head_project")
    return out


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
    dev = _device()
    T, V = _shape2(logits, "logits", dev)
    dt = logits.dtype
    xp, xs = _matrix(logits, "logits", dev, (T, V), dt)
    B = T if row_offsets is None else row_offsets.numel() - 1
    hp = ho = bt = bv = bo = mp = mi = None
    hn = nb = ms = mr = 0
    if history is not None or history_offsets is not None:
        if history is None or history_offsets is None:
            raise ValueError("history and history_offsets come together")
        hn = history.numel()
        hp = _vector(history, "history", dev, hn, _INTS)
        ho = _vector(history_offsets, "history_offsets", dev, B + 1, _INTS)
    if bias_tokens is not None or bias_values is not None or bias_offsets is not None:
        if bias_tokens is None or bias_values is None or bias_offsets is None:
            raise ValueError("bias_tokens, bias_values and bias_offsets come together")
        nb = bias_tokens.numel()
        bt = _vector(bias_tokens, "bias_tokens", dev, nb, _INTS)
        bv = _vector(bias_values, "bias_values", dev, nb, _F32)
        bo = _vector(bias_offsets, "bias_offsets", dev, B + 1, _INTS)
    if mask is not None:
        mr, words = _shape2(mask, "mask", dev)
        if mask.dtype not in _INTS or words < (V + 31) // 32:
            raise ValueError(f"mask must be int32 [rows, {(V + 31) // 32} or more]")
        mp, ms = _matrix(mask, "mask", dev, (mr, words), mask.dtype)
        mi = _vector(mask_index, "mask_index", dev, T, _INTS)
    elif mask_index is not None:
        raise ValueError("mask_index needs a mask")
    if out is None:
        out = _new((T, V), torch.float32, logits, stream)
    op, os_ = _matrix(out, "out", dev, (T, V), torch.float32)
    sp, sn = _scratch(workspace, dev)
    rc = _pkg().load().lp_head_process(
        xp, _DTYPES.get(dt, 99), T, V, xs, _vector(row_offsets, "row_offsets", dev, B + 1, _INTS), B, hp, ho, hn,
        _vector(prompt_lens, "prompt_lens", dev, B, _INTS), _vector(repetition, "repetition", dev, B, _F32),
        _vector(frequency, "frequency", dev, B, _F32), _vector(presence, "presence", dev, B, _F32), bt, bv, bo, nb,
        mp, ms, mr, mi, op, os_, sp, sn, _stream(stream, dev))
    if rc:
        _failed(rc, "lp_head_process")
    return out
