"""Operators that stand beside the recurrent layers (marshalling only).

``gated_scan`` (with its gradient, its prompt and its single-token form) is the
elementwise member of the recurrent family.  Every computation runs in the CUDA
library; shapes, dtypes and devices are checked here, so that a caller's mistake
becomes a Python exception before a pointer crosses the C ABI.

Conventions.  Tensors are contiguous CUDA tensors of one device, which need not
be the current one.  Work is queued on ``stream``, by default the current stream
of that device; outputs and temporaries are allocated for that stream.  ``err``
is an optional int32 [1] device tensor of zeros in which kernels raise the
DL_DEVERR_* bits (:func:`check_errors` reads and clears it).

Capture into a CUDA graph: call the explicit ``*_forward`` / ``*_backward`` pairs
rather than the autograd forms, whose backward pass the autograd engine may run
on another stream than the captured one.
"""
from __future__ import annotations

import functools

import torch

from . import _native as N
from .deltalog import DTYPES

_F32, _I32 = torch.float32, torch.int32


def _placed(fn):
    """Run ``fn`` with its first tensor's device current, on ``stream`` if given."""
    @functools.wraps(fn)
    def call(x, *args, stream=None, **kw):
        if stream is not None:
            if stream.device != x.device:
                raise ValueError(f"stream belongs to {stream.device}, the tensors to {x.device}")
            with torch.cuda.stream(stream):
                return fn(x, *args, **kw)
        if x.is_cuda and x.device.index != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return fn(x, *args, **kw)
        return fn(x, *args, **kw)
    return call


def _check(name, t, shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")


def _check_first(name, t, dims):
    """The tensor that sets the type and the device of a call; its DL_* type."""
    if not isinstance(t, torch.Tensor) or t.dim() not in dims:
        raise ValueError(f"{name} must be a tensor of {' or '.join(map(str, dims))} dimensions")
    if t.dtype not in DTYPES:
        raise ValueError(f"{name}: expected torch.bfloat16 or torch.float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return DTYPES[t.dtype]


def _check_cuda(name, t):
    """Last of the checks: the device itself (all other tensors are on t's)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")


def _check_index(name, t, device, n=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be 1-D" + (f" with {n} entries" if n is not None else ""))
    _check(name, t, t.shape, _I32, device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def check_errors(err):
    """Raise DeltaLogError if a kernel has raised bits in ``err``; clears them.
    Waits for the work queued on the current stream of its device."""
    _check("err", err, (1,), _I32, err.device)
    bits = int(err.item())
    if bits:
        err.zero_()
        names = {N.DL_DEVERR_SLOT_INDEX: "slot index past the pool", N.DL_DEVERR_SEQLEN: "invalid cu_seqlens range"}
        raise N.DeltaLogError("check_errors", -5, ", ".join(v for k, v in names.items() if bits & k) or hex(bits))


def _check_err(err, device):
    if err is not None:
        _check("err", err, (1,), _I32, device)


# -- gated linear recurrence -----------------------------------------------------------------

def _scan_sizes(x, cu_seqlens):
    """(rows, tokens, channels) of x [rows, T, C], or [total, C] with cu_seqlens."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x must be [rows, T, C], or [total, C] with cu_seqlens")
        return x.shape[0], x.shape[0] * x.shape[1], x.shape[2]
    if x.dim() != 2:
        raise ValueError("x must be [total, C] with cu_seqlens")
    _check_index("cu_seqlens", cu_seqlens, x.device)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold rows + 1 offsets")
    return cu_seqlens.numel() - 1, x.shape[0], x.shape[1]


@_placed
def gated_scan_forward(x, log_decay, h0=None, cu_seqlens=None, checkpoints=False, err=None):
    """:func:`gated_scan` without autograd: (h, h_last, ckpt), ckpt (None unless
    ``checkpoints``) being what :func:`gated_scan_backward` needs."""
    dt = _check_first("x", x, (2, 3))
    rows, total, C = _scan_sizes(x, cu_seqlens)
    _check("log_decay", log_decay, x.shape, _F32, x.device)
    if h0 is not None:
        _check("h0", h0, (rows, C), _F32, x.device)
    _check_err(err, x.device)
    _check_cuda("x", x)
    h = torch.empty_like(x)
    h_last = torch.empty((rows, C), dtype=_F32, device=x.device)
    ckpt = None
    if checkpoints:
        ckpt = torch.empty((total // N.DL_SCAN_CHUNK + rows, C), dtype=_F32, device=x.device)
    N.call("dl_scan", None, rows, rows, _ptr(cu_seqlens), total, C, dt, _ptr(x), _ptr(log_decay), _ptr(h0),
           _ptr(h_last), _ptr(h), _ptr(ckpt), _ptr(err), _stream(x))
    return h, h_last, ckpt


@_placed
def gated_scan_backward(x, log_decay, ckpt, dh, dh_last=None, cu_seqlens=None, err=None):
    """Gradients (dx, dlog_decay, dh0) of :func:`gated_scan_forward` for the
    gradients dh of h and dh_last of h_last (None: zeros)."""
    dt = _check_first("x", x, (2, 3))
    rows, total, C = _scan_sizes(x, cu_seqlens)
    _check("log_decay", log_decay, x.shape, _F32, x.device)
    _check("ckpt", ckpt, (total // N.DL_SCAN_CHUNK + rows, C), _F32, x.device)
    _check("dh", dh, x.shape, x.dtype, x.device)
    if dh_last is not None:
        _check("dh_last", dh_last, (rows, C), _F32, x.device)
    _check_err(err, x.device)
    _check_cuda("x", x)
    dx, dld = torch.empty_like(x), torch.empty_like(log_decay)
    dh0 = torch.empty((rows, C), dtype=_F32, device=x.device)
    N.call("dl_scan_backward", rows, _ptr(cu_seqlens), total, C, dt, _ptr(x), _ptr(log_decay), _ptr(ckpt), _ptr(dh),
           _ptr(dh_last), _ptr(dx), _ptr(dld), _ptr(dh0), _ptr(err), _stream(x))
    return dx, dld, dh0


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, log_decay, h0, cu_seqlens, err):
        h, h_last, ckpt = gated_scan_forward(x, log_decay, h0, cu_seqlens, checkpoints=True, err=err)
        ctx.save_for_backward(x, log_decay, ckpt, cu_seqlens)
        ctx.err = err
        ctx.set_materialize_grads(False)
        return h, h_last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dh_last):
        x, log_decay, ckpt, cu_seqlens = ctx.saved_tensors
        dh = torch.zeros_like(x) if dh is None else dh.contiguous()
        dh_last = None if dh_last is None else dh_last.contiguous()
        dx, dld, dh0 = gated_scan_backward(x, log_decay, ckpt, dh, dh_last, cu_seqlens, err=ctx.err)
        return dx, dld, dh0 if ctx.needs_input_grad[2] else None, None, None


@_placed
def gated_scan(x, log_decay, h0=None, cu_seqlens=None, err=None):
    """Gated linear recurrence per channel: h_t = exp(log_decay_t) h_{t-1} + x_t.

    x [rows, T, C] bf16 or fp32 and log_decay fp32 of the same shape (<= 0); or
    packed [total, C] with ``cu_seqlens`` (int32 [rows + 1], device).  h0 fp32
    [rows, C] (None: zeros).  Returns (h, h_last): h like x, h_last fp32
    [rows, C], the states after the last tokens.  Differentiable in x,
    log_decay and h0 (first derivatives)."""
    if torch.is_grad_enabled() and (x.requires_grad or log_decay.requires_grad or (h0 is not None and h0.requires_grad)):
        return _GatedScan.apply(x, log_decay, h0, cu_seqlens, err)
    return gated_scan_forward(x, log_decay, h0, cu_seqlens, err=err)[:2]


def _check_pool(state, new_state, C, device):
    if not isinstance(state, torch.Tensor) or state.dim() != 2 or state.shape[1] != C:
        raise ValueError(f"state must be [slots, {C}]")
    _check("state", state, state.shape, _F32, device)
    if new_state is not None:
        _check("new_state", new_state, state.shape, _F32, device)


def _check_slots(slot_idx, rows, slots, device):
    if slot_idx is not None:
        _check_index("slot_idx", slot_idx, device, rows)
    elif rows > slots:
        raise ValueError(f"{rows} rows without slot_idx need as many slots, got {slots}")


@_placed
def gated_scan_prefill(x, log_decay, state, cu_seqlens, slot_idx=None, zero_state=False, new_state=None, out=None,
                       err=None):
    """:func:`gated_scan` over packed prompts on a pool of states.

    x, log_decay [total, C], ``cu_seqlens`` int32 [rows + 1]; row r starts from
    ``state[slot_idx[r]]`` (fp32 [slots, C]; zeros with ``zero_state``) and leaves
    its last state there, or in ``new_state`` if given.  Rows with a negative or
    held slot (``slot | DeltaLog.HOLD``) are skipped, their outputs not written.
    Returns h [total, C]."""
    dt = _check_first("x", x, (2,))
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    rows, total, C = _scan_sizes(x, cu_seqlens)
    _check("log_decay", log_decay, x.shape, _F32, x.device)
    _check_pool(state, new_state, C, x.device)
    _check_slots(slot_idx, rows, state.shape[0], x.device)
    if out is not None:
        _check("out", out, x.shape, x.dtype, x.device)
    _check_err(err, x.device)
    _check_cuda("x", x)
    h = torch.empty_like(x) if out is None else out
    N.call("dl_scan", _ptr(slot_idx), state.shape[0], rows, _ptr(cu_seqlens), total, C, dt, _ptr(x), _ptr(log_decay),
           None if zero_state else _ptr(state), _ptr(state if new_state is None else new_state), _ptr(h), None,
           _ptr(err), _stream(x))
    return h


@_placed
def gated_scan_step(x, log_decay, state, slot_idx=None, new_state=None, out=None, err=None):
    """One token of :func:`gated_scan` for rows of a pool of states: x, log_decay
    [rows, C]; row r runs on ``state[slot_idx[r]]`` (fp32 [slots, C]), updated in
    place, or into ``new_state`` if given.  Rows with a negative or held slot are
    skipped, their outputs not written.  Returns h [rows, C]."""
    dt = _check_first("x", x, (2,))
    rows, C = x.shape
    _check("log_decay", log_decay, x.shape, _F32, x.device)
    _check_pool(state, new_state, C, x.device)
    _check_slots(slot_idx, rows, state.shape[0], x.device)
    if out is not None:
        _check("out", out, x.shape, x.dtype, x.device)
    _check_err(err, x.device)
    _check_cuda("x", x)
    h = torch.empty_like(x) if out is None else out
    N.call("dl_scan_step", _ptr(slot_idx), state.shape[0], rows, C, dt, _ptr(x), _ptr(log_decay), _ptr(state),
           _ptr(state if new_state is None else new_state), _ptr(h), _ptr(err), _stream(x))
    return h
