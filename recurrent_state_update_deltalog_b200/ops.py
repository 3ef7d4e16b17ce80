"""Operators that stand beside the recurrent layers (marshalling only).

``gated_scan`` (with its gradient, its prompt and its single-token form) is the
elementwise member of the recurrent family; ``block_norm`` the norms, gate and
residual around any block; ``paged_attention`` the decode step of attention layers
between recurrent ones.  Every computation runs in the CUDA library; shapes, dtypes and devices are checked here, so that a caller's mistake
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

import ctypes
import functools

import torch

from . import _native as N
from .deltalog import DTYPES

_F32, _I32 = torch.float32, torch.int32


def _placed(fn):
    """Run ``fn`` with its first tensor's device current, on ``stream`` if given."""
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        x = args[0] if args else kw.get(first)
        if not isinstance(x, torch.Tensor):
            raise ValueError(f"{first} must be a tensor")
        if stream is not None:
            if stream.device != x.device:
                raise ValueError(f"stream belongs to {stream.device}, {first} to {x.device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        if x.is_cuda and x.device.index != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return fn(*args, **kw)
        return fn(*args, **kw)
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
        names = {N.DL_DEVERR_SLOT_INDEX: "slot index past the pool", N.DL_DEVERR_SEQLEN: "invalid cu_seqlens range or length",
                 N.DL_DEVERR_PAGE: "page id outside the cache"}
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


# -- norms around a block ----------------------------------------------------------------------

def _norm_check(y, post_weight, gate, scale, residual, pre_weight, groups):
    dt = _check_first("y", y, range(1, 9))
    groups = int(groups)
    if groups > 1 and y.dim() >= 3 and y.shape[-2] == groups:      # [..., H, d]: the groups are a dimension
        D = groups * y.shape[-1]
    else:
        D = y.shape[-1]
    if groups < 1 or D < 1 or D % groups:
        raise ValueError(f"the last dimension ({D}) must be a positive multiple of groups ({groups})")
    for name, t in (("gate", gate), ("residual", residual)):
        if t is not None:
            _check(name, t, y.shape, y.dtype, y.device)
    for name, t, n in (("post_weight", post_weight, D // groups), ("scale", scale, D), ("pre_weight", pre_weight, D)):
        if t is not None:
            _check(name, t, (n,), _F32, y.device)
    return dt, y.numel() // D, D


def _block_norm(y, post_weight, gate, scale, residual, pre_weight, groups, eps, slot_idx, slots, out, normed):
    dt, rows, D = _norm_check(y, post_weight, gate, scale, residual, pre_weight, groups)
    if slot_idx is not None:
        _check_index("slot_idx", slot_idx, y.device, rows)
    if normed is not None and pre_weight is None:
        raise ValueError("normed_out goes with pre_weight")
    for name, t in (("out", out), ("normed_out", normed)):
        if t is not None:
            _check(name, t, y.shape, y.dtype, y.device)
    _check_cuda("y", y)
    out = torch.empty_like(y) if out is None else out
    if pre_weight is not None and normed is None:
        normed = torch.empty_like(y)
    N.call("dl_block_norm", _ptr(slot_idx), slots, rows, D, groups, dt, _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(scale),
           _ptr(residual), _ptr(pre_weight), eps, _ptr(out), _ptr(normed), _stream(y))
    return out, normed


@_placed
def block_norm_backward(y, dout, dnormed=None, post_weight=None, gate=None, scale=None, residual=None, pre_weight=None,
                        groups=1, eps=1e-6, need=(True,) * 6):
    """Gradients of :func:`block_norm` for dout and dnormed (each None: zeros), in the
    order y, post_weight, gate, scale, residual, pre_weight; None for absent parts and
    where ``need`` says False."""
    dt, rows, D = _norm_check(y, post_weight, gate, scale, residual, pre_weight, groups)
    if dnormed is not None and pre_weight is None:
        raise ValueError("dnormed goes with pre_weight")
    for name, t in (("dout", dout), ("dnormed", dnormed)):
        if t is not None:
            _check(name, t, y.shape, y.dtype, y.device)
    _check_cuda("y", y)
    parts = (y, post_weight, gate, scale, residual, pre_weight)
    grads = [torch.empty_like(t) if t is not None and k else None for t, k in zip(parts, need)]
    dy, dpost, dgate, dscale, dres, dpre = grads
    work = None
    if dpost is not None or dscale is not None or dpre is not None:
        nbytes = ctypes.c_size_t()
        N.call("dl_block_norm_workspace", rows, D, groups, ctypes.byref(nbytes))
        work = torch.empty(max(nbytes.value, 1), dtype=torch.uint8, device=y.device)
    N.call("dl_block_norm_backward", rows, D, groups, dt, _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(scale), _ptr(residual),
           _ptr(pre_weight), eps, _ptr(dout), _ptr(dnormed), _ptr(dy), _ptr(dgate), _ptr(dres), _ptr(dpost), _ptr(dscale),
           _ptr(dpre), _ptr(work), _stream(y))
    return tuple(grads)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, post_weight, gate, scale, residual, pre_weight, groups, eps):
        out, normed = _block_norm(y, post_weight, gate, scale, residual, pre_weight, groups, eps, None, 0, None, None)
        ctx.save_for_backward(y, post_weight, gate, scale, residual, pre_weight)
        ctx.groups, ctx.eps = groups, eps
        ctx.set_materialize_grads(False)
        return out if normed is None else (out, normed)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dnormed=None):
        y, post_weight, gate, scale, residual, pre_weight = ctx.saved_tensors
        grads = block_norm_backward(y, None if dout is None else dout.contiguous(),
                                    None if dnormed is None else dnormed.contiguous(), post_weight, gate, scale,
                                    residual, pre_weight, ctx.groups, ctx.eps, ctx.needs_input_grad[:6])
        return (*grads, None, None)


@_placed
def block_norm(y, post_weight=None, gate=None, scale=None, residual=None, pre_weight=None, groups=1, eps=1e-6,
               slot_idx=None, slots=None, out=None, normed_out=None):
    """Norms after and before a block, with its gate, residual scale and residual.

    u = RMSNorm(y) * post_weight (over ``groups`` groups of the last dimension), times
    silu(gate), times scale; out = residual + u; normed = RMSNorm(out) * pre_weight.
    Every part but y may be None.  y, gate, residual are bf16 or fp32 [..., D]; weights
    fp32: post_weight [D / groups], scale and pre_weight [D] (groups = 1 only).  With
    ``groups = H`` y may also be [..., H, d].  Returns out, or (out, normed) with a
    pre_weight; differentiable in every part.

    Serving (no gradients): ``out`` and ``normed_out`` may be y, gate or residual (in
    place); with ``slot_idx`` (int32 [rows]) rows of negative, held or, given ``slots``,
    too large slots are not written."""
    parts = (y, post_weight, gate, scale, residual, pre_weight)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in parts):
        if slot_idx is not None or out is not None or normed_out is not None:
            raise ValueError("slot_idx, out and normed_out are for calls without gradients")
        return _BlockNorm.apply(*parts, int(groups), float(eps))
    out, normed = _block_norm(*parts, int(groups), float(eps), slot_idx, 0x7fffffff if slots is None else int(slots), out,
                              normed_out)
    return out if normed is None else (out, normed)


# -- paged key-value cache -----------------------------------------------------------------------

def _cache_check(x, k_pages, v_pages, block_table, heads):
    """(num_pages, Hkv, page_size, d, slots, max_pages) of a cache for x [rows, heads, d]."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page, d = k_pages.shape
    _check("k_pages", k_pages, k_pages.shape, x.dtype, x.device)
    _check("v_pages", v_pages, k_pages.shape, x.dtype, x.device)
    if x.shape[2] != d or Hkv < 1 or x.shape[1] % Hkv or (heads and x.shape[1] != Hkv):
        raise ValueError(f"heads {tuple(x.shape[1:])} do not fit a cache of {Hkv} heads of {d}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [slots, max_pages]")
    _check("block_table", block_table, block_table.shape, _I32, x.device)
    return num_pages, Hkv, page, d, block_table.shape[0], block_table.shape[1]


@functools.lru_cache(maxsize=4096)
def _paged_workspace(rows, Hq, Hkv, d, dt, page, max_pages, window):
    nbytes = ctypes.c_size_t()
    N.call("dl_paged_attention_workspace", rows, Hq, Hkv, d, dt, page, max_pages, window, ctypes.byref(nbytes))
    return nbytes.value


@_placed
def paged_attention(q, k_pages, v_pages, block_table, lens, k=None, v=None, slot_idx=None, window=0, scale=None, out=None,
                    err=None):
    """Attention of one new token a row over a paged cache; returns o like q.

    q [rows, Hq, d] bf16 or fp32 (d 64 or 128); k_pages, v_pages [num_pages, Hkv,
    page_size, d] of the same type; block_table int32 [slots, max_pages]; lens int32
    [slots], the new token included; row r runs on slot ``slot_idx[r]`` (default r;
    negative or held: skipped, its output not written).  With k, v [rows, Hkv, d] the
    new token is stored at position lens - 1 first.  ``window`` > 0 keeps the last
    ``window`` positions.  scale defaults to d ** -0.5.  A slot of length 0 gives zeros."""
    dt = _check_first("q", q, (3,))
    num_pages, Hkv, page, d, slots, max_pages = _cache_check(q, k_pages, v_pages, block_table, False)
    rows = q.shape[0]
    _check_index("lens", lens, q.device, slots)
    _check_slots(slot_idx, rows, slots, q.device)
    if not 0 <= int(window) < 1 << 31:
        raise ValueError("window must be 0 (none) or a positive 32-bit number")
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    if k is not None:
        _check("k", k, (rows, Hkv, d), q.dtype, q.device)
        _check("v", v, (rows, Hkv, d), q.dtype, q.device)
    if out is not None:
        _check("out", out, q.shape, q.dtype, q.device)
    _check_err(err, q.device)
    _check_cuda("q", q)
    out = torch.empty_like(q) if out is None else out
    nbytes = _paged_workspace(rows, q.shape[1], Hkv, d, dt, page, max_pages, int(window))
    work = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    N.call("dl_paged_attention", _ptr(slot_idx), slots, rows, q.shape[1], Hkv, d, dt, page, num_pages, max_pages,
           _ptr(block_table), _ptr(lens), int(window), d ** -0.5 if scale is None else float(scale), _ptr(q), _ptr(k), _ptr(v),
           _ptr(k_pages), _ptr(v_pages), _ptr(out), _ptr(work), _ptr(err), _stream(q))
    return out


@_placed
def paged_write(k, v, k_pages, v_pages, block_table, cu_seqlens, starts=None, slot_idx=None, err=None):
    """Copy packed prompts k, v [total, Hkv, d] into a paged cache: row r's tokens
    [cu_seqlens[r], cu_seqlens[r + 1]) to positions starts[slot] + 0, 1, ... of its slot
    (``starts`` int32 [slots], default 0; slots as in :func:`paged_attention`)."""
    dt = _check_first("k", k, (3,))
    _check("v", v, k.shape, k.dtype, k.device)
    num_pages, Hkv, page, d, slots, max_pages = _cache_check(k, k_pages, v_pages, block_table, True)
    _check_index("cu_seqlens", cu_seqlens, k.device)
    rows = cu_seqlens.numel() - 1
    if rows < 0:
        raise ValueError("cu_seqlens must hold rows + 1 offsets")
    if starts is not None:
        _check_index("starts", starts, k.device, slots)
    _check_slots(slot_idx, rows, slots, k.device)
    _check_err(err, k.device)
    _check_cuda("k", k)
    N.call("dl_paged_write", _ptr(slot_idx), slots, rows, _ptr(cu_seqlens), k.shape[0], Hkv, d, dt, page, num_pages, max_pages,
           _ptr(block_table), _ptr(starts), _ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages), _ptr(err), _stream(k))
