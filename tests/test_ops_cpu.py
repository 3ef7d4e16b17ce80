"""Refusals of the stateless operators: the C ABI rejects bad arguments before any CUDA call, the Python layer turns
wrong shapes, types, layouts and devices into ValueError.  No GPU is touched."""
import ctypes

import pytest
import torch

from recurrent_state_update_deltalog_b200 import _native as N
from recurrent_state_update_deltalog_b200.build import build

ARG, UNSUPPORTED = -1, -2
P, ODD = ctypes.c_void_p(64), ctypes.c_void_p(65)


@pytest.fixture(scope="module")
def lib():
    build()
    return N.load()


def scan_args(**over):
    a = dict(slot_idx=None, slots=2, rows=2, cu=None, total=8, C=4, dtype=1, x=P, d=P, h0=None, h_last=None, h=P,
             ckpt=None, err=None)
    a.update(over)
    return list(a.values()) + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), ARG), (dict(C=0), ARG), (dict(C=(1 << 24) + 1), ARG), (dict(rows=-1), ARG), (dict(total=-8), ARG),
    (dict(rows=65536, slots=65536, total=65536), UNSUPPORTED), (dict(rows=0, total=8), ARG), (dict(total=9), ARG),
    (dict(slots=1), ARG), (dict(slot_idx=P, slots=0), ARG), (dict(x=None), ARG), (dict(d=None), ARG), (dict(h=None), ARG),
    (dict(x=ODD), ARG), (dict(h=ODD), ARG), (dict(d=ODD), ARG), (dict(h0=ODD), ARG), (dict(ckpt=ODD), ARG),
    (dict(err=ODD), ARG), (dict(slot_idx=ODD), ARG), (dict(cu=ODD), ARG), (dict(cu=P, total=1 << 31), UNSUPPORTED),
])
def test_scan_refusals(lib, over, status):
    assert lib.dl_scan(*scan_args(**over)) == status
    assert lib.dl_last_error()


@pytest.mark.parametrize("over,status", [
    (dict(dtype=-1), ARG), (dict(C=0), ARG), (dict(total=7), ARG), (dict(ckpt=None), ARG), (dict(dh=None), ARG),
    (dict(dx=None), ARG), (dict(dld=None), ARG), (dict(dh=ODD), ARG), (dict(dx=ODD), ARG), (dict(dh0=ODD), ARG),
    (dict(dh_last=ODD), ARG),
])
def test_scan_backward_refusals(lib, over, status):
    a = dict(rows=2, cu=None, total=8, C=4, dtype=1, x=P, d=P, ckpt=P, dh=P, dh_last=None, dx=P, dld=P, dh0=None, err=None)
    a.update(over)
    assert lib.dl_scan_backward(*a.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=5), ARG), (dict(C=-4), ARG), (dict(slots=1), ARG), (dict(state=None), ARG), (dict(new=None), ARG),
    (dict(h=None), ARG), (dict(state=ODD), ARG), (dict(rows=65536, slots=1 << 17), UNSUPPORTED),
])
def test_scan_step_refusals(lib, over, status):
    a = dict(slot_idx=None, slots=2, rows=2, C=4, dtype=0, x=P, d=P, state=P, new=P, h=P, err=None)
    a.update(over)
    assert lib.dl_scan_step(*a.values(), None) == status


def test_scan_without_rows_is_a_no_op(lib):
    assert lib.dl_scan(*scan_args(rows=0, total=0, x=None, d=None, h=None)) == 0
    assert lib.dl_scan_backward(0, None, 0, 4, 1, *[None] * 10) == 0
    assert lib.dl_scan_step(None, 1, 0, 4, 1, *[None] * 7) == 0


def test_scan_python_refusals(lib):
    from recurrent_state_update_deltalog_b200 import (gated_scan, gated_scan_backward, gated_scan_forward,
                                                      gated_scan_prefill, gated_scan_step)
    x, d = torch.zeros(2, 3, 4), torch.zeros(2, 3, 4)
    x2, d2, pool = x[0].contiguous(), d[0].contiguous(), torch.zeros(5, 4)
    cu = torch.zeros(3, dtype=torch.int32)
    for bad, match in [
        (lambda: gated_scan(x, d), "CUDA device"),
        (lambda: gated_scan(x.half(), d), "bfloat16"),
        (lambda: gated_scan(x, d.bfloat16()), "log_decay"),
        (lambda: gated_scan(x, d[:, :2]), "log_decay"),
        (lambda: gated_scan(x.transpose(0, 1), d.transpose(0, 1)), "contiguous"),
        (lambda: gated_scan(x2, d2), "cu_seqlens"),
        (lambda: gated_scan(x, d, cu_seqlens=cu), "total, C"),
        (lambda: gated_scan(x2, d2, cu_seqlens=cu.long()), "cu_seqlens"),
        (lambda: gated_scan(x2, d2, cu_seqlens=cu[:0]), "offsets"),
        (lambda: gated_scan(x, d, h0=torch.zeros(3, 4)), "h0"),
        (lambda: gated_scan(x, d, h0=torch.zeros(2, 4).bfloat16()), "h0"),
        (lambda: gated_scan_forward(x, d, err=torch.zeros(1)), "err"),
        (lambda: gated_scan_backward(x, d, torch.zeros(1, 4), d), "ckpt"),
        (lambda: gated_scan_backward(x, d, torch.zeros(2, 4), d2), "dh"),
        (lambda: gated_scan_prefill(x2, d2, pool, None), "cu_seqlens"),
        (lambda: gated_scan_prefill(x2, d2, pool[:1], cu), "slots"),
        (lambda: gated_scan_prefill(x2, d2, pool[:, :2], cu), "state"),
        (lambda: gated_scan_prefill(x2, d2, pool, cu, slot_idx=cu), "slot_idx"),
        (lambda: gated_scan_step(x2, d2, pool, slot_idx=cu[:2]), "slot_idx"),
        (lambda: gated_scan_step(x2, d2, pool, new_state=pool[:4]), "new_state"),
        (lambda: gated_scan_step(x2, d2, pool, out=x2[:2]), "out"),
        (lambda: gated_scan_step(x2, d2, pool.double()), "state"),
        (lambda: gated_scan_step(x2, d2, pool), "CUDA device"),
    ]:
        with pytest.raises(ValueError, match=match):
            bad()


def norm_args(**over):
    a = dict(slot_idx=None, slots=0, rows=2, D=8, groups=1, dtype=1, y=P, post=None, gate=None, scale=None, residual=None,
             pre=None, eps=1e-6, out=P, normed=None, stats=None)
    a.update(over)
    return list(a.values()) + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), ARG), (dict(rows=-1), ARG), (dict(D=0), ARG), (dict(groups=3), ARG), (dict(groups=0), ARG),
    (dict(D=8193), UNSUPPORTED), (dict(D=8200, groups=1), UNSUPPORTED), (dict(groups=2, scale=P), UNSUPPORTED),
    (dict(groups=2, pre=P, normed=P), UNSUPPORTED), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(y=None), ARG),
    (dict(out=None), ARG), (dict(pre=P), ARG), (dict(normed=P), ARG), (dict(y=ODD), ARG), (dict(out=ODD), ARG),
    (dict(post=ODD), ARG), (dict(stats=ctypes.c_void_p(68)), ARG), (dict(slot_idx=P, slots=0), ARG), (dict(slot_idx=ODD, slots=2), ARG),
    (dict(rows=1 << 30, groups=4), UNSUPPORTED),
])
def test_norm_refusals(lib, over, status):
    assert lib.dl_block_norm(*norm_args(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(D=8193), UNSUPPORTED), (dict(y=None), ARG), (dict(dgate=P), ARG), (dict(dresidual=P), ARG), (dict(dpost=P), ARG),
    (dict(dscale=P), ARG), (dict(dpre=P), ARG), (dict(dnormed=P), ARG), (dict(post=P, dpost=P, stats=P), ARG), (dict(post=P), ARG), (dict(pre=P), ARG),
    (dict(post=P, stats=ctypes.c_void_p(68)), ARG), (dict(dy=ODD), ARG),
    (dict(dout=ODD), ARG),
])
def test_norm_backward_refusals(lib, over, status):
    a = dict(rows=2, D=8, groups=1, dtype=1, y=P, post=None, gate=None, scale=None, residual=None, pre=None, eps=1e-6,
             stats=None, dout=P, dnormed=None, dy=P, dgate=None, dresidual=None, dpost=None, dscale=None, dpre=None, work=None)
    a.update(over)
    assert lib.dl_block_norm_backward(*a.values(), None) == status


def test_norm_workspace(lib):
    n = ctypes.c_size_t()
    assert lib.dl_block_norm_workspace(4, 64, 2, ctypes.byref(n)) == 0 and n.value == 8 * 3 * 32 * 4
    assert lib.dl_block_norm_workspace(4, 64, 3, ctypes.byref(n)) == ARG
    assert lib.dl_block_norm_workspace(4, 64, 2, None) == ARG
    assert lib.dl_block_norm(*norm_args(rows=0, y=None, out=None)) == 0


def test_norm_python_refusals(lib):
    from recurrent_state_update_deltalog_b200 import block_norm, block_norm_backward
    y, w = torch.zeros(3, 8), torch.ones(8)
    grad = y.clone().requires_grad_()
    idx = torch.zeros(3, dtype=torch.int32)
    for bad, match in [
        (lambda: block_norm(y, w), "CUDA device"),
        (lambda: block_norm(y.double(), w), "bfloat16"),
        (lambda: block_norm(y, w[:4]), "post_weight"),
        (lambda: block_norm(y, w.bfloat16()), "post_weight"),
        (lambda: block_norm(y, w, groups=2), "post_weight"),
        (lambda: block_norm(y, groups=3), "multiple"),
        (lambda: block_norm(y.t(), w[:3]), "contiguous"),
        (lambda: block_norm(y, gate=y[:2]), "gate"),
        (lambda: block_norm(y, gate=y.bfloat16()), "gate"),
        (lambda: block_norm(y, residual=torch.zeros(8, 3).t()), "residual"),
        (lambda: block_norm(y, normed_out=y), "pre_weight"),
        (lambda: block_norm(y, w, out=y[:2]), "out"),
        (lambda: block_norm(y, w, slot_idx=idx[:2]), "slot_idx"),
        (lambda: block_norm(grad, w, out=y), "without gradients"),
        (lambda: block_norm_backward(y, None, y, dnormed=y), "pre_weight"),
        (lambda: block_norm_backward(y, None, y[:2]), "dout"),
        (lambda: block_norm_backward(y, None, y, post_weight=w), "stats"),
        (lambda: block_norm_backward(y, w, y, post_weight=w), "stats"),
    ]:
        with pytest.raises(ValueError, match=match):
            bad()


def paged_args(**over):
    a = dict(slot_idx=None, slots=2, rows=2, Hq=4, Hkv=2, d=64, dtype=1, page=16, pages=8, max_pages=4, table=P, lens=P,
             window=0, scale=0.1, q=P, k=None, v=None, kp=P, vp=P, out=P, work=None, err=None)
    a.update(over)
    return list(a.values()) + [None]


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), ARG), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(rows=-1), ARG), (dict(Hkv=0), ARG),
    (dict(Hq=5), ARG), (dict(Hq=0), ARG), (dict(page=0), UNSUPPORTED), (dict(page=12), UNSUPPORTED),
    (dict(page=1 << 21), UNSUPPORTED), (dict(pages=-1), ARG), (dict(pages=1 << 31), UNSUPPORTED), (dict(pages=1 << 26), UNSUPPORTED), (dict(max_pages=-1), ARG),
    (dict(max_pages=1 << 28), UNSUPPORTED), (dict(slots=1), ARG), (dict(slot_idx=P, slots=0), ARG),
    (dict(rows=65536, slots=65536), UNSUPPORTED), (dict(window=-1), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(table=None), ARG), (dict(lens=None), ARG), (dict(q=None), ARG), (dict(out=None), ARG),
    (dict(kp=None), ARG), (dict(k=P), ARG), (dict(v=P), ARG), (dict(q=ctypes.c_void_p(72)), ARG), (dict(lens=ODD), ARG),
    (dict(table=ODD), ARG), (dict(work=ODD), ARG),
])
def test_paged_refusals(lib, over, status):
    assert lib.dl_paged_attention(*paged_args(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), ARG), (dict(total=1 << 31), ARG), (dict(cu=None), ARG), (dict(k=None), ARG), (dict(vp=None), ARG),
    (dict(k=ctypes.c_void_p(72)), ARG), (dict(starts=ODD), ARG), (dict(page=3), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
])
def test_paged_write_refusals(lib, over, status):
    a = dict(slot_idx=None, slots=2, rows=2, cu=P, total=4, Hkv=2, d=64, dtype=1, page=16, pages=8, max_pages=4, table=P,
             starts=None, k=P, v=P, kp=P, vp=P, err=None)
    a.update(over)
    assert lib.dl_paged_write(*a.values(), None) == status


def test_paged_workspace(lib):
    n = ctypes.c_size_t(1)
    assert lib.dl_paged_attention_workspace(256, 8, 8, 128, 1, 16, 32, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dl_paged_attention_workspace(1, 8, 1, 128, 1, 16, 8192, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.dl_paged_attention_workspace(1, 8, 1, 128, 1, 16, 8192, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dl_paged_attention_workspace(0, 8, 1, 128, 1, 16, 8192, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.dl_paged_attention_workspace(1, 8, 3, 128, 1, 16, 8, 0, ctypes.byref(n)) == ARG
    assert lib.dl_paged_attention_workspace(1, 8, 1, 128, 1, 16, 8, 0, None) == ARG


def test_paged_without_rows_is_a_no_op(lib):
    assert lib.dl_paged_attention(*paged_args(rows=0, q=None, out=None, lens=None)) == 0


def test_paged_python_refusals(lib):
    from recurrent_state_update_deltalog_b200 import paged_attention, paged_write
    q, kp, tb, ln = torch.zeros(2, 4, 64), torch.zeros(5, 2, 16, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k, cu = torch.zeros(2, 2, 64), torch.zeros(3, dtype=torch.int32)
    for bad, match in [
        (lambda: paged_attention(q, kp, kp, tb, ln), "CUDA device"),
        (lambda: paged_attention(q.half(), kp, kp, tb, ln), "bfloat16"),
        (lambda: paged_attention(q[0], kp, kp, tb, ln), "dimensions"),
        (lambda: paged_attention(q, kp.bfloat16(), kp, tb, ln), "k_pages"),
        (lambda: paged_attention(q, kp, kp[:4], tb, ln), "v_pages"),
        (lambda: paged_attention(q[:, :3].contiguous(), kp, kp, tb, ln), "heads"),
        (lambda: paged_attention(q, kp, kp, tb.long(), ln), "block_table"),
        (lambda: paged_attention(q, kp, kp, tb[0], ln), "block_table"),
        (lambda: paged_attention(q, kp, kp, tb, ln[:1]), "lens"),
        (lambda: paged_attention(q, kp, kp, tb, ln, k=k), "together"),
        (lambda: paged_attention(q, kp, kp, tb, ln, window=-1), "window"),
        (lambda: paged_attention(q, kp, kp, tb, ln, window=1 << 32), "window"),
        (lambda: paged_attention(q, kp, kp, tb, ln, k=k, v=k[:1]), "v: expected"),
        (lambda: paged_attention(q, kp, kp, tb[:1], ln[:1]), "slots"),
        (lambda: paged_attention(q, kp, kp, tb, ln, out=q[:1]), "out"),
        (lambda: paged_write(k, k[:1], kp, kp, tb, cu), "v: expected"),
        (lambda: paged_write(q, q, kp, kp, tb, cu), "heads"),
        (lambda: paged_write(k, k, kp, kp, tb, cu[:0]), "offsets"),
        (lambda: paged_write(k, k, kp, kp, tb, cu, starts=cu), "starts"),
        (lambda: paged_write(k, k, kp, kp, tb, cu), "CUDA device"),
    ]:
        with pytest.raises(ValueError, match=match):
            bad()
