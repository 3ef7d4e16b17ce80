"""Attention over a paged cache against the formula in 64 bits.

Bounds (U = 2^-24).  A score sums d products; its error is at most 2 d U of the sum of their magnitudes (the factor 2
because tensor cores may truncate where fp32 rounds), plus 4 U of itself for the scale and the subtracted maximum, whose
own value cancels.  exp2 adds 4 U, joining splits 2 U a join (at most 32 joins), a sum over T tokens 2 T U.  With bf16
each weight is rounded to bf16 on its way into the product with v (half a step, 2^-8) but not in the denominator.  So
each term of the numerator is off by a relative w_j, the denominator by max_j of the same without the rounding.
"""
import math

import pytest
import torch

from _bounds import U, assert_within, half, rounded

pytestmark = pytest.mark.gpu


def make(lens, Hkv, G, d, page, dtype, seed, spare_slots=0, width=None):
    """A cache whose every unused entry is NaN, with the table's unused entries out of range."""
    g = torch.Generator().manual_seed(seed)
    rows, slots = len(lens), len(lens) + spare_slots
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    ids = torch.randperm(pages, generator=g)
    table = torch.full((slots, width or max(max(need), 1)), -7, dtype=torch.int32)
    kp = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype)
    vp = kp.clone()
    K = [torch.randn(n, Hkv, d, generator=g).to(dtype) for n in lens]
    V = [torch.randn(n, Hkv, d, generator=g).to(dtype) for n in lens]
    order = torch.randperm(slots, generator=g)[:rows]
    at = 0
    lens_t = torch.full((slots,), -5, dtype=torch.int32)
    for r, n in enumerate(lens):
        table[order[r], :need[r]] = ids[at:at + need[r]].int()
        lens_t[order[r]] = n
        t = torch.arange(n)
        kp[ids[at + t // page], :, t % page] = K[r]
        vp[ids[at + t // page], :, t % page] = V[r]
        at += need[r]
    q = torch.randn(rows, Hkv * G, d, generator=g).to(dtype)
    return dict(q=q, kp=kp, vp=vp, table=table, lens=lens_t, slot=order.int(), K=K, V=V)


def reference(c, G, window, scale, dtype):
    outs, bounds = [], []
    for r, (K, V) in enumerate(zip(c["K"], c["V"])):
        n, Hkv, d = K.shape
        first = max(0, n - window) if window else 0
        k, v = K[first:].double(), V[first:].double()
        q = c["q"][r].double().view(Hkv, G, d)
        if k.shape[0] == 0:
            outs.append(torch.zeros(Hkv * G, d).double())
            bounds.append(torch.zeros(Hkv * G, d).double())
            continue
        s = torch.einsum("hgd,thd->hgt", q, k) * scale
        e_s = torch.einsum("hgd,thd->hgt", q.abs(), k.abs()) * abs(scale) * 2 * d * U + 4 * U * s.abs()
        p = torch.exp(s - s.amax(-1, keepdim=True))
        e_s = e_s + 4 * U * (s - s.amax(-1, keepdim=True)).abs()
        w = e_s + (4 + 64) * U
        l = p.sum(-1, keepdim=True)
        o = torch.einsum("hgt,thd->hgd", p, v) / l
        num = torch.einsum("hgt,thd->hgd", p * (w + (half(dtype) if dtype != torch.float32 else 0) + 2 * k.shape[0] * U), v.abs()) / l
        den = (p * w).sum(-1, keepdim=True) / l + 2 * k.shape[0] * U
        outs.append(o.reshape(-1, d))
        bounds.append((1.01 * (num + o.abs() * den)).reshape(-1, d))
    return torch.stack(outs), torch.stack(bounds)


def check(c, G, window, dtype, new=True, scale=None):
    """Runs with the new token handed over (its place in the pages left NaN), or already stored."""
    from recurrent_state_update_deltalog_b200 import check_errors, paged_attention
    rows, d = len(c["K"]), c["q"].shape[2]
    ref, bound = reference(c, G, window, d ** -0.5 if scale is None else scale, dtype)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    page = kp.shape[2]
    args = {}
    if new:
        k, v = torch.zeros(rows, kp.shape[1], d, dtype=dtype), torch.zeros(rows, kp.shape[1], d, dtype=dtype)
        for r, K in enumerate(c["K"]):
            if len(K):
                k[r], v[r] = K[-1], c["V"][r][-1]
                at = int(c["table"][c["slot"][r].long(), (len(K) - 1) // page])
                kp[at, :, (len(K) - 1) % page] = float("nan")
                vp[at, :, (len(K) - 1) % page] = float("nan")
        args = dict(k=k.cuda(), v=v.cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kp, vp = kp.cuda(), vp.cuda()
    o = paged_attention(c["q"].cuda(), kp, vp, c["table"].cuda(), c["lens"].cuda(), slot_idx=c["slot"].cuda(), window=window,
                        scale=scale, err=err, **args)
    check_errors(err)
    assert_within(o, ref, rounded(bound, ref, dtype), "o")
    assert torch.equal(kp.cpu().view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       c["kp"].view(torch.int16 if dtype == torch.bfloat16 else torch.int32))
    assert torch.equal(vp.cpu().nan_to_num(9.0), c["vp"].nan_to_num(9.0))
    return o


DT = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
@pytest.mark.parametrize("new", [True, False])
def test_ragged_lengths(page, d, dtype, new):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 300, 1000]
    check(make(lens, 2, 4, d, page, dtype, 1, spare_slots=3), 4, 0, dtype, new)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 2), (4, 3), (2, 5), (1, 8), (2, 9), (1, 16), (2, 17), (1, 33)])
def test_head_groups(Hkv, G, d, dtype):
    check(make([77, 1, 200], Hkv, G, d, 16, dtype, 2), G, 0, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("window", [1, 2, 16, 100, 5000])
def test_windows(window, dtype):
    check(make([0, 1, 16, 99, 100, 101, 1500], 2, 4, 128, 32, dtype, 3), 4, window, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lens", [[20000], [9000, 3], [4097, 4096, 1, 0, 2500]], ids=str)
def test_long_rows_split_over_clusters(lens, dtype):
    check(make(lens, 2, 8, 128, 16, dtype, 4), 8, 0, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,page,Hkv,G,window", [(128, 16, 2, 4, 0), (64, 8, 2, 4, 4700), (128, 64, 1, 12, 4700), (64, 1, 1, 9, 0),
                                                 (128, 8, 1, 17, 5001), (64, 128, 3, 1, 0)])
def test_evenly_shared_tables(d, page, Hkv, G, window, dtype):
    """Tables long enough that equal runs of all tiles are dealt out: empty, short and long rows, some of them cut,
    windows that start inside a tile, pages smaller than a tile; with and without the new token."""
    from recurrent_state_update_deltalog_b200 import _native as N
    import ctypes
    lens = [9000, 0, 4500, 17, 6001, 1, 0, 333]
    c = make(lens, Hkv, G, d, page, dtype, 11, spare_slots=2)
    need = ctypes.c_size_t()
    N.call("dl_paged_attention_workspace", len(lens), Hkv * G, Hkv, d, 1 if dtype == torch.bfloat16 else 0, page, c["table"].shape[1],
           window, ctypes.byref(need))
    assert need.value > 0
    for new in (True, False):
        check(c, G, window, dtype, new)


def test_evenly_shared_tables_captured_and_skipped():
    """The two launches of that form in a captured graph, with lengths changed between replays; rows of negative, held
    and too large slots are not written."""
    from recurrent_state_update_deltalog_b200 import DeltaLog, DeltaLogError, check_errors, paged_attention
    c = make([9000, 5000, 40, 7000], 2, 4, 128, 16, torch.bfloat16, 12)
    dev = {k: c[k].cuda() for k in ("q", "kp", "vp", "table", "lens")}
    slot = c["slot"].clone()
    slot[1], slot[3] = -1, int(slot[3]) | DeltaLog.HOLD
    slot = slot.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    live, out = dev["lens"].clone(), torch.full_like(dev["q"], 3.0)
    args = (dev["q"], dev["kp"], dev["vp"], dev["table"])
    want = [paged_attention(*args, n, slot_idx=slot, out=torch.full_like(out, 3.0)) for n in (dev["lens"], dev["lens"] - 39)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paged_attention(*args, live, slot_idx=slot, out=out, err=err)
    for n, w in ((dev["lens"] - 39, want[1]), (dev["lens"], want[0])):
        live.copy_(n)
        out.fill_(3.0)
        g.replay()
        assert torch.equal(out, w) and (out[[1, 3]] == 3.0).all()
    check_errors(err)
    ref, bound = reference(c, 4, 0, 128 ** -0.5, torch.bfloat16)
    i = [0, 2]
    assert_within(out[i], ref[i], rounded(bound, ref, torch.bfloat16)[i], "o")
    slot[2] = 4
    with pytest.raises(DeltaLogError, match="slot index"):
        paged_attention(*args, dev["lens"], slot_idx=slot, err=err)
        check_errors(err)


@pytest.mark.parametrize("dtype", DT)
def test_long_rows_without_a_workspace(dtype):
    """The C call without a workspace splits less, over one cluster; the values stay within the same bounds."""
    import ctypes
    from recurrent_state_update_deltalog_b200 import _native as N
    c = make([6000, 10], 1, 4, 64, 32, dtype, 10)
    ref, bound = reference(c, 4, 0, 0.125, dtype)
    dev = {k: c[k].cuda() for k in ("q", "kp", "vp", "table", "lens", "slot")}
    need = ctypes.c_size_t()
    code = 1 if dtype == torch.bfloat16 else 0
    N.call("dl_paged_attention_workspace", 2, 4, 1, 64, code, 32, c["table"].shape[1], 0, ctypes.byref(need))
    assert need.value > 0
    o = torch.empty_like(dev["q"])
    N.call("dl_paged_attention", dev["slot"].data_ptr(), 2, 2, 4, 1, 64, code, 32, dev["kp"].shape[0], c["table"].shape[1],
           dev["table"].data_ptr(), dev["lens"].data_ptr(), 0, 0.125, dev["q"].data_ptr(), None, None, dev["kp"].data_ptr(),
           dev["vp"].data_ptr(), o.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
    assert_within(o, ref, rounded(bound, ref, dtype), "o")


@pytest.mark.parametrize("dtype", DT)
def test_many_rows_and_a_wide_table(dtype):
    check(make([(i * 37) % 90 for i in range(260)], 4, 1, 64, 16, dtype, 5, width=64), 1, 0, dtype)


@pytest.mark.parametrize("dtype", DT)
def test_large_scores(dtype):
    """Scores of several hundred: the running maximum keeps every exponent at or below zero."""
    check(make([500, 40], 1, 4, 128, 16, dtype, 6), 4, 0, dtype, scale=30.0)


@pytest.mark.parametrize("dtype", DT)
def test_skipped_rows_bad_lengths_and_bad_pages(dtype):
    """Rows of negative, held and too large slots, and of lengths past the table, are not written; an absent page's
    positions do not count."""
    from recurrent_state_update_deltalog_b200 import DeltaLog, DeltaLogError, check_errors, paged_attention
    c = make([40, 40, 40, 40, 40, 40], 2, 4, 64, 16, dtype, 7)
    dev = {k: c[k].cuda() for k in ("q", "kp", "vp", "table", "lens")}
    slot = c["slot"].clone()
    want = check(c, 4, 0, dtype, new=False)
    slot[1], slot[2], slot[3] = -1, int(slot[2]) | DeltaLog.HOLD, 6
    lens = dev["lens"].clone()
    lens[int(slot[4])] = 16 * c["table"].shape[1] + 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(dev["q"], 3.0)
    paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], lens, slot_idx=slot.cuda(), out=out, err=err)
    with pytest.raises(DeltaLogError, match="slot index.*length"):
        check_errors(err)
    assert (out[1:5] == 3.0).all() and torch.equal(out[[0, 5]], want[[0, 5]])
    # the second page of row 0 is absent: positions 0-15 and 32-39 remain
    c["table"][int(c["slot"][0]), 1] = c["kp"].shape[0]
    keep = torch.tensor(list(range(16)) + list(range(32, 40)))
    c["K"][0], c["V"][0] = c["K"][0][keep], c["V"][0][keep]
    ref, bound = reference(c, 4, 0, 64 ** -0.5, dtype)
    o = paged_attention(dev["q"], dev["kp"], dev["vp"], c["table"].cuda(), dev["lens"], slot_idx=c["slot"].cuda(), err=err)
    with pytest.raises(DeltaLogError, match="page id"):
        check_errors(err)
    assert_within(o, ref, rounded(bound, ref, dtype), "o")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("page", [4, 16, 128])
def test_prompts_written_then_decoded(page, dtype):
    """Two prompts in two pieces each through paged_write, then three tokens; out over q in place."""
    from recurrent_state_update_deltalog_b200 import check_errors, paged_attention, paged_write
    Hkv, G, d, T, extra = 2, 4, 64, [70, 33], 3
    c = make([t + extra for t in T], Hkv, G, d, page, dtype, 8, spare_slots=1)
    kp, vp = torch.full_like(c["kp"], float("nan")).cuda(), torch.full_like(c["vp"], float("nan")).cuda()
    table, slot = c["table"].cuda(), c["slot"].cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, slots = [50, 33], [int(s) for s in c["slot"]]
    for piece in range(2):
        lo, hi = ([0, 0], first) if piece == 0 else (first, T)
        starts = torch.zeros(3, dtype=torch.int32)
        for r in range(2):
            starts[slots[r]] = lo[r]
        cu = torch.tensor([0, hi[0] - lo[0], hi[0] - lo[0] + hi[1] - lo[1]], dtype=torch.int32, device="cuda")
        k = torch.cat([c["K"][r][lo[r]:hi[r]] for r in range(2)]).cuda()
        v = torch.cat([c["V"][r][lo[r]:hi[r]] for r in range(2)]).cuda()
        paged_write(k, v, kp, vp, table, cu, starts=starts.cuda(), slot_idx=slot, err=err)
    for t in range(extra):
        lens = torch.zeros(3, dtype=torch.int32)
        part = dict(c, K=[c["K"][r][:T[r] + t + 1] for r in range(2)], V=[c["V"][r][:T[r] + t + 1] for r in range(2)])
        for r in range(2):
            lens[slots[r]] = T[r] + t + 1
        q = c["q"].cuda()
        k = torch.stack([c["K"][r][T[r] + t] for r in range(2)]).cuda()
        v = torch.stack([c["V"][r][T[r] + t] for r in range(2)]).cuda()
        o = paged_attention(q, kp, vp, table, lens.cuda(), k=k, v=v, slot_idx=slot, out=q, err=err)
        ref, bound = reference(part, G, 0, d ** -0.5, dtype)
        assert o.data_ptr() == q.data_ptr()
        assert_within(o, ref, rounded(bound, ref, dtype), "o")
    check_errors(err)
    assert torch.equal(kp.cpu().nan_to_num(9.0), c["kp"].nan_to_num(9.0))
    assert torch.equal(vp.cpu().nan_to_num(9.0), c["vp"].nan_to_num(9.0))


def test_write_reports_bad_ranges_and_pages():
    from recurrent_state_update_deltalog_b200 import DeltaLogError, check_errors, paged_write
    k = torch.ones(20, 1, 64, device="cuda")
    kp = torch.zeros(2, 1, 8, 64, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    for bad in (dict(cu_seqlens=cu(0, 17)), dict(cu_seqlens=cu(0, 21)), dict(cu_seqlens=cu(5, 4)),
                dict(cu_seqlens=cu(0, 8), starts=cu(9)), dict(cu_seqlens=cu(0, 8), starts=cu(-1))):
        paged_write(k, k, kp, vp, table, err=err, **bad)
        with pytest.raises(DeltaLogError, match="length"):
            check_errors(err)
    assert int(torch.count_nonzero(kp)) == 0
    paged_write(k, k, kp, vp, cu(0, 2).view(1, 2), cu(0, 16), err=err)
    with pytest.raises(DeltaLogError, match="page id"):
        check_errors(err)
    assert (kp[0] == 1).all() and (kp[1] == 0).all() and (vp[0] == 1).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: pages at its end are reached."""
    from recurrent_state_update_deltalog_b200 import paged_attention
    pages, Hkv, page, d = 270000, 1, 64, 128          # 2.2e9 elements, 4.4 GB each for keys and values
    kp = torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    K, V = torch.randn(150, 1, d).bfloat16(), torch.randn(150, 1, d).bfloat16()
    t = torch.arange(150, device="cuda")
    kp[table[0].long()[t // page], :, t % page] = K.cuda()
    vp[table[0].long()[t // page], :, t % page] = V.cuda()
    q = torch.randn(1, 4, d).bfloat16()
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    o = paged_attention(q.cuda(), kp, vp, table, lens)
    ref, bound = reference(dict(q=q, K=[K], V=[V]), 4, 0, d ** -0.5, torch.bfloat16)
    assert_within(o, ref, rounded(bound, ref, torch.bfloat16), "o")


def test_stream_and_captured_graph():
    """On another stream, and replayed with lengths that have grown since the capture."""
    from recurrent_state_update_deltalog_b200 import paged_attention
    c = make([700, 30], 2, 4, 128, 16, torch.bfloat16, 9)
    dev = {k: c[k].cuda() for k in ("q", "kp", "vp", "table", "lens", "slot")}
    args = (dev["q"], dev["kp"], dev["vp"], dev["table"])
    want = paged_attention(*args, dev["lens"], slot_idx=dev["slot"])
    short = dev["lens"] - 20
    want_short = paged_attention(*args, short, slot_idx=dev["slot"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = paged_attention(*args, dev["lens"], slot_idx=dev["slot"], stream=side)
    side.synchronize()
    assert torch.equal(o, want)
    live = short.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = paged_attention(*args, live, slot_idx=dev["slot"])
    g.replay()
    assert torch.equal(o, want_short)
    live.copy_(dev["lens"])
    g.replay()
    assert torch.equal(o, want)
    assert math.isfinite(float(o.float().sum()))
