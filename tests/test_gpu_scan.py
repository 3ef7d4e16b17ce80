"""The gated linear recurrence (forward, backward, single token) against its definition in 64 bits.

Bounds.  U = 2^-24, half an ulp of fp32, relative.  A decay a = 2^fl(d log2 e) is off by 2^-22 = 4 U of itself (ex2)
and by 1.5 |d| U of itself: log2 e and the product are rounded, 0.5 + 1 U of an exponent of |d| log2 e, and the
derivative of 2^t is ln 2 of it.  Each product of decays adds one rounding (U) a token, each multiply-add one (U);
folding runs of tokens adds at most one product and one multiply-add a token again.  So token t perturbs the state by
at most (8 + 1.5 |d_t|) U of its magnitude sum H_t = a_t H_{t-1} + |x_t| (a decay's own error meets a_t H_{t-1} only),
and the error obeys E_t = a_t E_{t-1} + (8 + 1.5 |d_t|) U a_t H_{t-1} + 8 U |x_t|.  The backward pass obeys the same
with |dh| in place of |x|.  Outputs in bf16 add half a step of their own.
"""
import pytest
import torch

from _bounds import U, assert_within, rounded

pytestmark = pytest.mark.gpu
C_ERR = 8 * U


def _inputs(lens, C, dtype, seed, strong=False):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    x = torch.randn(total, C, generator=g).to(dtype)
    d = torch.nn.functional.logsigmoid(torch.randn(total, C, generator=g) * (8.0 if strong else 1.5) + (0.0 if strong else 3.0))
    if strong and total:
        d[::7] = 0.0                    # keeps the state whole
        d[3::11] = float("-inf")        # forgets it
    return x, d, torch.randn(len(lens), C, generator=g), torch.randn(total, C, generator=g).to(dtype), torch.randn(len(lens), C, generator=g)


def _reference(lens, x, d, h0, dh=None, dlast=None):
    """h, its bound, h_last, its bound; with dh also dx, dlog_decay, dh0 and theirs."""
    x, a, h0 = x.double(), d.double().exp(), h0.double()
    c = (8 + 1.5 * d.double().abs().clamp(max=200.0)) * U      # past 200 a decay is 0 either way
    C = x.shape[1]
    h, eh = torch.zeros_like(x), torch.zeros_like(x)
    hp, ehp = torch.zeros_like(x), torch.zeros_like(x)      # a_t h_{t-1}
    last, elast = torch.zeros(len(lens), C).double(), torch.zeros(len(lens), C).double()
    dx, edx = torch.zeros_like(x), torch.zeros_like(x)
    dh0, edh0 = torch.zeros_like(last), torch.zeros_like(last)
    t0 = 0
    for r, n in enumerate(lens):
        s, m, e = h0[r], h0[r].abs(), torch.zeros(C).double()
        for t in range(t0, t0 + n):
            hp[t], ehp[t] = a[t] * s, a[t] * (e + c[t] * m)
            e = ehp[t] + C_ERR * x[t].abs()
            s, m = hp[t] + x[t], a[t] * m + x[t].abs()
            h[t], eh[t] = s, e
        last[r], elast[r] = s, e
        if dh is not None:
            R = dlast[r].double() if dlast is not None else torch.zeros(C).double()
            m, e = R.abs(), torch.zeros(C).double()
            for t in range(t0 + n - 1, t0 - 1, -1):
                G, m = dh[t].double() + R, dh[t].double().abs() + m
                e = e + C_ERR * m
                dx[t], edx[t] = G, e
                R, m, e = a[t] * G, a[t] * m, a[t] * (e + c[t] * m)
            dh0[r], edh0[r] = R, e
        t0 += n
    if dh is None:
        return h, eh, last, elast
    dld = hp * dx
    edld = (ehp * dx.abs() + hp.abs() * edx + ehp * edx) + 2 * U * dld.abs()
    return h, eh, last, elast, dx, edx, dld, edld, dh0, edh0


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to("cuda", torch.int32)


SHAPES = [([1], 64), ([1], 1), ([7, 0, 64, 65, 1], 66), ([63, 64, 65, 128, 129], 33), ([1000], 130), ([513, 2, 1029], 64),
          ([3000], 35), ([2] * 40, 96), ([0, 0, 5], 8), ([200, 300, 77, 8], 2048)]


@pytest.mark.parametrize("lens,C", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("strong", [False, True])
def test_packed_forward_and_gradients(lens, C, dtype, strong):
    from recurrent_state_update_deltalog_b200 import check_errors, gated_scan
    x, d, h0, dh, dlast = _inputs(lens, C, dtype, 1, strong)
    ref = _reference(lens, x, d, h0, dh, dlast)
    xs, ds, hs = (t.cuda().requires_grad_() for t in (x, d, h0))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, last = gated_scan(xs, ds, hs, cu_seqlens=_cu(lens), err=err)
    dx, dld, dh0 = torch.autograd.grad((h, last), (xs, ds, hs), (dh.cuda(), dlast.cuda()))
    check_errors(err)
    assert_within(h, ref[0], rounded(ref[1], ref[0], dtype), "h")
    assert_within(last, ref[2], rounded(ref[3], ref[2], torch.float32), "h_last")
    assert_within(dx, ref[4], rounded(ref[5], ref[4], dtype), "dx")
    assert_within(dld, ref[6], rounded(ref[7], ref[6], torch.float32), "dlog_decay")
    assert_within(dh0, ref[8], rounded(ref[9], ref[8], torch.float32), "dh0")


@pytest.mark.parametrize("rows,T,C,dtype", [(3, 70, 64, torch.bfloat16), (2, 1, 37, torch.float32), (1, 2500, 128, torch.float32),
                                            (5, 0, 16, torch.bfloat16)])
def test_equal_rows_without_offsets(rows, T, C, dtype):
    """[rows, T, C] gives what the packed form gives, bit for bit; h0 and either output gradient may be left out."""
    from recurrent_state_update_deltalog_b200 import gated_scan
    x, d, h0, dh, dlast = (t.cuda() for t in _inputs([T] * rows, C, dtype, 2))
    cu = _cu([T] * rows)
    x3, d3 = x.view(rows, T, C).requires_grad_(), d.view(rows, T, C).requires_grad_()
    x2, d2 = x.clone().requires_grad_(), d.clone().requires_grad_()
    h3, l3 = gated_scan(x3, d3)
    h2, l2 = gated_scan(x2, d2, cu_seqlens=cu)
    assert torch.equal(h3.reshape(h2.shape), h2) and torch.equal(l3, l2)
    for grads3, grads2 in (((dh.view(rows, T, C), None), (dh, None)), ((None, dlast), (None, dlast))):
        k = 0 if grads3[0] is not None else 1
        g3 = torch.autograd.grad((h3, l3)[k], (x3, d3), grads3[k], retain_graph=True)
        g2 = torch.autograd.grad((h2, l2)[k], (x2, d2), grads2[k], retain_graph=True)
        for p, q in zip(g3, g2):
            assert torch.equal(p.reshape(q.shape), q)


def test_gradient_against_differences():
    """x and h0 enter linearly and exp(log_decay) linearly, so central differences are exact: for x and h0 the
    gradient, for log_decay the gradient times sinh(s) / s with step s.  The loss is summed in 64 bits; each of the
    two losses is off by at most sum |w| E, which the difference divides by 2 s."""
    import math
    from recurrent_state_update_deltalog_b200 import gated_scan
    lens, C, s = [70, 5], 4, 0.25
    x, d, h0, w, wl = _inputs(lens, C, torch.float32, 3)
    ref = _reference(lens, x, d, h0, w, wl)
    slack = float((w.double().abs() * ref[1]).sum() + (wl.double().abs() * ref[3]).sum()) * 4 / (2 * s)
    cu = _cu(lens)

    def loss(x, d, h0):
        h, last = gated_scan(x.cuda(), d.cuda(), h0.cuda(), cu_seqlens=cu)
        return float((h.double().cpu() * w.double()).sum() + (last.double().cpu() * wl.double()).sum())

    ins = [t.cuda().requires_grad_() for t in (x, d, h0)]
    out = gated_scan(*ins, cu_seqlens=cu)
    grads = torch.autograd.grad(out, ins, (w.cuda(), wl.cuda()))
    for k, t in enumerate((x, d, h0)):
        for at in ((0, 0), (min(64, t.shape[0] - 1), 2), (t.shape[0] - 1, 3)):
            lo, hi = t.clone(), t.clone()
            lo[at] -= s
            hi[at] += s
            step = float(hi[at].double() - lo[at].double()) / 2     # what the rounding of the inputs left of s
            args = [x, d, h0]
            diff = (loss(*args[:k], hi, *args[k + 1:]) - loss(*args[:k], lo, *args[k + 1:])) / (2 * step)
            want = float(grads[k][at])
            if k == 1:
                want *= math.sinh(step) / step
            # the step itself is exact to 2^-24 of d, which moves exp(d) by as much
            assert abs(diff - want) <= slack + 1e-5 * abs(want), (k, at, diff, want, slack)


@pytest.mark.parametrize("C", [64, 33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompts_then_tokens_equal_one_sequence(C, dtype):
    """A prompt on the pool, continued by a second prompt and by single tokens, is the whole sequence; padded, held
    and unnamed slots and their outputs stay as they were; an index past the pool is skipped and reported."""
    from recurrent_state_update_deltalog_b200 import DeltaLog, DeltaLogError, check_errors, gated_scan_prefill, gated_scan_step
    lens, more = [66, 1, 130], [5, 70, 0]
    full = [a + b + 2 for a, b in zip(lens, more)]
    x, d, h0, _, _ = _inputs(full, C, dtype, 4)
    h0.zero_()
    ref = _reference(full, x, d, h0)
    starts = [0, full[0], full[0] + full[1]]
    slots, B = [4, 0, 2], 6
    state = torch.full((B, C), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def part(t, at, n):
        return torch.cat([t[s + a:s + a + k] for s, a, k in zip(starts, at, n)]).cuda()

    def check(h, at, n):
        i = torch.cat([torch.arange(s + a, s + a + k) for s, a, k in zip(starts, at, n)])
        assert_within(h, ref[0][i], rounded(ref[1], ref[0], dtype)[i], "h")

    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    h = gated_scan_prefill(part(x, [0] * 3, lens), part(d, [0] * 3, lens), state, _cu(lens), idx, zero_state=True, err=err)
    check(h, [0] * 3, lens)
    h = gated_scan_prefill(part(x, lens, more), part(d, lens, more), state, _cu(more), idx, err=err)
    check(h, lens, more)
    at = [a + b for a, b in zip(lens, more)]
    rows = torch.tensor([slots[0], -1, slots[1], slots[2], 3 | DeltaLog.HOLD], dtype=torch.int32, device="cuda")
    pick = [0, None, 1, 2, None]
    for t in range(2):
        xs = torch.stack([x[starts[p] + at[p] + t] if p is not None else torch.full((C,), 9.0, dtype=dtype) for p in pick]).cuda()
        ds = torch.stack([d[starts[p] + at[p] + t] if p is not None else torch.zeros(C) for p in pick]).cuda()
        out = torch.full((5, C), -3.0, dtype=dtype, device="cuda")
        kept, before = torch.empty_like(state).fill_(5.0), state.clone()
        h2 = gated_scan_step(xs, ds, state, rows, new_state=kept, err=err)
        assert torch.equal(state, before)
        gated_scan_step(xs, ds, state, rows, out=out, err=err)
        assert (out[1] == -3.0).all() and (out[4] == -3.0).all()
        live = [0, 2, 3]
        assert torch.equal(out[live], h2[live]) and torch.equal(kept[slots], state[slots])
        assert (kept[[1, 3, 5]] == 5.0).all()
        check(out[live], [a + t for a in at], [1] * 3)
    check_errors(err)
    assert (state[[1, 3, 5]] == 7.0).all()
    assert_within(state[slots], ref[2], rounded(ref[3], ref[2], torch.float32), "state")
    before = state.clone()
    past = torch.tensor([B, 1], dtype=torch.int32, device="cuda")
    gated_scan_step(torch.zeros(2, C, dtype=dtype, device="cuda"), torch.zeros(2, C, device="cuda"), state, past, err=err)
    with pytest.raises(DeltaLogError, match="slot index"):
        check_errors(err)
    check_errors(err)                     # cleared
    assert torch.equal(state, before)


def test_invalid_ranges_are_skipped_and_reported():
    from recurrent_state_update_deltalog_b200 import DeltaLogError, check_errors, gated_scan_prefill
    x, d = torch.ones(10, 8, device="cuda"), torch.zeros(10, 8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu in ([0, 4, 11], [0, 4, 2], [-1, 4, 4]):
        state, out = torch.zeros(2, 8, device="cuda"), torch.full((10, 8), -1.0, device="cuda")
        gated_scan_prefill(x, d, state, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out, err=err)
        with pytest.raises(DeltaLogError, match="cu_seqlens"):
            check_errors(err)
        assert (out[4:] == -1.0).all()


@pytest.mark.parametrize("n,C", [(100, 64), (700, 33), (5, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_views_and_in_place(n, C, dtype):
    """Tensors that start on odd addresses take element-wise loads; h may overwrite x."""
    from recurrent_state_update_deltalog_b200 import gated_scan, gated_scan_prefill
    x, d, h0, dh, dlast = _inputs([n], C, dtype, 5)
    ref = _reference([n], x, d, h0, dh, dlast)

    def odd(t):
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        return flat[1:].view(t.shape).copy_(t)

    xv, dv = odd(x).requires_grad_(), odd(d).requires_grad_()
    h, last = gated_scan(xv, dv, h0.cuda(), cu_seqlens=_cu([n]))
    dx, dld = torch.autograd.grad((h, last), (xv, dv), (odd(dh), dlast.cuda()))
    assert_within(h, ref[0], rounded(ref[1], ref[0], dtype), "h")
    assert_within(dx, ref[4], rounded(ref[5], ref[4], dtype), "dx")
    assert_within(dld, ref[6], rounded(ref[7], ref[6], torch.float32), "dlog_decay")
    for xs, ds in ((odd(x), odd(d)), (x.cuda(), d.cuda())):
        state = h0.cuda()
        got = gated_scan_prefill(xs, ds, state, _cu([n]), out=xs)
        assert got.data_ptr() == xs.data_ptr()
        assert_within(got, ref[0], rounded(ref[1], ref[0], dtype), "h")
        assert_within(state, ref[2], rounded(ref[3], ref[2], torch.float32), "state")


def test_stream_and_captured_graphs():
    """Forward and backward on a stream of their own, and captured twice; replays on new inputs give the eager bits."""
    from recurrent_state_update_deltalog_b200 import gated_scan_backward, gated_scan_forward, gated_scan_step
    lens, C = [300, 70], 128
    x, d, h0, dh, dlast = (t.cuda() for t in _inputs(lens, C, torch.bfloat16, 6))
    x2, d2, h02, dh2, dl2 = (t.cuda() for t in _inputs(lens, C, torch.bfloat16, 7))
    cu = _cu(lens)

    def both():
        h, last, ckpt = gated_scan_forward(x, d, h0, cu, checkpoints=True)
        return (h, last, *gated_scan_backward(x, d, ckpt, dh, dlast, cu))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, last, ckpt = gated_scan_forward(x, d, h0, cu, checkpoints=True, stream=side)
    got = (h, last, *gated_scan_backward(x, d, ckpt, dh, dlast, cu, stream=side))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs))
    for t, u in ((x, x2), (d, d2), (h0, h02), (dh, dh2), (dlast, dl2)):
        t.copy_(u)
    want = [t.clone() for t in both()]
    for g, outs in graphs:
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(outs, want))

    state = torch.randn(4, C, device="cuda")
    s0, xs, ds = state.clone(), x[:4].clone(), d[:4].clone()
    eager = s0.clone()
    gated_scan_step(xs, ds, eager)
    gated_scan_step(xs, ds, eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gated_scan_step(xs, ds, state)
    state.copy_(s0)
    g.replay()
    g.replay()
    assert torch.equal(state, eager)
