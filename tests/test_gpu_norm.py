"""The norms around a block, forward and backward, against the formulas in 64 bits.

Bounds (first order, U = 2^-24 = half an ulp of fp32, relative).  A mean over a row in fp32 is off by at most 30 U of
the mean of its terms' magnitudes: a thread adds up to 16 terms in turn, 5 + 5 exchange steps follow, and the terms
carry 2 to 4 roundings.  So 1 / sqrt(mean + eps) is off by 15 U, 4 U of rsqrtf and 2 U: 21 U.  The sigmoid of q is
1 / (1 + e) with e = 2^fl(-q log2 e): e is off by 4 U of itself (ex2 is good to 2^-22) and by 1.5 |q| U (log2 e and
the product are rounded, 0.5 + 1 U of an exponent of |q| log2 e, and 2^t has the slope ln 2 of itself), which reaches
the sum by e / (1 + e) <= 1; the sum adds U and the reciprocal 2 U (1 ulp): (7 + 1.5 |q|) U, taken as a = 9 + 1.5 |q|,
and 1 U more in q * sigmoid.  Products add 1 U a factor.  What a bound says of
one value is carried into the next below, term by term.  A sum over R rows is off by at most R U of the sum of its
terms' magnitudes, in any order.
"""
import pytest
import torch

from _bounds import U, assert_within, rounded

pytestmark = pytest.mark.gpu


def make(rows, D, groups, dtype, seed, parts):
    g = torch.Generator().manual_seed(seed)
    t = {"y": (torch.randn(rows, D, generator=g) * 2).to(dtype)}
    if "gate" in parts:
        t["gate"] = (torch.randn(rows, D, generator=g) * 3).to(dtype)
    if "residual" in parts:
        t["residual"] = (torch.randn(rows, D, generator=g) * 2).to(dtype)
    for name, n in (("post_weight", D // groups), ("scale", D), ("pre_weight", D)):
        if name in parts:
            t[name] = 1 + 0.3 * torch.randn(n, generator=g)
    t["dout"] = torch.randn(rows, D, generator=g).to(dtype)
    t["dnormed"] = torch.randn(rows, D, generator=g).to(dtype)
    return t


def reference(t, groups, eps):
    """{name: (value, bound)} of the outputs and gradients."""
    v = {k: x.double() for k, x in t.items()}
    y = v["y"]
    rows, D = y.shape
    one = torch.ones(D).double()

    def mean(x):                                          # over the groups of a row, spread over the row again
        return x.view(rows, groups, D // groups).mean(-1, keepdim=True).expand(rows, groups, D // groups).reshape(rows, D)

    post = v["post_weight"].repeat(groups) if "post_weight" in v else one
    scale, pre = v.get("scale", one), v.get("pre_weight", one)
    normed = "post_weight" in v
    r1 = (mean(y * y) + eps).rsqrt() if normed else torch.ones_like(y)
    yn = y * r1
    e_yn = 22 * U * yn.abs()
    if "gate" in v:
        q = v["gate"]
        sg = torch.sigmoid(q)
        act, slope = q * sg, sg + q * sg * (1 - sg)
        far = 1.5 * q.abs().clamp(max=200.0) * U          # past 200 a sigmoid is 0 or 1 either way
        e_slope = (14 * U + far) * sg + (24 * U + 2 * far) * act.abs()
    else:
        act, slope, e_slope, far = torch.ones_like(y), torch.zeros_like(y), torch.zeros_like(y), 0.0
    u = scale * post * act * yn
    out = u + v.get("residual", torch.zeros_like(y))
    e_out = (40 * U + far) * u.abs() + U * out.abs()
    res = {"out": (out, e_out)}
    D_, e_D = v["dout"], torch.zeros_like(y)
    if "pre_weight" in v:
        whole = lambda x: x.mean(-1, keepdim=True)        # noqa: E731
        r2 = (whole(out * out) + eps).rsqrt()
        rho = whole(out.abs() * e_out) / (whole(out * out) + eps) + 21 * U
        on = out * r2
        e_on = r2 * e_out + on.abs() * (rho + U)
        res["normed"] = (on * pre, e_on * pre.abs() + U * (on * pre).abs())
        dn = v["dnormed"]
        d = dn * pre
        k = whole(d * on)
        e_k = whole(d.abs() * e_on) + 32 * U * whole((d * on).abs()) + rho * k.abs()
        D_ = v["dout"] + r2 * (d - on * k)
        e_D = (U * D_.abs() + (rho + 4 * U) * r2 * (d.abs() + (on * k).abs())
               + r2 * (e_on * k.abs() + on.abs() * e_k))
        res["pre_weight"] = ((dn * on).sum(0), (dn.abs() * e_on).sum(0) + (rows + 2) * U * (dn * on).abs().sum(0))
    if "residual" in v:
        res["residual"] = (D_, e_D)
    terms = D_ * act * post * yn
    e_terms = e_D * (act * post * yn).abs() + (40 * U + far) * terms.abs()
    if "scale" in v:
        res["scale"] = (terms.sum(0), e_terms.sum(0) + rows * U * terms.abs().sum(0))
    if normed:
        p = D_ * scale * act * yn
        e_p = e_D * (scale * act * yn).abs() + (40 * U + far) * p.abs()
        fold = lambda x: x.sum(0).view(groups, D // groups).sum(0)  # noqa: E731
        res["post_weight"] = (fold(p), fold(e_p) + rows * groups * U * fold(p.abs()))
    if "gate" in v:
        m = scale * post * yn
        g = D_ * m * slope
        res["gate"] = (g, (D_ * m).abs() * e_slope + e_D * (m * slope).abs() + 30 * U * g.abs())
    e = D_ * scale * act * post
    e_e = e_D * (scale * act * post).abs() + (16 * U + far) * e.abs()
    if normed:
        k = mean(e * yn)
        e_k = mean(e_e * yn.abs() + e.abs() * e_yn) + 32 * U * mean((e * yn).abs())
        dy = r1 * (e - yn * k)
        e_dy = r1 * (e_e + e_yn * k.abs() + yn.abs() * e_k) + 26 * U * r1 * (e.abs() + (yn * k).abs())
    else:
        dy, e_dy = e, e_e + U * e.abs()
    res["y"] = (dy, e_dy)
    return res


ALL = ("gate", "residual", "post_weight", "scale", "pre_weight")
PARTS = [ALL, ("post_weight",), ("post_weight", "gate"), ("residual", "pre_weight"), ("gate",), ("residual", "scale"),
         ("post_weight", "residual", "pre_weight"), ("gate", "residual", "scale", "pre_weight")]
ROW = ("gate", "residual", "post_weight", "scale", "pre_weight", "y")


def compare(t, groups, eps, dtype, call_groups=None):
    from recurrent_state_update_deltalog_b200 import block_norm
    ref = reference(t, groups, eps)
    dev = {k: x.cuda() for k, x in t.items()}
    leaves = {k: x.requires_grad_() for k, x in dev.items() if k not in ("dout", "dnormed")}
    got = block_norm(**leaves, groups=groups, eps=eps)
    outs = {"out": got} if "pre_weight" not in t else {"out": got[0], "normed": got[1]}
    grads = torch.autograd.grad(got, list(leaves.values()), [dev["dout"], dev["dnormed"]][:len(outs)])
    outs |= dict(zip(leaves, grads))
    assert set(outs) == set(ref)
    for name, value in outs.items():
        kind = torch.float32 if name.endswith("weight") or name == "scale" else dtype
        assert value.dtype == kind
        assert_within(value, ref[name][0], rounded(ref[name][1], ref[name][0], kind), name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 5), (70, 64), (33, 128), (40, 250), (9, 256), (5, 257), (17, 520), (300, 1111),
                                    (2, 2048), (260, 4096), (3, 4100), (2, 8192), (2, 8191), (0, 64)])
def test_every_part(rows, D, dtype):
    compare(make(rows, D, 1, dtype, rows + D, ALL), 1, 1e-5, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts", PARTS[1:], ids="-".join)
@pytest.mark.parametrize("D", [96, 1000])
def test_parts(parts, D, dtype):
    compare(make(21, D, 1, dtype, 5, parts), 1, 1e-6, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts", PARTS, ids="-".join)
@pytest.mark.parametrize("rows,D", [(1500, 2048), (4800, 512), (4737, 520)])
def test_many_rows(rows, D, parts, dtype):
    """Enough rows that each CTA takes several, the last ones fewer."""
    compare(make(rows, D, 1, dtype, 6, parts), 1, 1e-6, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("parts", [ALL, ("post_weight", "gate"), ("residual", "pre_weight"), ("scale",)], ids="-".join)
@pytest.mark.parametrize("rows,D", [(2960, 33), (2961, 65), (5003, 95), (2977, 127), (9000, 163), (2963, 255), (4000, 257), (2999, 511),
                                    (2960, 513), (3001, 1001), (2965, 2047)])
def test_many_odd_rows(rows, D, parts, dtype):
    """Rows on any address, enough of them that the next is fetched ahead."""
    compare(make(rows, D, 1, dtype, 9, parts), 1, 1e-6, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_odd_heads(dtype):
    compare(make(500, 7 * 163, 7, dtype, 10, ("post_weight", "gate", "residual")), 7, 1e-6, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [163, 301])
def test_many_odd_rows_in_place_and_skipped(D, dtype):
    from recurrent_state_update_deltalog_b200 import DeltaLog, block_norm
    gen = torch.Generator(device="cuda").manual_seed(D)
    rows = 3333
    y, g, r = (torch.randn(rows, D, device="cuda", generator=gen).to(dtype) for _ in range(3))
    w, w2 = (torch.rand(D, device="cuda", generator=gen) + 0.5 for _ in range(2))
    out, normed = block_norm(y, w, g, None, r, w2)
    idx = torch.arange(rows, dtype=torch.int32, device="cuda")
    idx[5::7] = -1
    idx[3::11] |= DeltaLog.HOLD
    skipped = (idx < 0) | (idx & DeltaLog.HOLD != 0)
    y2, r2 = y.clone(), r.clone()
    block_norm(y2, w, g, None, r2, w2, slot_idx=idx, slots=rows, out=r2, normed_out=y2)
    assert torch.equal(r2, torch.where(skipped[:, None], r, out)) and torch.equal(y2, torch.where(skipped[:, None], y, normed))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H,d", [(1, 1, 64), (5, 3, 64), (700, 4, 128), (3, 7, 33), (2, 5, 300), (1500, 2, 16)])
@pytest.mark.parametrize("parts", [("post_weight", "gate"), ("post_weight", "residual")], ids="-".join)
def test_groups(rows, H, d, parts, dtype):
    compare(make(rows, H * d, H, dtype, 8, parts), H, 1e-6, dtype)


def test_zero_rows_and_large_values():
    """A row of zeros with eps > 0 gives zeros, not NaN; gates far out give silu's limits."""
    from recurrent_state_update_deltalog_b200 import block_norm
    y = torch.zeros(2, 512, device="cuda")
    y[1] = 2.0
    gate = torch.tensor([[-200.0, 200.0] * 256] * 2, device="cuda")
    w = torch.ones(512, device="cuda")
    out = block_norm(y, w, gate=gate, eps=1e-6)
    assert (out[0] == 0).all() and (out[1, ::2].abs() < 1e-30).all()
    assert torch.allclose(out[1, 1::2], torch.tensor(200.0, device="cuda"), rtol=1e-5)


def test_gradient_against_differences():
    """Central differences of the fp32 forward.  The step is 2^-6 of values of order 1: the cubic term and the
    rounding of the loss (2^-24 of about 3000 terms of order 1, over the step) both stay under 2% of a gradient of
    order 1, which is what is asked for."""
    from recurrent_state_update_deltalog_b200 import block_norm
    t = make(4, 96, 1, torch.float32, 11, ALL)
    dev = {k: x.cuda() for k, x in t.items()}
    leaves = {k: x.requires_grad_() for k, x in dev.items() if k not in ("dout", "dnormed")}
    grads = dict(zip(leaves, torch.autograd.grad(block_norm(**leaves), list(leaves.values()), [dev["dout"], dev["dnormed"]])))

    def loss(**kw):
        o, n = block_norm(**kw)
        return float((o.double() * dev["dout"].double()).sum() + (n.double() * dev["dnormed"].double()).sum())

    with torch.no_grad():
        for name, leaf in leaves.items():
            g = torch.Generator().manual_seed(1)
            way = torch.randn(leaf.shape, generator=g).cuda()
            way /= way.norm()
            s = 2.0 ** -6
            diff = (loss(**{**leaves, name: leaf + s * way}) - loss(**{**leaves, name: leaf - s * way})) / (2 * s)
            want = float((grads[name].double() * way.double()).sum())
            assert abs(diff - want) < 0.02 * max(1.0, abs(want)), (name, diff, want)


def test_in_place_and_skipped_rows():
    """The residual stream updated in place; rows of padded, held and too large slots keep what they held."""
    from recurrent_state_update_deltalog_b200 import DeltaLog, block_norm
    t = make(5, 256, 1, torch.bfloat16, 12, ALL)
    dev = {k: x.cuda() for k, x in t.items() if k not in ("dout", "dnormed")}
    want, wantn = block_norm(**dev)
    kept = dev["residual"].clone()
    idx = torch.tensor([2, -1, 0, 1 | DeltaLog.HOLD, 9], dtype=torch.int32, device="cuda")
    normed = torch.full_like(kept, 4.0)
    out, n = block_norm(**dev, slot_idx=idx, slots=9, out=dev["residual"], normed_out=normed)
    assert out.data_ptr() == dev["residual"].data_ptr() and n.data_ptr() == normed.data_ptr()
    assert torch.equal(out[[0, 2]], want[[0, 2]]) and torch.equal(n[[0, 2]], wantn[[0, 2]])
    assert torch.equal(out[[1, 3, 4]], kept[[1, 3, 4]]) and (n[[1, 3, 4]] == 4.0).all()


def test_unaligned_views():
    """Tensors that start on odd addresses take the narrow loads; the values stay within the same bounds."""
    t = make(6, 264, 1, torch.bfloat16, 13, ALL)
    odd = {}
    for k, x in t.items():
        flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
        odd[k] = flat[1:].view(x.shape)
        odd[k].copy_(x)
    from recurrent_state_update_deltalog_b200 import block_norm
    ref = reference(t, 1, 1e-6)
    out, normed = block_norm(**{k: x for k, x in odd.items() if k not in ("dout", "dnormed")})
    assert_within(out, ref["out"][0], rounded(ref["out"][1], ref["out"][0], torch.bfloat16), "out")
    assert_within(normed, ref["normed"][0], rounded(ref["normed"][1], ref["normed"][0], torch.bfloat16), "normed")


def test_stream_and_captured_graphs():
    """Backward on another stream, and in two captured graphs with a workspace each, gives the eager bits."""
    from recurrent_state_update_deltalog_b200 import block_norm_backward, block_norm_forward
    t = {k: x.cuda() for k, x in make(600, 512, 1, torch.bfloat16, 14, ALL).items()}

    def back(**kw):
        parts = (t["post_weight"], t["gate"], t["scale"], t["residual"], t["pre_weight"])
        out, normed, stats = block_norm_forward(t["y"], *parts, **kw)
        return (out, normed, *block_norm_backward(t["y"], stats, t["dout"], t["dnormed"], *parts, **kw))

    want = [x.clone() for x in back()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = back(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = back()
        graphs.append((g, outs))
    t["y"].copy_(make(600, 512, 1, torch.bfloat16, 15, ALL)["y"])
    want = [x.clone() for x in back()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_shared_input_gradients_add_up():
    """y used as residual too: its gradient is the sum of both parts' (autograd adds them)."""
    from recurrent_state_update_deltalog_b200 import block_norm
    t = make(4, 64, 1, torch.float32, 16, ("post_weight",))
    y = t["y"].cuda().requires_grad_()
    w = t["post_weight"].cuda()
    out = block_norm(y, w, residual=y)
    (both,) = torch.autograd.grad(out.sum(), y)
    one = torch.autograd.grad(block_norm(y, w).sum(), y)[0]
    assert torch.allclose(both, one + 1.0, rtol=1e-6, atol=1e-6)


def test_refusals_of_the_library_reach_python():
    from recurrent_state_update_deltalog_b200 import DeltaLogError, block_norm, paged_attention
    y = torch.zeros(2, 8193, device="cuda")
    with pytest.raises(DeltaLogError, match="8192") as e:
        block_norm(y)
    assert e.value.status == -2
    q = torch.zeros(1, 2, 96, device="cuda")
    kp = torch.zeros(1, 2, 16, 96, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(DeltaLogError, match="64, 128"):
        paged_attention(q, kp, kp, one.view(1, 1), one)
    with pytest.raises(ValueError, match="stream"):
        block_norm(torch.zeros(2, 8), stream=torch.cuda.current_stream())


def test_no_second_derivative_and_no_graph_without_need():
    """Differentiating twice raises; inputs without gradients give plain outputs; a leaf used in place is noticed."""
    from recurrent_state_update_deltalog_b200 import block_norm, gated_scan, gated_scan_step
    x = torch.randn(2, 16, device="cuda", requires_grad=True)
    w = torch.ones(16, device="cuda")
    (g,) = torch.autograd.grad(block_norm(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    s = torch.randn(1, 5, 16, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(gated_scan(s, torch.zeros(1, 5, 16, device="cuda"))[0].square().sum(), s, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    assert not block_norm(x.detach(), w).requires_grad
    with torch.no_grad():
        assert not block_norm(x, w).requires_grad
    pool = torch.ones(2, 16, device="cuda")
    y = (x * pool).sum()
    gated_scan_step(torch.zeros(2, 16, device="cuda"), torch.zeros(2, 16, device="cuda"), pool)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()


def test_groups_as_a_dimension_or_inside_the_last():
    """[T, H, d] with a weight [d] is [T, H d]; [T, H, D] with a weight [D / H] keeps its groups in the last dimension."""
    from recurrent_state_update_deltalog_b200 import block_norm
    t = make(6, 8 * 64, 8, torch.float32, 17, ("post_weight", "gate"))
    y, gate, w = t["y"].cuda(), t["gate"].cuda(), t["post_weight"].cuda()
    want = block_norm(y, w, gate=gate, groups=8)
    assert torch.equal(block_norm(y.view(6, 8, 64), w, gate=gate.view(6, 8, 64), groups=8).view_as(y), want)
    y3 = y.repeat_interleave(8, 0).view(6, 8, 512)
    got = block_norm(y3, w, gate=gate.repeat_interleave(8, 0).view(6, 8, 512), groups=8)
    assert torch.equal(got, want.repeat_interleave(8, 0).view(6, 8, 512))
