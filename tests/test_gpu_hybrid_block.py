"""The operators together, as one decode of a small hybrid model uses them: a GDN layer with its gated head norms, a
gated-scan layer, an attention layer over a paged cache, joined by the block norms; prompts first, then tokens, on slots
of shared pools with padding rows.  Every output is compared with the whole sequences computed in 64 bits.  fp32
throughout; the tolerance is the library's own for fp32 inputs (1e-4 of the largest output), which test_gpu_parity.py
applies to the recurrent layer alone: the other operators stay within about 1e-6 of their outputs (their own tests),
and none amplifies an error of its inputs by more than the norms' few units."""
import pytest
import torch

pytestmark = pytest.mark.gpu
H, D, W = 2, 64, 128          # heads, head dimension, model width H * D


def _weights(g):
    def w(*shape, scale=1.0):
        return torch.randn(*shape, generator=g) * scale
    return dict(qkv=w(W, 3 * W, scale=W ** -0.5), gate=w(W, W, scale=W ** -0.5), gdn_norm=1 + 0.2 * w(D), gdn_out=w(W, W, scale=W ** -0.5),
                scan_x=w(W, W, scale=W ** -0.5), scan_d=w(W, W, scale=W ** -0.5), att=w(W, 3 * W, scale=W ** -0.5),
                scale=[1 + 0.2 * w(W) for _ in range(3)], pre=[1 + 0.2 * w(W) for _ in range(4)], post=[1 + 0.2 * w(W) for _ in range(3)],
                beta=w(W, H, scale=W ** -0.5), decay=w(W, H, scale=W ** -0.5))


def _project(p, n):
    """What the GDN layer takes from its normalised input n [tokens, W]."""
    q, k, v = (n @ p["qkv"]).split(W, -1)
    q, k, v = (t.reshape(-1, H, D) for t in (q, k, v))
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    return q, k, v, torch.nn.functional.logsigmoid(n @ p["decay"] + 2), torch.sigmoid(n @ p["beta"]), n @ p["gate"]


def _reference(p, x):
    """One sequence x [T, W] in 64 bits."""
    f = lambda o: {k: ([t.double() for t in v] if isinstance(v, list) else v.double()) for k, v in o.items()}  # noqa: E731
    p, x = f(p), x.double()
    rms = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    join = lambda r, y, i: r + p["scale"][i] * rms(y) * p["post"][i]          # noqa: E731
    T = x.shape[0]
    q, k, v, ld, beta, gate = _project(p, rms(x) * p["pre"][0])
    S, o = torch.zeros(H, D, D).double(), []
    for t in range(T):
        S = S * ld[t].exp()[:, None, None]
        b = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * b[:, None]
        o.append(torch.einsum("hkv,hk->hv", S, q[t]))
    o = rms(torch.stack(o)) * p["gdn_norm"] * torch.nn.functional.silu(gate).view(T, H, D)
    r = join(x, o.reshape(T, W) @ p["gdn_out"], 0)
    n = rms(r) * p["pre"][1]
    sx, sd = n @ p["scan_x"], torch.nn.functional.logsigmoid(n @ p["scan_d"] + 3)
    h, hs = torch.zeros(W).double(), []
    for t in range(T):
        h = sd[t].exp() * h + sx[t]
        hs.append(h)
    r = join(r, torch.stack(hs), 1)
    n = rms(r) * p["pre"][2]
    q, k, v = ((n @ p["att"]).view(T, 3, H, D)).unbind(1)
    s = torch.einsum("thd,shd->hts", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(T, T).triu(1).bool(), float("-inf"))
    a = torch.einsum("hts,shd->thd", s.softmax(-1), v).reshape(T, W)
    r = join(r, a, 2)
    return rms(r) * p["pre"][3]


def test_hybrid_decode_equals_whole_sequences():
    from recurrent_state_update_deltalog_b200 import (DeltaLog, block_norm, check_errors, gated_scan_prefill, gated_scan_step,
                                                      paged_attention, paged_write)
    g = torch.Generator().manual_seed(3)
    lens, extra, slots, B, page = [37, 70, 1], 9, [3, 0, 2], 4, 16
    p = _weights(g)
    xs = [torch.randn(n + extra, W, generator=g) for n in lens]
    ref = [_reference(p, x) for x in xs]
    dev = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in p.items()}
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens).cumsum(0).to("cuda", torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = DeltaLog(B, H, D, D, M=4, op="gdn", dtype=torch.float32)
    pool = torch.zeros(B, W, device="cuda")
    need = [-(-(n + extra) // page) for n in lens]
    kp = torch.full((sum(need), H, page, D), float("nan"), device="cuda")
    vp, table = kp.clone(), torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(sum(need), generator=g).to(torch.int32)
    for s, n, i in zip(slots, need, range(len(need))):
        table[s, :n] = ids[sum(need[:i]):sum(need[:i + 1])].cuda()
    kv_lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def model(x, gdn, scan, attend):
        n = block_norm(x, dev["pre"][0])
        q, k, v, ld, beta, gate = _project(dev, n)
        o = gdn(q.contiguous(), k.contiguous(), v.contiguous(), ld.contiguous(), beta.contiguous(), gate.view(-1, H, D))
        r, n = block_norm(o.reshape(-1, W) @ dev["gdn_out"], dev["post"][0], scale=dev["scale"][0], residual=x, pre_weight=dev["pre"][1])
        y = scan(n @ dev["scan_x"], torch.nn.functional.logsigmoid(n @ dev["scan_d"] + 3))
        r, n = block_norm(y, dev["post"][1], scale=dev["scale"][1], residual=r, pre_weight=dev["pre"][2], out=r)
        q, k, v = (t.contiguous() for t in (n @ dev["att"]).view(-1, 3, H, D).unbind(1))
        a = attend(q, k, v)
        return block_norm(a.reshape(-1, W), dev["post"][2], scale=dev["scale"][2], residual=r, pre_weight=dev["pre"][3])[1]

    def check(got, want, what):
        rel = float((got.double().cpu() - want).abs().max() / want.abs().max())
        assert rel < 1e-4, (what, rel)

    # prompts: the attention layer's own prompt pass is not the library's; its outputs come from torch
    def prompt_attention(q, k, v):
        paged_write(k, v, kp, vp, table, cu, slot_idx=idx, err=err)
        out = []
        for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
            s = torch.einsum("thd,shd->hts", q[a:b], k[a:b]) * D ** -0.5
            s = s.masked_fill(torch.ones(b - a, b - a, device="cuda").triu(1).bool(), float("-inf"))
            out.append(torch.einsum("hts,shd->thd", s.softmax(-1), v[a:b]))
        return torch.cat(out)

    def prompt_gdn(q, k, v, ld, beta, gate):
        o = h.prefill(q, k, v, ld, beta, cu_seqlens=cu, slot_idx=idx, zero_state=True)
        return block_norm(o, dev["gdn_norm"], gate=gate, groups=H)

    out = model(torch.cat([x[:n] for x, n in zip(xs, lens)]).cuda(), prompt_gdn,
                lambda x, d: gated_scan_prefill(x, d, pool, cu, idx, zero_state=True, err=err), prompt_attention)
    check(out, torch.cat([r[:n] for r, n in zip(ref, lens)]), "prompts")
    for s, n in zip(slots, lens):
        kv_lens[s] = n

    # tokens: a padding row between the sequences
    rows = torch.tensor([slots[0], -1, slots[1], slots[2]], dtype=torch.int32, device="cuda")
    live = [0, 2, 3]
    for t in range(extra):
        kv_lens[torch.tensor(slots, device="cuda")] += 1
        x = torch.zeros(4, W)
        for r, (s, n) in zip(live, zip(xs, lens)):
            x[r] = s[n + t]
        x[1] = 0.5
        out = model(x.cuda(),
                    lambda q, k, v, ld, beta, gate: h.step(q, k, v, ld, beta, slot_idx=rows, norm_weight=dev["gdn_norm"], gate=gate,
                                                           out=torch.zeros_like(v)),
                    lambda x, d: gated_scan_step(x, d, pool, rows, out=torch.zeros_like(x), err=err),
                    lambda q, k, v: paged_attention(q, kp, vp, table, kv_lens, k=k, v=v, slot_idx=rows, out=torch.zeros_like(q), err=err))
        check(out[live], torch.stack([r[n + t] for r, n in zip(ref, lens)]), f"token {t}")
    h.check_device()
    check_errors(err)
    h.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step_with_norm_is_the_norm_of_the_step(dtype):
    from recurrent_state_update_deltalog_b200 import DeltaLog, block_norm
    B, d = 5, 128
    g = torch.Generator().manual_seed(1)
    q, k, v, gate = (torch.randn(B, H, d, generator=g).to("cuda", dtype) for _ in range(4))
    k = torch.nn.functional.normalize(k.float(), dim=-1).to(dtype)
    ld, beta = torch.full((B, H), -0.1, device="cuda"), torch.full((B, H), 0.5, device="cuda")
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    idx = torch.tensor([4, -1, 0, 2 | DeltaLog.HOLD, 1], dtype=torch.int32, device="cuda")
    a, b = (DeltaLog(B, H, d, d, M=3, op="gdn", dtype=dtype) for _ in range(2))
    for _ in range(4):
        want = torch.full_like(v, 2.0)
        a.step(q, k, v, ld, beta, slot_idx=idx, out=want)
        plain = want.clone()
        want = block_norm(plain, w, gate=gate, groups=H, eps=1e-5)
        got = torch.full_like(v, 2.0)
        assert b.step(q, k, v, ld, beta, slot_idx=idx, out=got, norm_weight=w, gate=gate, norm_eps=1e-5) is got
        live = [0, 2, 4]
        assert torch.equal(got[live], want[live]) and (got[[1, 3]] == 2.0).all()
    n = b.log_len
    for bad in (dict(gate=gate), dict(norm_weight=w[:64]), dict(norm_weight=w, gate=gate[:2])):
        with pytest.raises(ValueError):
            b.step(q, k, v, ld, beta, slot_idx=idx, **bad)
    assert b.log_len == n                     # a refused call takes no step
    a.close()
    b.close()
