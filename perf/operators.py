"""The recurrent-block and hybrid-attention operators as workloads: inputs, plain forms, exact values and work.

Three operators: the gated linear recurrence (one token, a ragged prompt batch, a training step), the norms around a
block with its gate and residual scale (one token, a training step), and the attention of one new token over a paged
key-value cache.  The plain forms are elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # one token of one sequence: a decode loop at its latency floor
        {"name": "scan_step_1", "op": "scan_step", "rows": 1, "C": 4096, "type": "bf16"},
        # one token of a full serving batch, rows on scattered slots of the state pool
        {"name": "scan_step_256", "op": "scan_step", "rows": 256, "C": 4096, "type": "bf16"},
        # a ragged batch of new prompts, 64 of up to 1024 tokens
        {"name": "scan_prompts_64", "op": "scan_prompts", "rows": 64, "T": 1024, "C": 4096, "type": "bf16"},
        # a training step on a batch of equal sequences
        {"name": "scan_train_4x4096", "op": "scan_train", "rows": 4, "T": 4096, "C": 4096, "type": "bf16"},
        # a training step on one long sequence of odd sizes
        {"name": "scan_train_1x16385", "op": "scan_train", "rows": 1, "T": 16385, "C": 1001, "type": "fp32"},
        # the joint between two blocks for one token
        {"name": "norm_join_1", "op": "norm_join", "rows": 1, "D": 4096, "type": "bf16"},
        # the joint between two blocks in a training step
        {"name": "norm_train_16384", "op": "norm_train", "rows": 16384, "D": 4096, "type": "bf16"},
        # odd sizes in 32 bits
        {"name": "norm_train_777", "op": "norm_train", "rows": 777, "D": 1111, "type": "fp32"},
        # the norm of each head's output with its gate, between a recurrence and its projection, in a training step
        {"name": "norm_heads_8192", "op": "norm_heads", "rows": 8192, "H": 32, "d": 128, "type": "bf16"},
        # one sequence with a long context
        {"name": "paged_1x131072", "op": "paged", "rows": 1, "T": 131072, "Hq": 32, "Hkv": 8, "d": 128, "page": 16,
         "window": 0, "type": "bf16"},
        # a ragged serving batch
        {"name": "paged_64x16384", "op": "paged", "rows": 64, "T": 16384, "Hq": 32, "Hkv": 4, "d": 128, "page": 32,
         "window": 0, "type": "bf16"},
        # few short sequences with a window, three query heads to a key head, 32 bits
        {"name": "paged_5x700", "op": "paged", "rows": 5, "T": 700, "Hq": 12, "Hkv": 4, "d": 64, "page": 64,
         "window": 300, "type": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_prompts", "scan_train", "norm_join", "norm_train", "norm_heads", "paged", "paged"])
    c = {"op": op, "type": rng.choice(["bf16", "bf16", "fp32"])}
    if op.startswith("scan"):
        c["C"] = _log_int(rng, 64, 8192) if rng.random() < 0.5 else 64 * rng.randint(1, 128)
        if op == "scan_step":
            c["rows"] = _log_int(rng, 1, 256)
        else:
            c["rows"] = _log_int(rng, 1, 128)
            most = (40 << 20) // (c["rows"] * c["C"])  # tokens a row, so that rows * T * C stays under the largest listed
            c["T"] = _log_int(rng, 1, max(1, min(32768, most)))
    elif op == "norm_heads":
        c |= {"H": rng.randint(1, 64), "d": rng.choice([64, 128, rng.randint(16, 300)])}
        c["rows"] = _log_int(rng, 1, (32 << 20) // (c["H"] * c["d"]))
    elif op.startswith("norm"):
        c["D"] = _log_int(rng, 64, 8192) if rng.random() < 0.5 else 8 * rng.randint(8, 1024)
        c["rows"] = _log_int(rng, 1, 256) if op == "norm_join" else _log_int(rng, 1, (64 << 20) // c["D"])
    else:
        c["Hkv"] = rng.choice([1, 2, 4, 8])
        c |= {"Hq": c["Hkv"] * rng.randint(1, 10), "d": rng.choice([64, 128]), "page": rng.choice([8, 16, 32, 64, 128])}
        c["rows"] = _log_int(rng, 1, 128)
        most = (512 << 20) // (c["rows"] * c["Hkv"] * c["d"] * SIZE[c["type"]] * 2)
        c["T"] = _log_int(rng, 1, max(1, min(131072, most)))
        c["window"] = rng.choice([0, 0, rng.randint(1, c["T"])])
    return c


def _lens(case):
    """The rows' lengths of a ragged case: between a sixteenth of T and T, one of them T."""
    r = random.Random("%d %d" % (case["rows"], case["T"]))
    lens = [r.randint(max(1, case["T"] // 16), case["T"]) for _ in range(case["rows"])]
    lens[r.randrange(len(lens))] = case["T"]
    return lens


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(int(seed))
    dt, op = TYPES[case["type"]], case["op"]

    def normal(*shape, dtype=dt, scale=1.0, grad=False):
        t = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(generator=g).mul_(scale).to(dtype)
        return t.requires_grad_(grad)

    def decay(*shape, grad=False):  # log sigmoid of gates around 3: memories of a few to a few hundred tokens
        t = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(generator=g).mul_(1.5).add_(3.0)
        return torch.nn.functional.logsigmoid(t).requires_grad_(grad)

    def weight(*shape, grad=False):
        return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(generator=g).mul_(0.2).add_(1.0).requires_grad_(grad)

    s = {"case": dict(case)}
    if op == "scan_step":
        rows, C = case["rows"], case["C"]
        slots = rows + rows // 4
        s |= {"x": normal(rows, C), "log_decay": decay(rows, C), "state": normal(slots, C, dtype=torch.float32),
              "new_state": torch.zeros(slots, C, device=DEV),
              "slot_idx": torch.randperm(slots, generator=g, device=DEV)[:rows].to(torch.int32)}
    elif op == "scan_prompts":
        rows, C, lens = case["rows"], case["C"], _lens(case)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        s |= {"x": normal(int(cu[-1]), C), "log_decay": decay(int(cu[-1]), C), "cu": cu.to(DEV, torch.int32),
              "longest": max(lens), "state": torch.zeros(rows, C, device=DEV),
              "slot_idx": torch.randperm(rows, generator=g, device=DEV).to(torch.int32)}
    elif op == "scan_train":
        rows, T, C = case["rows"], case["T"], case["C"]
        s |= {"x": normal(rows, T, C, grad=True), "log_decay": decay(rows, T, C, grad=True),
              "h0": normal(rows, C, dtype=torch.float32, grad=True), "dh": normal(rows, T, C),
              "dlast": normal(rows, C, dtype=torch.float32)}
    elif op in ("norm_join", "norm_train"):
        rows, D, grad = case["rows"], case["D"], op == "norm_train"
        s |= {"y": normal(rows, D, scale=2.0, grad=grad), "gate": normal(rows, D, grad=grad),
              "residual": normal(rows, D, scale=3.0, grad=grad), "post": weight(D, grad=grad),
              "scale": weight(D, grad=grad), "pre": weight(D, grad=grad)}
        if grad:
            s |= {"dout": normal(rows, D), "dnormed": normal(rows, D)}
    elif op == "norm_heads":
        rows, H, d = case["rows"], case["H"], case["d"]
        s |= {"y": normal(rows, H * d, grad=True), "gate": normal(rows, H * d, grad=True), "post": weight(d, grad=True),
              "dout": normal(rows, H * d)}
    else:
        rows, Hq, Hkv, d, page = (case[k] for k in ("rows", "Hq", "Hkv", "d", "page"))
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        ids = torch.randperm(sum(need) + 3, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(rows, max(need), dtype=torch.int32, device=DEV)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
        s |= {"q": normal(rows, Hq, d), "k": normal(rows, Hkv, d), "v": normal(rows, Hkv, d),
              "k_pages": normal(sum(need) + 3, Hkv, page, d), "v_pages": normal(sum(need) + 3, Hkv, page, d),
              "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    return s


# -- plain forms ---------------------------------------------------------------------------------------------------

def _shifted(t, n, fill):
    """t one axis-0 shift of n later, the first n filled."""
    return torch.cat([torch.full_like(t[:n], fill), t[:-n]])


def _scan(a, x, longest):
    """h_t = a_t h_{t-1} + x_t along axis 0, by doubling: after each pass an entry spans twice as many steps."""
    n = 1
    while n < longest:
        x = x + a * _shifted(x, n, 0.0)
        a = a * _shifted(a, n, 0.0)
        n *= 2
    return x


def _scan_step(s):
    at = s["slot_idx"].long()
    h = s["state"][at] * torch.exp(s["log_decay"]) + s["x"].float()
    s["new_state"][at] = h
    return [h.to(s["x"].dtype), s["new_state"]]


def _scan_prompts(s):
    a, starts = torch.exp(s["log_decay"]), s["cu"][:-1].long()
    a[starts] = 0.0  # every prompt starts from nothing
    h = _scan(a, s["x"].float(), s["longest"])
    s["state"][s["slot_idx"].long()] = h[s["cu"][1:].long() - 1]
    return [h.to(s["x"].dtype), s["state"]]


def _scan_train(s):
    x, dt = s["x"].detach().float().transpose(0, 1), s["x"].dtype
    a = torch.exp(s["log_decay"].detach()).transpose(0, 1)
    h0, T = s["h0"].detach(), x.shape[0]
    x = x.clone()
    x[0] += a[0] * h0
    h = _scan(a, x, T)
    before = torch.cat([h0[None], h[:-1]])
    g = s["dh"].float().transpose(0, 1).clone()
    g[-1] += s["dlast"]
    later = torch.cat([a[1:], torch.zeros_like(a[:1])])
    G = _scan(later.flip(0), g.flip(0), T).flip(0)
    return [h.transpose(0, 1).to(dt), h[-1], G.transpose(0, 1).to(dt), (a * before * G).transpose(0, 1), a[0] * G[0]]


def _rstd(u):
    return torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)


def _norm_join(s):
    y, gate, dt = s["y"].detach().float(), s["gate"].detach().float(), s["y"].dtype
    out = s["residual"].detach().float() + s["scale"].detach() * (gate * torch.sigmoid(gate)) * (y * _rstd(y) * s["post"].detach())
    return [out.to(dt), (out * _rstd(out) * s["pre"].detach()).to(dt)]


def _norm_train(s):
    y, gate, dt = s["y"].detach().float(), s["gate"].detach().float(), s["y"].dtype
    post, scale, pre = s["post"].detach(), s["scale"].detach(), s["pre"].detach()
    sig = torch.sigmoid(gate)
    act, r1 = gate * sig, _rstd(y)
    yn = y * r1
    out = s["residual"].detach().float() + scale * act * yn * post
    r2 = _rstd(out)
    on, dn = out * r2, s["dnormed"].float()
    d = dn * pre
    dres = s["dout"].float() + r2 * (d - on * (d * on).mean(-1, keepdim=True))
    dpre = (dn * on).sum(0)
    dscale = (dres * act * yn * post).sum(0)
    dpost = (dres * scale * act * yn).sum(0)
    dgate = dres * scale * yn * post * (sig + act * (1 - sig))
    e = dres * scale * act * post
    dy = r1 * (e - yn * (e * yn).mean(-1, keepdim=True))
    return [out.to(dt), (on * pre).to(dt), dy.to(dt), dgate.to(dt), dres.to(dt), dpost, dscale, dpre]


def _norm_heads(s):
    rows, d, dt = s["y"].shape[0], s["post"].shape[0], s["y"].dtype
    y, gate = s["y"].detach().float().view(rows, -1, d), s["gate"].detach().float().view(rows, -1, d)
    sig, r1, post = torch.sigmoid(gate), _rstd(y), s["post"].detach()
    act, yn, do = gate * sig, y * r1, s["dout"].float().view(rows, -1, d)
    e = do * act * post
    dy = r1 * (e - yn * (e * yn).mean(-1, keepdim=True))
    dgate = do * yn * post * (sig + act * (1 - sig))
    flat = (rows, s["y"].shape[1])
    return [(yn * post * act).reshape(flat).to(dt), dy.reshape(flat).to(dt), dgate.reshape(flat).to(dt), (do * act * yn).sum((0, 1))]


def _paged(s):
    c = s["case"]
    rows, Hq, Hkv, d, page = c["rows"], c["Hq"], c["Hkv"], c["d"], c["page"]
    lens = s["lens"].long()
    r = torch.arange(rows, device=DEV)
    last = lens - 1
    at = s["table"][r, last // page].long()
    s["k_pages"][at, :, last % page] = s["k"]
    s["v_pages"][at, :, last % page] = s["v"]
    table = s["table"].long()
    k = s["k_pages"][table].float().transpose(1, 2).reshape(rows, Hkv, -1, d)  # [rows, Hkv, tokens, d]
    v = s["v_pages"][table].float().transpose(1, 2).reshape(rows, Hkv, -1, d)
    q = s["q"].float().view(rows, Hkv, Hq // Hkv, d)
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = torch.arange(k.shape[2], device=DEV)
    keep = j[None] < lens[:, None]
    if c["window"]:
        keep &= j[None] >= lens[:, None] - c["window"]
    score = score.masked_fill(~keep[:, None, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    return [o.reshape(rows, Hq, d).to(s["q"].dtype), s["k_pages"], s["v_pages"]]


PLAIN = {"scan_step": _scan_step, "scan_prompts": _scan_prompts, "scan_train": _scan_train, "norm_join": _norm_join,
         "norm_train": _norm_train, "norm_heads": _norm_heads, "paged": _paged}


# -- the framework's calls -----------------------------------------------------------------------------------------

def _calls(s):
    import recurrent_state_update_deltalog_b200 as dl
    op = s["case"]["op"]
    if op == "scan_step":
        h = dl.gated_scan_step(s["x"], s["log_decay"], s["state"], slot_idx=s["slot_idx"], new_state=s["new_state"])
        return [h, s["new_state"]]
    if op == "scan_prompts":
        h = dl.gated_scan_prefill(s["x"], s["log_decay"], s["state"], s["cu"], slot_idx=s["slot_idx"], zero_state=True)
        return [h, s["state"]]
    if op == "scan_train":
        ins = (s["x"], s["log_decay"], s["h0"])
        h, last = dl.gated_scan(*ins)
        return [h.detach(), last.detach(), *torch.autograd.grad((h, last), ins, (s["dh"], s["dlast"]))]
    if op == "norm_join":
        return list(dl.block_norm(s["y"], s["post"], gate=s["gate"], scale=s["scale"], residual=s["residual"],
                               pre_weight=s["pre"], eps=EPS))
    if op == "norm_train":
        out, normed = dl.block_norm(s["y"], s["post"], gate=s["gate"], scale=s["scale"], residual=s["residual"],
                                 pre_weight=s["pre"], eps=EPS)
        ins = tuple(s[k] for k in ("y", "gate", "residual", "post", "scale", "pre"))
        return [out.detach(), normed.detach(), *torch.autograd.grad((out, normed), ins, (s["dout"], s["dnormed"]))]
    if op == "norm_heads":
        out = dl.block_norm(s["y"], s["post"], gate=s["gate"], groups=s["case"]["H"], eps=EPS)
        return [out.detach(), *torch.autograd.grad(out, (s["y"], s["gate"], s["post"]), s["dout"])]
    o = dl.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], k=s["k"], v=s["v"],
                        window=s["case"]["window"])
    return [o, s["k_pages"], s["v_pages"]]


def run(state):
    if own:
        return _calls(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    n, op = SIZE[case["type"]], case["op"]
    if op == "scan_step":  # x, log_decay, state in; h, state out
        e = case["rows"] * case["C"]
        return {"bytes": e * (2 * n + 12) + 4 * case["rows"], "flops": 2 * e}
    if op == "scan_prompts":
        e = sum(_lens(case)) * case["C"]
        return {"bytes": e * (2 * n + 4) + 4 * case["rows"] * case["C"], "flops": 2 * e}
    if op == "scan_train":  # forward x, log_decay -> h; backward x, log_decay, dh -> dx, dlog_decay
        e, ends = case["rows"] * case["T"] * case["C"], case["rows"] * case["C"]
        return {"bytes": e * (5 * n + 12) + 16 * ends, "flops": 8 * e}
    if op == "norm_join":
        return {"bytes": case["rows"] * case["D"] * 5 * n + 12 * case["D"], "flops": 14 * case["rows"] * case["D"]}
    if op == "norm_train":  # forward y, gate, residual -> out, normed; backward those, two gradients -> three
        return {"bytes": case["rows"] * case["D"] * 13 * n + 36 * case["D"], "flops": 50 * case["rows"] * case["D"]}
    if op == "norm_heads":  # forward y, gate -> out; backward y, gate, dout -> dy, dgate
        e = case["rows"] * case["H"] * case["d"]
        return {"bytes": e * 8 * n + 12 * case["d"], "flops": 30 * e}
    lens = [min(t, case["window"]) if case["window"] else t for t in _lens(case)]
    kv = sum(lens) * case["Hkv"] * case["d"]
    return {"bytes": 2 * kv * n + case["rows"] * case["d"] * n * (2 * case["Hq"] + 2 * case["Hkv"]),
            "flops": 4 * sum(lens) * case["Hq"] * case["d"]}


# -- from the definitions, in 64 bits ------------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "scan_step":
        new = s["new_state"].double()
        rows = []
        for r, slot in enumerate(s["slot_idx"].tolist()):
            new[slot] = s["state"][slot].double() * s["log_decay"][r].double().exp() + s["x"][r].double()
            rows.append(new[slot])
        return [torch.stack(rows), new]
    if op == "scan_prompts":
        x, ld, state, cu = s["x"], s["log_decay"], s["state"].double(), s["cu"].tolist()
        if cu[-1] > 100000:
            return None
        h = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        for r, slot in enumerate(s["slot_idx"].tolist()):
            now = torch.zeros(x.shape[1], dtype=torch.float64, device=DEV)
            for t in range(cu[r], cu[r + 1]):
                now = torch.addcmul(x[t].double(), ld[t].double().exp_(), now)
                h[t] = now
            state[slot] = now
        return [h, state]
    if op == "scan_train":
        x, ld, dh = s["x"].detach(), s["log_decay"].detach(), s["dh"]
        T, h0 = x.shape[1], s["h0"].detach().double()
        h = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        now = h0
        for t in range(T):
            now = torch.addcmul(x[:, t].double(), ld[:, t].double().exp_(), now)
            h[:, t] = now
        dx, dld = torch.empty_like(h), torch.empty_like(h)
        back = s["dlast"].double()
        for t in range(T - 1, -1, -1):
            G, a = dh[:, t].double() + back, ld[:, t].double().exp_()
            back = a * G
            dx[:, t] = G
            dld[:, t] = back * (h[:, t - 1] if t else h0)
        return [h, h[:, -1].clone(), dx, dld, back]
    if op in ("norm_join", "norm_train", "norm_heads"):
        names = [k for k in ("y", "gate", "residual", "post", "scale", "pre") if k in s]
        v = {k: s[k].detach().double().requires_grad_() for k in names}

        def rms(t, w):
            return t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * w

        silu = v["gate"] / (1 + torch.exp(-v["gate"]))
        if op == "norm_heads":
            rows, d = s["y"].shape[0], s["post"].shape[0]
            o = (rms(v["y"].view(rows, -1, d), v["post"]) * silu.view(rows, -1, d)).reshape(rows, -1)
            return [o.detach(), *torch.autograd.grad(o, [v[k] for k in names], s["dout"].double())]
        o = v["residual"] + v["scale"] * silu * rms(v["y"], v["post"])
        n = rms(o, v["pre"])
        if op == "norm_join":
            return [o.detach(), n.detach()]
        got = torch.autograd.grad((o, n), [v[k] for k in names], (s["dout"].double(), s["dnormed"].double()))
        return [o.detach(), n.detach(), *got]
    page, d, win = case["page"], case["d"], case["window"]
    G = case["Hq"] // case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"].tolist()):
        first = max(0, n - win) if win else 0
        t = torch.arange(first, n, device=DEV)
        pid = s["table"][r].long()[t // page]
        k, v = s["k_pages"][pid, :, t % page].double(), s["v_pages"][pid, :, t % page].double()  # [tokens, Hkv, d]
        k[-1], v[-1] = s["k"][r].double(), s["v"][r].double()
        w = torch.softmax(torch.einsum("hgd,thd->hgt", s["q"][r].double().view(-1, G, d), k) / d ** 0.5, -1)
        out[r] = torch.einsum("hgt,thd->hgd", w, v).reshape(-1, d)
    return [out, None, None]
