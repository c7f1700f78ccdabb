"""The products of the routed experts as they are trained and decoded, and the cases they are measured on.

Four groups, each with its gradient:

  experts   matrix products grouped by expert: rows in expert order, ragged, in 16 bits; the gradients of rows and weights
  swiglu    silu(gate) * up between the two products of an expert
  combine   the weighted sum over a token's experts behind them
  w4        products of few tokens with 4-bit weights that have a scale for each group along a row: of one matrix (a
            shared expert, a projection), or of the experts that each token is routed to

With `own` false `run` computes them from elementary torch operations in 32 bits; with `own` true it makes the calls of
`quantized_mixture_experts_moe_gb300.binding`.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token through the gate and up projections of its 8 experts of 128
        dict(name="experts_T1", op="experts", T=1, E=128, k=8, N=1536, K=2048, type="bf16", gather=True, skew=0.0, dir="fwd"),
        # a long prompt through the gate and up projections
        dict(name="experts_T8192", op="experts", T=8192, E=64, k=8, N=2816, K=4096, type="bf16", gather=True, skew=0.0, dir="fwd"),
        # a ragged batch, odd widths, experts that few or no tokens choose: a down projection of rows in expert order
        dict(name="experts_T1021_odd", op="experts", T=1021, E=24, k=4, N=2047, K=1407, type="f16", gather=False, skew=1.2, dir="fwd"),
        # training: the gradients of the down projection, unevenly loaded experts
        dict(name="experts_bwd_T4096", op="experts", T=4096, E=128, k=8, N=2048, K=768, type="bf16", gather=False, skew=0.8, dir="bwd"),
        # training: gate and up projections, forward and both gradients
        dict(name="experts_step_T8192", op="experts", T=8192, E=64, k=4, N=2816, K=2048, type="bf16", gather=True, skew=0.3, dir="step"),
        # one decoded token between the two products of its experts
        dict(name="swiglu_T1", op="swiglu", P=8, I=768, type="bf16", dir="fwd"),
        # training: the gradient, with the activation made again for the gradient of the down projection
        dict(name="swiglu_bwd_P65536", op="swiglu", P=65536, I=1408, type="bf16", dir="bwd"),
        # the gradient of the weighted sum for a few sequences being fine-tuned
        dict(name="combine_bwd_T64", op="combine", T=64, k=8, H=2048, type="bf16", drop=0.0, dir="bwd"),
        # the same for a large batch, some pairs not routed
        dict(name="combine_bwd_T8192", op="combine", T=8192, k=10, H=4096, type="bf16", drop=0.05, dir="bwd"),
        # one decoded token through a shared expert's gate and up projection in int4
        dict(name="w4_T1", op="w4", T=1, N=2816, K=2048, type="bf16", format="int4", group=32, E=0, k=1, dir="fwd"),
        # four decoded tokens through the gate and up projections of their 10 experts of 512, in E2M1
        dict(name="w4_experts_T4", op="w4", T=4, N=2048, K=4096, type="bf16", format="mxfp4", group=32, E=512, k=10, dir="fwd"),
        # fine-tuning beside a frozen 4-bit layer: the product and the gradient of its input
        dict(name="w4_step_T2048", op="w4", T=2048, N=2816, K=4096, type="f16", format="int4", group=128, E=0, k=1, dir="step"),
    ]


WIDTHS = (64, 128, 256, 512, 768, 1024, 1408, 1536, 2048, 2816, 4096)
MOST = 2.0 * 65536 * 2816 * 4096   # operations of the largest case
WEIGHTS = 64 * 2816 * 4096         # elements of the largest expert weight


def _ragged(rng, lo, hi):
    """A size spread over its logarithm that no tile divides."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n + (n > 64 and n % 64 == 0)))


def _width(rng, lo, hi):
    return rng.choice([w for w in WIDTHS if lo <= w <= hi]) if rng.random() < 0.7 else _ragged(rng, lo, hi)


def draw(rng):
    op = rng.choice(["experts", "experts", "experts", "swiglu", "combine", "w4", "w4"])
    T = 2 ** rng.randint(0, 13) if rng.random() < 0.4 else _ragged(rng, 1, 8192)
    type = rng.choice(["bf16", "bf16", "f16"])
    if op == "experts":
        E = rng.choice([8, 16, 64, 128, 512, _ragged(rng, 8, 512)])
        N, K, k = _width(rng, 64, 4096), _width(rng, 64, 4096), rng.randint(1, min(E, 10))
        while E * N * K > WEIGHTS:
            E = max(8, E // 2)
        k, dir = min(k, E), rng.choice(["fwd", "fwd", "bwd", "step"])
        while (6.0 if dir == "step" else 4.0 if dir == "bwd" else 2.0) * T * k * N * K > MOST:
            T = max(1, T // 2)
        return dict(op=op, T=T, E=E, k=k, N=N, K=K, type=type, gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.3, 0.8, 1.2]), dir=dir)
    if op == "swiglu":
        P = min(65536, T * rng.randint(1, 10))
        return dict(op=op, P=P, I=_width(rng, 64, 1408), type=rng.choice(["bf16", "f16", "f32"]) if P <= 32768 else type, dir=rng.choice(["fwd", "bwd"]))
    if op == "combine":
        return dict(op=op, T=T, k=rng.randint(1, 10), H=_width(rng, 64, 4096), type=type, drop=rng.choice([0.0, 0.05, 0.5]), dir=rng.choice(["fwd", "bwd"]))
    format = rng.choice(["int4", "int4", "mxfp4"])
    group = 32 if format == "mxfp4" else rng.choice([32, 64, 128])
    N, K = _width(rng, 64, 4096), max(group, _width(rng, 64, 4096) // group * group)
    if rng.random() < 0.4:
        T = rng.randint(1, 16)
        E = rng.choice([8, 64, 128, 512, _ragged(rng, 8, 512)])
        return dict(op=op, T=T, N=N, K=K, type=type, format=format, group=group, E=E, k=rng.randint(1, 8), dir="fwd")
    return dict(op=op, T=T if rng.random() < 0.5 else _ragged(rng, 1, 128), N=N, K=K, type=type, format=format, group=group, E=0, k=1, dir=rng.choice(["fwd", "fwd", "step"]))


def work(c):
    s = SIZE[c["type"]]
    if c["op"] == "experts":
        P, N, K = c["T"] * c["k"], c["N"], c["K"]
        x, w, y = (c["T"] if c["gather"] else P) * K * s, min(c["E"], P) * N * K, P * N * s
        fwd = {"bytes": x + w * s + y, "flops": 2.0 * P * N * K}
        # dy, x, w -> dx in expert order, dw in 32 bits for all experts
        bwd = {"bytes": y + x + w * s + P * K * s + 4 * c["E"] * N * K, "flops": 4.0 * P * N * K}
        if c["dir"] != "step":
            return fwd if c["dir"] == "fwd" else bwd
        return {"bytes": x + w * s + 2 * y + P * K * s + 4 * c["E"] * N * K, "flops": fwd["flops"] + bwd["flops"]}
    if c["op"] == "swiglu":
        n = c["P"] * c["I"]
        return {"bytes": n * s * (3 if c["dir"] == "fwd" else 6), "flops": n * (6 if c["dir"] == "fwd" else 14)}
    if c["op"] == "combine":
        P, H, T = c["T"] * c["k"], c["H"], c["T"]
        n = round(P * (1.0 - c["drop"])) * H
        if c["dir"] == "fwd":
            return {"bytes": (n + T * H) * s + 8 * P, "flops": 2.0 * n}
        return {"bytes": (n + P * H + T * H) * s + 12 * P, "flops": 3.0 * n}
    N, K, T = c["N"], c["K"], c["T"]
    w = N * K // 2 + N * (K // c["group"]) * (2 if c["format"] == "int4" else 1)
    if c["E"]:
        return {"bytes": min(c["E"], T * c["k"]) * w + T * K * s + T * c["k"] * (N * s + 4), "flops": 2.0 * T * c["k"] * N * K}
    step = c["dir"] == "step"
    return {"bytes": w + T * (K + N) * s * (2 if step else 1), "flops": 2.0 * T * N * K * (2 if step else 1)}


# ------------------------------------------------------------------ inputs

def _routing(s, g, T, E, k, skew, drop=0.0):
    """k different experts for each token, chosen with a Zipf law of exponent `skew`; of the pairs a share `drop` is routed
    nowhere.  Adds what the routing sort gives: offsets, the pair of each slot and the slot of each pair."""
    score = -skew * torch.log(1.0 + torch.arange(E, device=DEVICE)) - torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEVICE).clamp(1e-12, 1.0 - 1e-7)))
    ids = score.topk(k, dim=1).indices.reshape(-1)
    if drop:
        ids = ids.masked_fill(torch.rand(T * k, generator=g, device=DEVICE) < drop, E)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    s["ids"] = ids.masked_fill(ids == E, -1).int().view(T, k)
    s["counts"] = counts.tolist()
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    n = sum(s["counts"])
    there = torch.arange(T * k, device=DEVICE) < n
    s["pairs"] = torch.where(there, order, -1).int()
    slot = torch.full((T * k,), -1, dtype=torch.int32, device=DEVICE)
    slot[order[:n]] = torch.arange(n, dtype=torch.int32, device=DEVICE)
    s["pair_slot"] = slot.view(T, k)


def prepare(c, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))

    def normal(*shape, scale=1.0, type="f32"):
        t = torch.empty(*shape, dtype=TYPES[type], device=DEVICE)
        return t.normal_(generator=g).mul_(scale)

    s, t = {"case": dict(c)}, c["type"]
    if c["op"] == "experts":
        T, N, K = c["T"], c["N"], c["K"]
        _routing(s, g, T, c["E"], c["k"], c["skew"])
        P = T * c["k"]
        # normed activations, a few channels far larger than the rest
        s["x"] = (normal(T if c["gather"] else P, K) * (1.0 + 7.0 * (torch.rand(K, generator=g, device=DEVICE) < 0.01).float())).to(TYPES[t])
        s["w"] = normal(c["E"], N, K, scale=K ** -0.5, type=t)
        if c["dir"] != "fwd":
            s["dy"] = normal(P, N, scale=0.05, type=t)
        return s
    if c["op"] == "swiglu":
        s["gu"] = normal(c["P"], 2 * c["I"], scale=1.5, type=t)
        if c["dir"] == "bwd":
            s["dh"] = normal(c["P"], c["I"], scale=0.1, type=t)
        return s
    if c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        _routing(s, g, T, max(16, 2 * k), k, 0.3, c["drop"])
        s["y"] = normal(T * k, H, scale=0.5, type=t)
        s["w"] = torch.softmax(normal(T, k), 1)
        if c["dir"] == "bwd":
            s["dout"] = normal(T, H, scale=0.1, type=t)
        return s
    T, N, K, group = c["T"], c["N"], c["K"], c["group"]
    lead = (c["E"],) if c["E"] else ()
    if c["E"]:
        _routing(s, g, T, c["E"], c["k"], 0.5)
    # activations of unlike rows, a few channels far larger than the rest
    s["x"] = (normal(T, K) * (0.5 + torch.rand(T, 1, generator=g, device=DEVICE)) * (1.0 + 7.0 * (torch.rand(K, generator=g, device=DEVICE) < 0.01).float())).to(TYPES[t])
    if c["format"] == "int4":
        # codes n = q + 8 with q in [-7, 7], element 2i in the low nibble of byte i
        q = torch.randint(1, 16, (*lead, N, K // 2, 2), generator=g, device=DEVICE, dtype=torch.uint8)
        s["w_q"] = q[..., 0] | q[..., 1] << 4
        s["w_s"] = (0.005 + 0.015 * torch.rand(*lead, N, K // group, generator=g, device=DEVICE)).half()
    else:
        s["w_q"] = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device=DEVICE, dtype=torch.uint8)
        s["w_s"] = torch.randint(119, 124, (*lead, N, K // 32), generator=g, device=DEVICE, dtype=torch.uint8)
    if c["dir"] == "step":
        s["dy"] = normal(T, N, scale=0.05, type=t)
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_experts(s):
    c, w, counts = s["case"], s["w"], s["counts"]
    x = s["x"].float()
    if c["gather"]:
        x = x[s["pairs"].long() // c["k"]]
    P, N, K = x.shape[0], c["N"], c["K"]
    out = []
    if c["dir"] != "bwd":
        y = torch.zeros(P, N, dtype=w.dtype, device=w.device)
        at = 0
        for e, n in enumerate(counts):
            if n:
                y[at:at + n] = x[at:at + n] @ w[e].float().t()
            at += n
        out.append(y)
    if c["dir"] != "fwd":
        dy = s["dy"].float()
        dx = torch.zeros(P, K, dtype=w.dtype, device=w.device)
        dw = torch.zeros(w.shape, device=w.device)
        at = 0
        for e, n in enumerate(counts):
            if n:
                dx[at:at + n] = dy[at:at + n] @ w[e].float()
                torch.matmul(dy[at:at + n].t(), x[at:at + n], out=dw[e])
            at += n
        out += [dx, dw]
    return out


def _plain_swiglu(s):
    gu, I = s["gu"], s["case"]["I"]
    a, b = gu[:, :I].float(), gu[:, I:].float()
    sig = 1.0 / (1.0 + torch.exp(-a))
    h = (a * sig * b).to(gu.dtype)
    if s["case"]["dir"] == "fwd":
        return [h]
    dh = s["dh"].float()
    return [torch.cat([dh * b * sig * (1.0 + a * (1.0 - sig)), dh * a * sig], 1).to(gu.dtype), h]


def _plain_combine(s):
    y, w, slot = s["y"], s["w"], s["pair_slot"].long()
    on = (slot >= 0).float()
    at = slot.clamp(min=0)
    if s["case"]["dir"] == "fwd":
        out = torch.zeros(w.shape[0], y.shape[1], device=y.device)
        for j in range(w.shape[1]):
            out += (w[:, j] * on[:, j]).unsqueeze(1) * y[at[:, j]].float()
        return [out.to(y.dtype)]
    dout = s["dout"].float()
    dy, dw = torch.zeros(y.shape[0] + 1, y.shape[1], dtype=y.dtype, device=y.device), torch.zeros_like(w)
    for j in range(w.shape[1]):
        dw[:, j] = (y[at[:, j]].float() * dout).sum(1) * on[:, j]
        dy[slot[:, j]] = (w[:, j].unsqueeze(1) * dout).to(y.dtype)  # what is routed nowhere goes to the last row
    return [dy[:-1], dw]


def _plain_weight(s, q, scale):
    low, high = q & 15, q >> 4
    n = torch.stack([low, high], -1).reshape(*q.shape[:-1], -1)
    if s["case"]["format"] == "int4":
        v, f = n.float() - 8.0, scale.float()
    else:
        e, m = (n >> 1 & 3).float(), (n & 1).float()
        v = torch.where(e > 0, (2.0 + m) * torch.exp2(e - 2.0), 0.5 * m) * torch.where(n > 7, -1.0, 1.0)
        f = torch.exp2(scale.float() - 127.0)
    return v * f.repeat_interleave(s["case"]["group"], -1)


def _plain_w4(s):
    c, x = s["case"], s["x"].float()
    if c["E"]:
        ids = s["ids"].reshape(-1).long()
        y = [_plain_weight(s, q, f) @ x[p // c["k"]] for p, (q, f) in enumerate(zip(s["w_q"][ids], s["w_s"][ids]))]
        return [torch.stack(y).to(s["x"].dtype)]
    w = _plain_weight(s, s["w_q"], s["w_s"])
    out = [(x @ w.t()).to(s["x"].dtype)]
    if c["dir"] == "step":
        out.append((s["dy"].float() @ w).to(s["x"].dtype))
    return out


PLAIN = {"experts": _plain_experts, "swiglu": _plain_swiglu, "combine": _plain_combine, "w4": _plain_w4}


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    from quantized_mixture_experts_moe_gb300 import binding as qb

    c = s["case"]
    if c["op"] == "experts":
        how = dict(pairs=s["pairs"], k=c["k"]) if c["gather"] else {}
        out = [] if c["dir"] == "bwd" else [qb.expert_linear(s["x"], s["w"], s["offsets"], **how)]
        if c["dir"] != "fwd":
            out += qb.expert_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], **how)
        return out
    if c["op"] == "swiglu":
        if c["dir"] == "fwd":
            return [qb.swiglu(s["gu"])]
        return list(qb.swiglu_backward(s["dh"], s["gu"], h_too=True))
    if c["op"] == "combine":
        if c["dir"] == "fwd":
            return [qb.combine(s["y"], s["w"], s["pair_slot"])]
        return list(qb.combine_backward(s["dout"], s["y"], s["w"], s["pair_slot"], s["offsets"]))
    if c["E"]:
        return [qb.w4_linear(s["x"], s["w_q"], s["w_s"], ids=s["ids"])]
    out = [qb.w4_linear(s["x"], s["w_q"], s["w_s"])]
    if c["dir"] == "step":
        out.append(qb.w4_linear_backward(s["dy"], s["w_q"], s["w_s"]))
    return out


def run(s):
    return _own_run(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions, in 64 bits

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_experts(s):
    c, w, ids = s["case"], s["w"], s["ids"].reshape(-1)
    P = ids.numel()
    slot = s["pair_slot"].reshape(-1).long()
    y = torch.zeros(P, c["N"], dtype=torch.float64, device=DEVICE) if c["dir"] != "bwd" else None
    dx = torch.zeros(P, c["K"], dtype=torch.float64, device=DEVICE) if c["dir"] != "fwd" else None
    dw = torch.zeros(w.shape, dtype=torch.float64, device=DEVICE) if c["dir"] != "fwd" else None
    for e in range(c["E"]):
        mine = (ids == e).nonzero().squeeze(1)  # the expert's pairs
        if not mine.numel():
            continue
        rows = slot[mine]
        a, m = s["x"][mine // c["k"] if c["gather"] else rows].double(), w[e].double()
        if y is not None:
            y[rows] = torch.einsum("sk,nk->sn", a, m)
        if dx is not None:
            b = s["dy"][rows].double()
            dx[rows] = torch.einsum("sn,nk->sk", b, m)
            dw[e] = torch.einsum("sn,sk->nk", b, a)
    return [t for t in (y, dx, dw) if t is not None]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "experts":
        return _exact_experts(s)
    if c["op"] == "swiglu":
        gu = s["gu"].double().requires_grad_(c["dir"] == "bwd")
        g, u = gu.split(c["I"], 1)
        h = g / (1.0 + torch.exp(-g)) * u
        if c["dir"] == "fwd":
            return [h]
        return [torch.autograd.grad(h, gu, s["dh"].double())[0], h.detach()]
    if c["op"] == "combine":
        y, w = s["y"].double().requires_grad_(True), s["w"].double().requires_grad_(True)
        T, k = w.shape
        weight = torch.cat([y, y.new_zeros(1, y.shape[1])])[s["pair_slot"].long().view(-1)].view(T, k, -1)  # -1: the row of zeros
        out = (weight * w.unsqueeze(2)).sum(1)
        if c["dir"] == "fwd":
            return [out.detach()]
        return list(torch.autograd.grad(out, (y, w), s["dout"].double()))

    def dense(q, scale):
        codes = torch.empty(q.shape[0], q.shape[1] * 2, dtype=torch.int64, device=DEVICE)
        codes[:, 0::2], codes[:, 1::2] = q.long() % 16, q.long() // 16
        if c["format"] == "int4":
            v, f = (codes - 8).double(), scale.double()
        else:
            v = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=torch.float64, device=DEVICE)[codes]
            f = torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.int() - 127)
        return (v.view(q.shape[0], -1, c["group"]) * f.unsqueeze(2)).view(q.shape[0], -1)

    x = s["x"].double()
    if c["E"]:
        y = torch.empty(c["T"] * c["k"], c["N"], dtype=torch.float64, device=DEVICE)
        for p, e in enumerate(s["ids"].reshape(-1).tolist()):
            y[p] = (dense(s["w_q"][e], s["w_s"][e]) * x[p // c["k"]]).sum(1)
        return [y]
    w = dense(s["w_q"], s["w_s"])
    return [x @ w.t()] + ([s["dy"].double() @ w] if c["dir"] == "step" else [])
