"""Operators around the routed experts of a Mixture-of-Experts block, and the cases they are measured on.

Three groups, each with its gradient:

  norm_pre, norm_post   root-mean-square norms before and after a block; the one after it is fused with the block's gate,
                        the residual scale, the residual sum and, where asked, the next block's norm
  route                 top-k routing with the balance loss and the per-expert counts
  fp8_linear, fp8_step  the matrix product in 8-bit floating point (E4M3) with one fp32 scale for each 128 values of an
                        activation row and each 128 x 128 block of a weight, with the quantisation of its inputs

With `own` false `run` computes them from elementary torch operations in 32 bits; with `own` true it makes the calls of
`quantized_mixture_experts_moe_gb300.binding`.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
BLK = 128          # values that share one scale
FP8_MAX = 448.0    # largest E4M3 value
TINY = 2.0 ** -100  # least magnitude that a block's scale is made for


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token: the end of a block, with the norm that opens the next one
        dict(name="post_next_T1", op="norm_post", T=1, H=4096, stream="bf16", block="bf16", post=True, gate="token", next=True, dir="fwd"),
        # prefill of 4096 tokens through the same sandwich
        dict(name="post_next_T4096", op="norm_post", T=4096, H=4096, stream="bf16", block="bf16", post=True, gate="token", next=True, dir="fwd"),
        # training, a stream kept in 32 bits, a learned gate for each channel: every gradient of the sandwich
        dict(name="post_next_bwd_T8192", op="norm_post", T=8192, H=4096, stream="f32", block="bf16", post=True, gate="channel", next=True, dir="bwd"),
        # an odd width and a ragged batch: the gradient of the norm that opens a block
        dict(name="pre_bwd_T1021_odd", op="norm_pre", T=1021, H=2047, stream="f16", block="f16", dir="bwd"),
        # one decoded token routed to 10 of 512 experts
        dict(name="route_T1", op="route", T=1, E=512, k=10, dtype="bf16", renorm=True, bias=False, mask=False, holes=False, coef=0.0, dir="fwd"),
        # prefill with padding, experts that are switched off, a selection bias, and the load statistics
        dict(name="route_T8192", op="route", T=8192, E=512, k=10, dtype="bf16", renorm=True, bias=True, mask=True, holes=True, coef=0.01, dir="fwd"),
        # training: routing, balance loss and the gradient of the logits
        dict(name="route_step_T8192", op="route", T=8192, E=128, k=8, dtype="f32", renorm=False, bias=False, mask=True, holes=False, coef=0.01, dir="step"),
        # one decoded token through a shared expert's gate and up projection
        dict(name="linear_T1", op="fp8_linear", T=1, N=2048, K=4096, dtype="bf16"),
        # a decode batch on a projection of ragged width
        dict(name="linear_T60_odd", op="fp8_linear", T=60, N=1407, K=2040, dtype="f16"),
        # a short prompt
        dict(name="linear_T256", op="fp8_linear", T=256, N=2816, K=4096, dtype="bf16"),
        # a long prompt
        dict(name="linear_T8192", op="fp8_linear", T=8192, N=2816, K=4096, dtype="bf16"),
        # training: the product, the gradient of its input and of its weight, with all quantisation
        dict(name="linear_step_T4096", op="fp8_step", T=4096, N=2048, K=4096, dtype="bf16"),
    ]


WIDTHS = (64, 128, 256, 512, 768, 1024, 1408, 2048, 2816, 4096)  # hidden, intermediate and gate/up widths of the layers here, and narrow ones


def _ragged(rng, lo, hi):
    """A size spread over its logarithm that no tile divides."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n + (n > 64 and n % 64 == 0)))


def _width(rng, hi):
    return rng.choice([w for w in WIDTHS if w <= hi]) if rng.random() < 0.6 else _ragged(rng, 64, hi)


def draw(rng):
    op = rng.choice(["norm_pre", "norm_post", "route", "route", "fp8_linear", "fp8_linear", "fp8_step"])
    T = 2 ** rng.randint(0, 13) if rng.random() < 0.4 else _ragged(rng, 1, 8192)
    if op in ("norm_pre", "norm_post"):
        H = rng.choice([_width(rng, 4096), _width(rng, 4096), 8192, _ragged(rng, 4096, 8192)])
        while T * H > 8192 * 4096:
            T = max(1, T // 2)
        stream, block = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")])
        c = dict(op=op, T=T, H=H, stream=stream, block=block, dir=rng.choice(["fwd", "bwd"]))
        if op == "norm_post":
            c.update(post=rng.random() < 0.7, gate=rng.choice(["none", "token", "channel", "full"]), next=rng.random() < 0.6)
        return c
    if op == "route":
        E = rng.choice([8, 64, 128, 512, _ragged(rng, 8, 512), _ragged(rng, 8, 512)])
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 16)), dtype=rng.choice(["bf16", "f32", "f16"]), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.5, mask=rng.random() < 0.5, holes=rng.random() < 0.5, coef=rng.choice([0.001, 0.01, 1.0]),
                    dir=rng.choice(["fwd", "step"]))
    N, K = _width(rng, 4096), _width(rng, 4096)
    while op == "fp8_step" and T * N * K > 4096 * 2048 * 4096 or T * N * K > 8192 * 2816 * 4096:
        T = max(1, T // 2)
    return dict(op=op, T=T, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "f16"]))


def _blocks(n):
    return -(-n // BLK)


def work(c):
    T = c["T"]
    if c["op"] in ("norm_pre", "norm_post"):
        H, s, b = c["H"], SIZE[c["stream"]], SIZE[c["block"]]
        fwd, n = c["dir"] == "fwd", T * c["H"]
        if c["op"] == "norm_pre":
            per = s + b if fwd else b + s + s + s                         # x -> n;  dn, dres, x -> dx
            return {"bytes": n * per + 4 * H * (1 if fwd else 2) + 4 * T, "flops": n * (4 if fwd else 10)}
        gates = {"none": 0, "token": 4 * T, "channel": 4 * H, "full": b * n}[c["gate"]]
        vec = 4 * H * ((1 if c["post"] else 0) + (1 if c["next"] else 0))
        stats = 4 * T * ((1 if c["post"] else 0) + (1 if c["next"] else 0))
        if fwd:
            per = s + b + s + (b if c["next"] else 0)                     # r, y -> out, n
            return {"bytes": n * per + gates + vec + stats, "flops": n * 10}
        per = s + b + s + b + ((b + s) if c["next"] else 0)               # dout, y [, dn, out] -> dr, dy
        return {"bytes": n * per + 2 * gates + 2 * vec + stats, "flops": n * 22}
    if c["op"] == "route":
        E, k, s = c["E"], c["k"], SIZE[c["dtype"]]
        some = T * (8 * k + 4) + (T if c["mask"] else 0) + (4 * E if c["bias"] else 0) + (8 * E if c["coef"] else 0)
        if c["dir"] == "fwd":
            return {"bytes": T * E * s + some, "flops": T * E * 6}
        # the step reads the logits again: the loss's gradient needs the counts of all tokens
        return {"bytes": 3 * T * E * s + 2 * some + 4 * T * k, "flops": T * E * 12}
    N, K, s = c["N"], c["K"], SIZE[c["dtype"]]
    if c["op"] == "fp8_linear":
        return {"bytes": T * K * s + N * K + 4 * _blocks(N) * _blocks(K) + T * N * s, "flops": 2.0 * T * N * K}
    return {"bytes": T * K * s + N * K * s + T * N * s + T * N * s + T * K * s + 4 * N * K, "flops": 6.0 * T * N * K}


# ------------------------------------------------------------------ inputs

def _rms(x):
    return torch.rsqrt(x.float().square().mean(-1) + EPS)


def _block_scale(amax):
    """(what a block's values are multiplied by, what its codes are multiplied by); both are true divisions: a number over a
    tensor would be taken as the tensor's rounded reciprocal, which moves codes that lie between two values."""
    amax = amax.clamp(min=TINY)
    top = torch.full_like(amax, FP8_MAX)
    return top / amax, amax / top


def prepare(c, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))

    def normal(*shape, scale=1.0, type="f32"):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(TYPES[type])

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEVICE)

    s, T = {"case": dict(c)}, c["T"]
    if c["op"] == "norm_pre":
        H = c["H"]
        # a residual stream: rows of unlike sizes, a few channels far larger than the rest
        s["x"] = (normal(T, H) * (0.5 + 2.0 * uniform(T, 1)) * (1.0 + 10.0 * (uniform(H) < 0.01).float())).to(TYPES[c["stream"]])
        s["w"] = 1.0 + normal(H, scale=0.1)
        if c["dir"] == "bwd":
            s["dn"], s["dres"] = normal(T, H, type=c["block"]), normal(T, H, type=c["stream"])
            s["rstd"] = _rms(s["x"])
        return s
    if c["op"] == "norm_post":
        H = c["H"]
        s["y"] = normal(T, H, scale=0.3, type=c["block"])
        s["w"] = 1.0 + normal(H, scale=0.1) if c["post"] else None
        s["w_next"] = 1.0 + normal(H, scale=0.1) if c["next"] else None
        s["alpha"] = 0.7
        s["gate"] = {"none": None, "token": uniform(T), "channel": 1.0 + normal(H, scale=0.2), "full": uniform(T, H).to(TYPES[c["block"]])}[c["gate"]]
        stream = normal(T, H) * (0.5 + 2.0 * uniform(T, 1))
        if c["dir"] == "fwd":
            s["r"] = stream.to(TYPES[c["stream"]])
            return s
        s["dout"] = normal(T, H, type=c["stream"])
        s["rstd"] = _rms(s["y"]) if c["post"] else None
        s["out"] = s["dn"] = s["rstd_next"] = None
        if c["next"]:
            s["out"], s["dn"] = stream.to(TYPES[c["stream"]]), normal(T, H, type=c["block"])
            s["rstd_next"] = _rms(s["out"])
        return s
    if c["op"] == "route":
        E, k = c["E"], c["k"]
        lg = normal(T, E, scale=1.5) + normal(E, scale=0.5)  # some experts are liked by all tokens
        if c["holes"]:
            lg = lg.masked_fill(uniform(E) < 0.1, -math.inf).masked_fill(uniform(T, 1) < 0.02, -math.inf)
        s["logits"] = lg.to(TYPES[c["dtype"]])
        s["bias"] = normal(E, scale=0.1) if c["bias"] else None
        s["mask"] = uniform(T) < 0.9 if c["mask"] else None
        if c["dir"] == "step":
            s["dw"], s["dloss"] = normal(T, k, scale=0.01), 0.5 + uniform(1)
        return s
    N, K = c["N"], c["K"]
    # activations with a few channels far larger than the rest
    s["x"] = (normal(T, K) * (1.0 + 10.0 * (uniform(K) < 0.01).float())).to(TYPES[c["dtype"]])
    w = normal(N, K, scale=K ** -0.5)
    if c["op"] == "fp8_linear":
        # the weight as a checkpoint holds it: E4M3 codes, one scale for each 128 x 128 block
        pad = torch.zeros(_blocks(N) * BLK, _blocks(K) * BLK, device=DEVICE)
        pad[:N, :K] = w
        inv, s["w_s"] = _block_scale(pad.view(_blocks(N), BLK, _blocks(K), BLK).abs().amax((1, 3)))
        inv = inv.repeat_interleave(BLK, 0).repeat_interleave(BLK, 1)
        codes = torch.zeros(N, -(-K // 16) * 16, device=DEVICE)  # rows start on 16-byte boundaries
        codes[:, :K] = (pad * inv).clamp(-FP8_MAX, FP8_MAX)[:N, :K]
        s["w_q"] = codes.to(torch.float8_e4m3fn)[:, :K]
        return s
    s["w"], s["dy"] = w.to(TYPES[c["dtype"]]), normal(T, N, scale=0.05, type=c["dtype"])
    return s


# ------------------------------------------------------------------ the plain forms

def _norm_bwd(dn, x, rstd, w):
    """Gradients of n = x * rstd * w with rstd = rsqrt(mean(x^2) + eps)."""
    xhat = x * rstd[:, None]
    dxhat = dn * w
    return rstd[:, None] * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True)), (dn * xhat).sum(0)


def _plain_norm_pre(s):
    c, x = s["case"], s["x"].float()
    if c["dir"] == "fwd":
        rstd = _rms(s["x"])
        return [(x * rstd[:, None] * s["w"]).to(TYPES[c["block"]]), rstd]
    dx, dw = _norm_bwd(s["dn"].float(), x, s["rstd"], s["w"])
    return [(dx + s["dres"].float()).to(TYPES[c["stream"]]), dw]


def _wide_gate(s):
    c = s["case"]
    if c["gate"] == "none":
        return 1.0
    return s["gate"][:, None] if c["gate"] == "token" else s["gate"].float()


def _plain_norm_post(s):
    c, y = s["case"], s["y"].float()
    st, bt, g, alpha = TYPES[c["stream"]], TYPES[c["block"]], _wide_gate(s), s["alpha"]
    if c["dir"] == "fwd":
        rstd, z = None, y
        if c["post"]:
            rstd = _rms(y)
            z = y * rstd[:, None] * s["w"]
        out = s["r"].float() + alpha * g * z
        n = rstd_next = None
        if c["next"]:
            rstd_next = _rms(out)
            n = (out * rstd_next[:, None] * s["w_next"]).to(bt)
        return [out.to(st), n, rstd, rstd_next]
    d, dw_next = s["dout"].float(), None
    if c["next"]:
        through, dw_next = _norm_bwd(s["dn"].float(), s["out"].float(), s["rstd_next"], s["w_next"])
        d = d + through
    z = y * s["rstd"][:, None] * s["w"] if c["post"] else y
    dgate = alpha * d * z
    dgate = {"none": None, "token": dgate.sum(1), "channel": dgate.sum(0), "full": dgate.to(bt)}[c["gate"]]
    dy, dw = alpha * g * d, None
    if c["post"]:
        dy, dw = _norm_bwd(dy, y, s["rstd"], s["w"])
    return [d.to(st), dy.to(bt), dw, dgate, dw_next]


def _plain_route(s):
    c, lg = s["case"], s["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    valid = (lg > -math.inf).any(-1)
    if s["mask"] is not None:
        valid = valid & s["mask"]
    score = lg if s["bias"] is None else lg + s["bias"]
    top, ids = torch.sort(score, dim=-1, descending=True, stable=True)  # equal scores: the lowest expert first
    top, ids = top[:, :k], ids[:, :k]
    there = (top > -math.inf) & valid[:, None]
    high = torch.where(valid, lg.amax(-1), 0.0)
    e = torch.where(valid[:, None], torch.exp(lg - high[:, None]), 0.0)
    total = e.sum(-1)
    p = e / torch.where(valid, total, 1.0)[:, None]
    lse = torch.where(valid, high + torch.log(total), -math.inf)
    chosen = torch.where(there, lg.gather(1, ids), -math.inf)
    if c["renorm"]:
        best = torch.where(valid, chosen.amax(-1), 0.0)
        w = torch.exp(chosen - best[:, None])
        w = w / torch.where(valid, w.sum(-1), 1.0)[:, None]
    else:
        w = torch.where(there, p.gather(1, ids), 0.0)
    ids = torch.where(there, ids, -1)
    out = {"ids": ids.int(), "w": w, "lse": lse}
    counts = (ids[:, :, None] == torch.arange(E, device=ids.device)).sum((0, 1)) if T * k * E < 1 << 22 else torch.bincount(ids.flatten() + 1, minlength=E + 1)[1:]
    n_valid = valid.sum()
    if c["coef"]:
        share, mean = counts / (n_valid * k).clamp(min=1), p.sum(0) / n_valid.clamp(min=1)
        out.update(counts=torch.cat([counts, n_valid[None]]).int(), probs=mean, loss=(c["coef"] * E * (share * mean).sum())[None])
    if c["dir"] == "fwd":
        return out
    dl = torch.zeros_like(lg)
    wdw = w * s["dw"]
    if c["renorm"]:
        dl.scatter_add_(1, ids.clamp(min=0).long(), wdw - w * wdw.sum(-1, keepdim=True))
        dp = torch.zeros_like(p)
    else:
        dl.scatter_add_(1, ids.clamp(min=0).long(), wdw)
        dp = -wdw.sum(-1, keepdim=True).expand_as(p)
    if c["coef"]:
        a = s["dloss"] * c["coef"] * E * share / n_valid.clamp(min=1)
        dp = dp + a - (p * a).sum(-1, keepdim=True)
    out["dlogits"] = (dl + p * dp).to(s["logits"].dtype)
    return out


def _plain_rows(x):
    """What 32-bit rows stand for once they are E4M3 codes with one scale for each 128 values of a row."""
    T, K = x.shape
    pad = torch.nn.functional.pad(x, (0, _blocks(K) * BLK - K)).view(T, -1, BLK)
    inv, scale = _block_scale(pad.abs().amax(-1, keepdim=True))
    q = (pad * inv).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).float()
    return (q * scale).reshape(T, -1)[:, :K]


def _plain_weight(w):
    N, K = w.shape
    pad = torch.nn.functional.pad(w, (0, _blocks(K) * BLK - K, 0, _blocks(N) * BLK - N)).view(_blocks(N), BLK, _blocks(K), BLK)
    inv, scale = _block_scale(pad.abs().amax((1, 3), keepdim=True))
    q = (pad * inv).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).float()
    return (q * scale).reshape(_blocks(N) * BLK, -1)[:N, :K]


def _plain_linear(s):
    N, K = s["w_q"].shape
    w = s["w_q"].float() * s["w_s"].repeat_interleave(BLK, 0)[:N].repeat_interleave(BLK, 1)[:, :K]
    return [(_plain_rows(s["x"].float()) @ w.t()).to(s["x"].dtype)]


def _plain_step(s):
    x, w, dy = s["x"].float(), _plain_weight(s["w"].float()), s["dy"].float()
    y = _plain_rows(x) @ w.t()
    dx = _plain_rows(dy) @ w
    dw = _plain_rows(dy.t()) @ _plain_rows(x.t()).t()
    return [y.to(s["x"].dtype), dx.to(s["x"].dtype), dw]


PLAIN = {"norm_pre": _plain_norm_pre, "norm_post": _plain_norm_post, "route": _plain_route, "fp8_linear": _plain_linear, "fp8_step": _plain_step}


# ------------------------------------------------------------------ the framework's calls

def _own_run(s):
    from quantized_mixture_experts_moe_gb300 import binding as qb

    c = s["case"]
    if c["op"] == "norm_pre":
        if c["dir"] == "fwd":
            return list(qb.norm_pre(s["x"], s["w"], eps=EPS, out_dtype=TYPES[c["block"]]))
        return list(qb.norm_pre_backward(s["dn"], s["x"], s["rstd"], s["w"], dres=s["dres"]))
    if c["op"] == "norm_post":
        if c["dir"] == "fwd":
            return list(qb.norm_post(s["r"], s["y"], w=s["w"], gate=s["gate"], alpha=s["alpha"], w_next=s["w_next"], eps=EPS))
        return list(qb.norm_post_backward(s["dout"], s["y"], w=s["w"], rstd=s["rstd"], gate=s["gate"], alpha=s["alpha"],
                                          dn=s["dn"], out=s["out"], w_next=s["w_next"], rstd_next=s["rstd_next"]))
    if c["op"] == "route":
        r = qb.route_topk(s["logits"], c["k"], bias=s["bias"], mask=s["mask"], renorm=c["renorm"], coef=c["coef"] or None)
        out = {"ids": r.ids, "w": r.w, "lse": r.lse}
        if c["coef"]:
            out.update(counts=r.counts, probs=r.probs, loss=r.loss)
        if c["dir"] == "step":
            out["dlogits"] = qb.route_topk_backward(s["logits"], r, dw=s["dw"], dloss=s["dloss"])
        return out
    if c["op"] == "fp8_linear":
        return [qb.fp8_linear(s["x"], s["w_q"], s["w_s"])]
    x, w, dy = s["x"], s["w"], s["dy"]
    w_q, w_s, wt_q = qb.fp8_quant_blocks(w, transposed=True)
    y = qb.fp8_linear(x, w_q, w_s)
    dx, dw = qb.fp8_linear_backward(dy, x, wt_q, w_s)
    return [y, dx, dw]


def run(s):
    return _own_run(s) if own else PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _leaf(t):
    return None if t is None else t.double().requires_grad_(True)


def _exact_norm(x, w):
    rstd = 1.0 / torch.sqrt((x * x).sum(-1) / x.shape[-1] + EPS)
    return x * rstd.unsqueeze(1) * w, rstd


def _exact_fp8(x, tall):
    """What blocks of `tall` x 128 values stand for once they are E4M3 codes.  The definition forms a block's factor and each
    value's product with it in 32 bits, so that a code is the same wherever it is made; all else here is in 64 bits."""
    R, C = x.shape
    out = torch.zeros(-(-R // tall) * tall, _blocks(C) * BLK, device=x.device)
    out[:R, :C] = x.float()
    v = out.reshape(out.shape[0] // tall, tall, out.shape[1] // BLK, BLK)
    top = torch.clamp(v.abs().max(3).values.max(1).values, min=TINY)[:, None, :, None]
    code = torch.clamp(v * torch.div(torch.full_like(top, FP8_MAX), top), -FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return (code.double() * (top.double() / FP8_MAX)).reshape(out.shape)[:R, :C]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_pre":
        x, w = _leaf(s["x"]), _leaf(s["w"])
        n, rstd = _exact_norm(x, w)
        if c["dir"] == "fwd":
            return [n.detach(), rstd.detach()]
        dx, dw = torch.autograd.grad(n, (x, w), s["dn"].double())
        return [dx + s["dres"].double(), dw]
    if c["op"] == "norm_post":
        y, w, w_next, gate = _leaf(s["y"]), _leaf(s["w"]), _leaf(s["w_next"]), _leaf(s["gate"])
        z, rstd = _exact_norm(y, w) if c["post"] else (y, None)
        add = s["alpha"] * (z if gate is None else gate.unsqueeze(1) * z if c["gate"] == "token" else gate * z)
        if c["dir"] == "fwd":
            out = s["r"].double() + add
            n, rstd_next = _exact_norm(out, w_next) if c["next"] else (None, None)
            return [None if t is None else t.detach() for t in (out, n, rstd, rstd_next)]
        d, dw_next = s["dout"].double(), None
        if c["next"]:
            out = _leaf(s["out"])
            through, dw_next = torch.autograd.grad(_exact_norm(out, w_next)[0], (out, w_next), s["dn"].double())
            d = d + through
        asked = [t for t in (y, w, gate) if t is not None]
        got = iter(torch.autograd.grad(add, asked, d))
        dy = next(got)
        return [d, dy, None if w is None else next(got), None if gate is None else next(got), dw_next]
    if c["op"] == "route":
        lg = _leaf(s["logits"])
        T, E, k = c["T"], c["E"], c["k"]
        # the selection goes by the 32-bit sum of logit and bias
        score = s["logits"].float() + (0 if s["bias"] is None else s["bias"])
        live = torch.isfinite(score).any(1) & (torch.ones(T, dtype=torch.bool, device=lg.device) if s["mask"] is None else s["mask"])
        ids = torch.argsort(-score, dim=1, stable=True)[:, :k]
        on = torch.isfinite(score.gather(1, ids)) & live[:, None]
        safe = lg.masked_fill(~live[:, None], 0.0)
        lse = torch.logsumexp(safe, 1)
        p = torch.exp(safe - lse[:, None]) * live[:, None]
        if c["renorm"]:
            picked = safe.gather(1, ids).masked_fill(~on & live[:, None], -math.inf)
            w = torch.softmax(picked, 1) * on
        else:
            w = p.gather(1, ids) * on
        ids = ids.masked_fill(~on, -1)
        out = {"ids": ids.int(), "w": w.detach(), "lse": lse.detach().masked_fill(~live, -math.inf)}
        total, grad = 0.0, None
        if c["coef"]:
            flat = ids[on]
            counts = torch.zeros(E, dtype=torch.int64, device=lg.device).index_add_(0, flat, torch.ones_like(flat))
            n = int(live.sum())
            probs = p.sum(0) / max(n, 1)
            loss = c["coef"] * E * (counts.double() / max(n * k, 1) * probs).sum()
            out.update(counts=torch.cat([counts, counts.new_tensor([n])]).int(), probs=probs.detach(), loss=loss.detach()[None])
            total = loss * s["dloss"].double().item() if c["dir"] == "step" else 0.0
        if c["dir"] == "step":
            total = total + (w * s["dw"].double()).sum()
            out["dlogits"] = torch.nan_to_num(torch.autograd.grad(total, lg)[0])
        return out
    if c["op"] == "fp8_linear":
        N, K = s["w_q"].shape
        at_n, at_k = torch.arange(N, device=DEVICE) // BLK, torch.arange(K, device=DEVICE) // BLK
        w = s["w_q"].double() * s["w_s"].double()[at_n][:, at_k]
        return [_exact_fp8(s["x"], 1) @ w.t()]
    x, w, dy = s["x"], _exact_fp8(s["w"], BLK), s["dy"]
    return [_exact_fp8(x, 1) @ w.t(), _exact_fp8(dy, 1) @ w, _exact_fp8(dy.t().contiguous(), 1) @ _exact_fp8(x.t().contiguous(), 1).t()]
