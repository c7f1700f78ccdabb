"""Plain 64-bit forms of the operators around the experts (norms, routing, FP8 products), for the tests: torch on the CPU,
written from the definitions in include/qmoe.h."""

import math

import torch

ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff: 24, 8 and 11 significant bits
LEAST = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}                # absolute, among subnormals


def close(got, ref, slack, what=""):
    """|got - ref| <= one rounding of got's type + slack (fp32 arithmetic), element by element."""
    ref = torch.as_tensor(ref).double()
    diff = (got.detach().cpu().double() - ref).abs()
    bound = ROUND[got.dtype] * 1.01 * (ref.abs() + slack) + LEAST[got.dtype] + slack
    bad = ~(diff <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((diff / bound.clamp(min=1e-300)).max()):.3g} of the bound"


def norm(x, w, eps):
    rstd = 1.0 / torch.sqrt(x.square().mean(-1) + eps)
    return x * rstd[:, None] * w, rstd


def post(r, y, w, gate, alpha, w_next, eps):
    """(out, n) with 64-bit inputs; gate already of a shape that broadcasts to [T, H]."""
    z = y if w is None else norm(y, w, eps)[0]
    out = r + alpha * (z if gate is None else gate * z)
    return out, None if w_next is None else norm(out, w_next, eps)[0]


def route(logits, k, bias, mask, renorm, scale, coef):
    """dict(ids, w, lse, counts, probs, loss, p); differentiable in `logits` (64 bits, no NaN or +inf)."""
    T, E = logits.shape
    live = (logits > -math.inf).any(1)
    if mask is not None:
        live = live & mask
    score = logits.detach().float() + (0 if bias is None else bias)
    ids = torch.argsort(-score, dim=1, stable=True)[:, :k]
    on = (score.gather(1, ids) > -math.inf) & live[:, None]
    safe = torch.where(live[:, None], logits, torch.zeros_like(logits))
    lse = torch.logsumexp(safe, 1)
    p = torch.softmax(safe, 1) * live[:, None]  # not exp(safe - lse): lse loses log(E) beside a mask's lowest value
    if renorm:
        w = scale * torch.softmax(torch.where(on | ~live[:, None], safe.gather(1, ids), torch.full((), -math.inf).double()), 1) * on
    else:
        w = scale * p.gather(1, ids) * on
    w = torch.where(on, w, torch.zeros_like(w))
    flat = ids[on]
    counts = torch.bincount(flat, minlength=E)[:E]
    n = int(live.sum())
    probs = p.sum(0) / max(n, 1)
    loss = coef * E * (counts.double() / max(n * k, 1) * probs).sum()
    return dict(ids=torch.where(on, ids, torch.full_like(ids, -1)).int(), w=w, lse=torch.where(live, lse, torch.full((), -math.inf).double()),
                counts=torch.cat([counts, torch.tensor([n])]).int(), probs=probs, loss=loss, p=p)


def quant(x, tall):
    """(codes float8_e4m3fn [R, C], scales fp32) of blocks of `tall` x 128 values, by the fp32 steps of the definition."""
    R, C = x.shape
    rb, cb = -(-R // tall), -(-C // 128)
    pad = torch.zeros(rb * tall, cb * 128)
    pad[:R, :C] = x.float()
    v = pad.view(rb, tall, cb, 128)
    amax = v.abs().amax((1, 3)).clamp(min=2.0 ** -100)
    top = torch.full_like(amax, 448.0)
    q = (v * (top / amax)[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(rb * tall, cb * 128)[:R, :C], amax / top


def dequant(q, s):
    """64-bit values of codes [R, C] with scales [R or ceil(R / 128), ceil(C / 128)]."""
    R, C = q.shape
    tall = 1 if s.shape[0] == R else 128
    return q.double() * s.double()[torch.arange(R) // tall][:, torch.arange(C) // 128]


def product(a, b):
    """(a b^T, the bound on fp32 sums of it): each block of 128 is summed in four steps and carried on in a fifth."""
    blocks = -(-a.shape[1] // 128)
    return a @ b.t(), (a.abs() @ b.abs().t()) * (5 * blocks + 8) * 2.0 ** -23
