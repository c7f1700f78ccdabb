"""Plain 64-bit forms of the experts' products, SwiGLU, the weighted sum and the 4-bit products, for the tests: torch, written
from the definitions in include/qmoe.h, with bounds on what fp32 sums may be off by."""

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=torch.float64)


def sums(length):
    """Roundings of a tensor-core sum of `length` products, each at most 2^-23 of the sum of magnitudes: one for each 16 values,
    and a few for how the products of a step are aligned."""
    return (length / 16 + 8) * 2.0 ** -23


def spans(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def gather(x, pairs, k):
    """x[pairs // k], rows of zeros where a pair is not in x."""
    if pairs is None:
        return x
    t = torch.div(pairs.long(), k, rounding_mode="floor")
    there = (pairs >= 0) & (t < x.shape[0])
    return torch.where(there[:, None], x[t.clamp(0, max(x.shape[0] - 1, 0))], torch.zeros((), dtype=x.dtype))


def linear(x, w, offsets):
    """(y, its slack)."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    m = torch.zeros_like(y)
    for e, a, b in spans(offsets):
        y[a:b] = x[a:b] @ w[e].t()
        m[a:b] = x[a:b].abs() @ w[e].abs().t()
    return y, m * sums(x.shape[1])


def linear_dx(dy, w, offsets):
    return linear(dy, w.transpose(1, 2), offsets)


def linear_dw(dy, x, offsets):
    E = offsets.numel() - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    m = torch.zeros_like(dw)
    for e, a, b in spans(offsets):
        dw[e] = dy[a:b].t() @ x[a:b]
        m[e] = dy[a:b].abs().t() @ x[a:b].abs() * sums(b - a)
    return dw, m


def swiglu(gu):
    g, u = gu.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def combine(y, w, pair_slot):
    T, k = pair_slot.shape
    out = torch.zeros(T, y.shape[1], dtype=y.dtype)
    for j in range(k):
        s = pair_slot[:, j].long()
        on = ((s >= 0) & (s < y.shape[0])).to(y.dtype)
        f = on if w is None else on * w[:, j]
        out = out + f[:, None] * y[s.clamp(0, y.shape[0] - 1)]
    return out


def codes4(q, s):
    """64-bit weights of packed 4-bit codes [..., K / 2] and their scales."""
    n = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1).long()
    if s.dtype == torch.float16:
        v, f = (n - 8).double(), s.double()
    else:
        v, f = E2M1[n], torch.exp2(s.double() - 127)
    return v * f.repeat_interleave(v.shape[-1] // f.shape[-1], -1)


def w4_slack(x, w, s, K):
    """Bound on the fp32 sums of y = x w^T: for int4 a group's sum passes through values up to 31 + 24 scales."""
    group = w.shape[-1] // s.shape[-1]
    f = s.double() if s.dtype == torch.float16 else torch.exp2(s.double() - 127)
    through = 55.0 if s.dtype == torch.float16 else 6.0
    return 2.0 ** -23 * (12 * through * (x.abs() @ f.repeat_interleave(group, -1).t()) + (K / 256 + 16) * (x.abs() @ w.abs().t()))
