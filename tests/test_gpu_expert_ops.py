"""GPU tests of the experts' products, SwiGLU, the weighted sum and the 4-bit products against plain 64-bit forms.  Tolerances:
one rounding of the output's type, and fp32 sums bounded by the number of their roundings (tests/expert_ref.py)."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from tests import expert_ref as ref
from tests.block_ref import ROUND, close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def offsets_of(counts):
    return torch.tensor([0] + counts).cumsum(0).int()


def status():
    return int(qb.status_word("cuda").item())


# ------------------------------------------------------------------ grouped products

# counts of the experts' rows, rows of none behind them, N, K
SHAPES = [
    ([1], 0, 8, 8),
    ([0, 1, 0], 0, 64, 64),
    ([1, 1, 2, 0, 1], 3, 128, 192),
    ([3, 0, 5, 16], 0, 136, 72),
    ([17, 15, 33, 0], 5, 200, 264),
    ([100, 40, 0, 96], 1, 264, 136),
    ([128, 129, 127], 0, 320, 64),
    ([256, 257, 0, 255], 7, 128, 128),
    ([300, 700], 0, 72, 520),
    ([1000], 0, 256, 192),
    ([0, 0, 0], 4, 64, 64),
    ([512, 1, 0, 63, 64, 65], 0, 392, 328),
    ([2] * 70, 0, 64, 64),
]
ODD = [([5, 0, 3], 2, 7, 9), ([40, 21, 1], 0, 131, 65), ([300, 20], 3, 129, 127), ([260, 0, 33], 0, 66, 67), ([3, 9], 0, 1, 1)]


def routed(g, counts, extra, K, dtype, gather):
    """(x, pairs, k, offsets, rows in expert order in 64 bits)"""
    P, offsets = sum(counts) + extra, offsets_of(counts)
    if not gather:
        x = randn(g, P, K, dtype=dtype)
        return x, None, 1, offsets, x.double()
    k = 3
    T = -(-P // k)
    x = randn(g, T, K, dtype=dtype)
    pairs = torch.randperm(T * k, generator=g)[:P].int()
    pairs[sum(counts):] = -1
    return x, pairs, k, offsets, ref.gather(x.double(), pairs, k)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES + ODD)))
def test_expert_linear(i, shape, gather):
    counts, extra, N, K = shape
    dtype = (BF16, F16)[i % 2]
    g = gen(1000 + i)
    x, pairs, k, offsets, rows = routed(g, counts, extra, K, dtype, gather)
    w = randn(g, len(counts), N, K, dtype=dtype, scale=K ** -0.5)
    want, slack = ref.linear(rows, w.double(), offsets)
    for out in (None, F32):
        y = qb.expert_linear(dev(x), dev(w), dev(offsets), pairs=dev(pairs), k=k, out_dtype=out)
        assert y.dtype == (out or dtype)
        close(y, want, slack, f"y {out}")
    assert status() == 0


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES + ODD)))
def test_expert_linear_backward(i, shape, gather):
    counts, extra, N, K = shape
    dtype = (F16, BF16)[i % 2]
    g = gen(2000 + i)
    x, pairs, k, offsets, rows = routed(g, counts, extra, K, dtype, gather)
    w, dy = randn(g, len(counts), N, K, dtype=dtype, scale=K ** -0.5), randn(g, sum(counts) + extra, N, dtype=dtype)
    dx, dw = qb.expert_linear_backward(dev(dy), dev(x), dev(w), dev(offsets), pairs=dev(pairs), k=k)
    assert dx.dtype == dtype and dw.dtype == F32
    close(dx, *ref.linear_dx(dy.double(), w.double(), offsets), "dx")
    wide, slack = ref.linear_dw(dy.double(), rows, offsets)
    close(dw, wide, slack, "dw")
    none, narrow = qb.expert_linear_backward(dev(dy), dev(x), dev(w), dev(offsets), pairs=dev(pairs), k=k, dw_dtype=dtype, need_dx=False)
    assert none is None and narrow.dtype == dtype
    close(narrow, wide, slack, "dw in 16 bits")
    # differences of the plain form along a random direction
    d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (rows, w)]
    f = lambda h: (ref.linear(rows + h * d[0], w.double() + h * d[1], offsets)[0] * dy.double()).sum()
    slope = float((f(1e-4) - f(-1e-4)) / 2e-4)
    own = float((dx.cpu().double() * d[0]).sum() + (dw.cpu().double() * d[1]).sum())
    size = float((dx.cpu().double() * d[0]).abs().sum() + (dw.cpu().double() * d[1]).abs().sum())
    assert abs(slope - own) <= size * (ROUND[dtype] + 1e-5) + 1e-6
    assert status() == 0


@pytest.mark.parametrize("E,most,steps", [(400, 92, 13), (700, 9, 5), (700, 9, 1), (310, 40, 3), (40, 3, 7)])
def test_expert_linear_many_odd(E, most, steps):
    """Several tiles a CTA, each of an odd number of steps of 64: no step may be taken for the one two rounds before it."""
    g = gen(50 + E + steps)
    counts = torch.randint(1, most + 1, (E,), generator=g).tolist()
    P, K, N, offsets = sum(counts), 64 * steps - 43, 64, offsets_of(counts)
    x, dx_of = randn(g, P, K, dtype=BF16), randn(g, P, K, dtype=BF16)
    w, wt = randn(g, E, N, K, dtype=BF16, scale=K ** -0.5), randn(g, E, K, N, dtype=BF16, scale=K ** -0.5)
    want, back = ref.linear(x.double(), w.double(), offsets), ref.linear_dx(dx_of.double(), wt.double(), offsets)
    args = [dev(t) for t in (x, w, dx_of, wt, offsets)]
    held = randn(g, P, N, dtype=BF16).cuda()
    for i in range(12):
        y = qb.expert_linear(args[0], args[1], args[4])
        dx, _ = qb.expert_linear_backward(args[2], held, args[3], args[4], need_dw=False)
        if i == 0:
            first = (y, dx)
        assert torch.equal(y, first[0]) and torch.equal(dx, first[1])
    close(first[0], *want, "y")
    close(first[1], *back, "dx")
    assert status() == 0


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 24), (0, 1)])
def test_expert_linear_strides(shift, pad):
    """Views: rows that start off the 16-byte boundaries, and rows with a stride."""
    counts, N, K = [20, 0, 75, 130], 72, 88
    g = gen(7 + shift)
    P, E, offsets = sum(counts), len(counts), offsets_of(counts)

    def view(*shape):
        base = randn(g, *shape[:-1], shape[-1] + shift + pad, dtype=BF16)
        return base.cuda()[..., shift:shift + shape[-1]], base[..., shift:shift + shape[-1]]

    (x, cx), (w, cw), (dy, cdy) = view(P, K), view(E, N, K), view(P, N)
    close(qb.expert_linear(x, w, dev(offsets)), *ref.linear(cx.double(), cw.double(), offsets), "y")
    dx, dw = qb.expert_linear_backward(dy, x, w, dev(offsets))
    close(dx, *ref.linear_dx(cdy.double(), cw.double(), offsets), "dx")
    close(dw, *ref.linear_dw(cdy.double(), cx.double(), offsets), "dw")
    every = w[1:3]
    close(qb.expert_linear(x[20:95], every, dev(offsets[1:4] - 20)), *ref.linear(cx.double()[20:95], cw.double()[1:3], offsets[1:4] - 20), "y of some experts")


def test_expert_linear_keeps_others_out():
    """Rows of another expert, and of none, may hold anything."""
    counts, N, K = [5, 40, 70, 0, 9], 136, 200
    g = gen(3)
    P, offsets = sum(counts) + 6, offsets_of(counts)
    x, w, dy = randn(g, P, K, dtype=F16), randn(g, 5, N, K, dtype=F16, scale=0.1), randn(g, P, N, dtype=F16)
    for e, a, b in ref.spans(offsets):
        if e % 2 == 0:
            x[a:b], dy[a:b], w[e] = float("nan"), float("inf"), float("nan")
    x[sum(counts):], dy[sum(counts):] = float("nan"), float("nan")
    y = qb.expert_linear(dev(x), dev(w), dev(offsets)).cpu()
    dx, dw = (t.cpu() for t in qb.expert_linear_backward(dev(dy), dev(x), dev(w), dev(offsets)))
    clean = lambda t: torch.nan_to_num(t.double(), nan=0.0, posinf=0.0, neginf=0.0)
    (ry, sy), (rx, sx), (rw, sw) = (ref.linear(clean(x), clean(w), offsets), ref.linear_dx(clean(dy), clean(w), offsets),
                                    ref.linear_dw(clean(dy), clean(x), offsets))
    a, b = 5, 45
    close(y[a:b], ry[a:b], sy[a:b], "y")
    close(dx[a:b], rx[a:b], sx[a:b], "dx")
    close(dw[1], rw[1], sw[1], "dw")
    assert (dw[3] == 0).all() and (y[sum(counts):] == 0).all() and (dx[sum(counts):] == 0).all()
    assert y[:5].isnan().all() and dw[0].isnan().all()


@pytest.mark.parametrize("offsets", [[0, 5, 3, 12], [0, 4, 40, 50], [-3, 2, 4, 12], [2, 4, 6, 12], [0, 12, 12, -1]])
def test_bad_offsets_are_reported(offsets):
    x, w = torch.ones(12, 64, device="cuda", dtype=BF16), torch.ones(3, 64, 64, device="cuda", dtype=BF16)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for f in (lambda s: qb.expert_linear(x, w, off, dev_status=s), lambda s: qb.expert_linear_backward(x, x, w, off, need_dw=False, dev_status=s),
              lambda s: qb.expert_linear_backward(x, x, w, off, need_dx=False, dev_status=s)):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        f(word)
        assert int(word.item()) == qb.DEV_BAD_OFFSETS


def test_bad_pairs_are_rows_of_zeros():
    g = gen(5)
    counts, k, T, K, N = [7, 30, 3], 4, 10, 72, 64
    offsets = offsets_of(counts)
    x, w, dy = randn(g, T, K, dtype=BF16), randn(g, 3, N, K, dtype=BF16, scale=0.1), randn(g, 40, N, dtype=BF16)
    pairs = torch.randperm(40, generator=g).int()
    pairs[[0, 9, 22, 38]] = torch.tensor([-1, 40, 2 ** 31 - 1, -2 ** 31]).int()
    rows = ref.gather(x.double(), pairs, k)
    close(qb.expert_linear(dev(x), dev(w), dev(offsets), pairs=dev(pairs), k=k), *ref.linear(rows, w.double(), offsets), "y")
    _, dw = qb.expert_linear_backward(dev(dy), dev(x), dev(w), dev(offsets), pairs=dev(pairs), k=k, need_dx=False)
    close(dw, *ref.linear_dw(dy.double(), rows, offsets), "dw")


def test_expert_linear_no_rows():
    w, off = torch.ones(2, 64, 64, device="cuda", dtype=BF16), torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    assert qb.expert_linear(x, w, off).shape == (0, 64)
    dx, dw = qb.expert_linear_backward(x, x, w, off)
    assert dx.shape == (0, 64) and dw.shape == (2, 64, 64) and (dw == 0).all()


def test_expert_linear_far_offsets():
    """Outputs and inputs past 2^31 elements."""
    P, N, K = 70_001, 32_768, 64
    x = torch.randn(P, K, device="cuda", dtype=F32).to(BF16)
    w = (torch.randn(2, N, K, device="cuda") * 0.1).to(BF16)
    off = torch.tensor([0, 35_000, P], dtype=torch.int32, device="cuda")
    y = qb.expert_linear(x, w, off)
    rows = torch.tensor([0, 34_999, 35_000, 65_535, 65_536, 65_537, P - 1])
    got = y[rows.cuda()].cpu()
    want = torch.stack([x[r].cpu().double() @ w[int(r >= 35_000)].cpu().double().t() for r in rows])
    size = torch.stack([x[r].cpu().double().abs() @ w[int(r >= 35_000)].cpu().double().abs().t() for r in rows])
    close(got, want, size * ref.sums(K), "y")
    _, dw = qb.expert_linear_backward(y, x, w, off, need_dx=False)
    ys, xs = y[35_000:, -256:].double(), x[35_000:].double()
    close(dw[1, -256:].cpu(), (ys.t() @ xs).cpu(), (ys.abs().t() @ xs.abs()).cpu() * ref.sums(35_001), "dw")


# ------------------------------------------------------------------ SwiGLU

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("i,size", list(enumerate([(1, 1), (3, 7), (8, 768), (65, 129), (33, 1408), (2, 4100), (1000, 64), (0, 8)])))
def test_swiglu(i, size, dtype):
    P, I = size
    g = gen(50 + i)
    gu, dh = randn(g, P, 2 * I, dtype=dtype, scale=3.0), randn(g, P, I, dtype=dtype)
    if P > 1:
        gu[0, :I] = torch.tensor([0.0, 60.0, -60.0, 1e-3])[torch.arange(I) % 4].to(dtype)
    h = qb.swiglu(dev(gu))
    leaf = gu.double().requires_grad_()
    want = ref.swiglu(leaf)
    # 1 + e^-v, its reciprocal, two products; the fast exponential is off by 2 ulp and 2^-23 |v| of its argument's rounding
    fast = 0.0 if dtype == F32 else 1.0
    v = gu[:, :I].double().abs()
    err = (10 + 2 * v + fast * 4) * U
    close(h, want.detach(), err * want.detach().abs() + 1e-38, "h")
    dgu, again = qb.swiglu_backward(dev(dh), dev(gu), h_too=True)
    assert torch.equal(again, h)
    grad, = torch.autograd.grad(want, leaf, dh.double())
    gd, ud, s = gu[:, :I].double(), gu[:, I:].double(), torch.sigmoid(gu[:, :I].double())
    size_g = (dh.double() * ud * s).abs() * (1 + gd.abs())
    close(dgu, grad, 2 * torch.cat([err * size_g, err * (dh.double() * gd * s).abs()], 1) + 1e-38, "dgu")
    assert qb.swiglu_backward(dev(dh), dev(gu))[1] is None
    if P:
        step = torch.randn(gu.shape, generator=g, dtype=torch.float64)
        f = lambda t: (ref.swiglu(gu.double() + t * step) * dh.double()).sum()
        slope, own = float((f(1e-5) - f(-1e-5)) / 2e-5), float((dgu.cpu().double() * step).sum())
        assert abs(slope - own) <= float((grad * step).abs().sum()) * (ROUND[dtype] + 1e-5) + 1e-6


def test_swiglu_strides():
    g = gen(8)
    base, dbase = randn(g, 20, 300, dtype=BF16), randn(g, 20, 150, dtype=BF16)
    for a, I in ((0, 128), (1, 100), (8, 64), (4, 33)):
        gu, dh = base[:, a:a + 2 * I], dbase[:, a:a + I]
        h = qb.swiglu(base.cuda()[:, a:a + 2 * I])
        assert torch.equal(h, qb.swiglu(gu.contiguous().cuda()))
        d, _ = qb.swiglu_backward(dbase.cuda()[:, a:a + I], base.cuda()[:, a:a + 2 * I])
        assert torch.equal(d, qb.swiglu_backward(dh.contiguous().cuda(), gu.contiguous().cuda())[0])


# ------------------------------------------------------------------ weighted sum

def slots(g, T, k, drop):
    P = T * k
    on = torch.rand(T, k, generator=g) >= drop
    n = int(on.sum())
    slot = torch.full((T, k), -1, dtype=torch.int32)
    slot[on] = torch.randperm(n, generator=g).int()
    return slot, torch.tensor([0, n // 2, n], dtype=torch.int32), P, n


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("i,size", list(enumerate([(1, 1, 1), (1, 8, 64), (5, 3, 7), (33, 10, 136), (7, 2, 2049), (70, 8, 1024), (3, 33, 4104)])))
def test_combine(i, size, drop, dtype):
    T, k, H = size
    g = gen(70 + i)
    slot, offsets, P, n = slots(g, T, k, drop)
    y, w, dout = randn(g, P, H, dtype=dtype), randn(g, T, k), randn(g, T, H, dtype=dtype)
    y[n:] = float("nan")  # rows that no pair names
    y64 = torch.nan_to_num(y.double())
    for weight in (w, None):
        want = ref.combine(y64, None if weight is None else weight.double(), slot)
        size_of = ref.combine(y64.abs(), None if weight is None else weight.double().abs(), slot)
        close(qb.combine(dev(y), dev(weight), dev(slot)), want, (k + 1) * U * size_of, "out")
        dy, dw = qb.combine_backward(dev(dout), dev(y), dev(weight), dev(slot), dev(offsets))
        ly, lw = y64.clone().requires_grad_(), w.double().requires_grad_()
        ry, rw = torch.autograd.grad(ref.combine(ly, lw if weight is not None else torch.ones_like(lw) + 0 * lw, slot), (ly, lw), dout.double())
        close(dy, ry, U * ry.abs(), "dy")
        assert (dy[n:] == 0).all()
        if weight is None:
            assert dw is None
        else:
            mag = torch.autograd.grad(ref.combine(y64.abs(), lw, slot), lw, dout.double().abs())[0]
            close(dw, rw, (H / 32 + 8) * U * mag, "dw")


def test_combine_out_of_range_slots():
    y = torch.ones(4, 64, device="cuda", dtype=BF16)
    slot = torch.tensor([[0, 4], [-7, 2 ** 31 - 1], [3, 1]], dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    assert torch.equal(qb.combine(y, w, slot)[:, 0].cpu(), torch.tensor([1.0, 0.0, 2.0]).to(BF16))
    dy, dw = qb.combine_backward(torch.ones(3, 64, device="cuda", dtype=BF16), y, w, slot, torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    assert torch.equal(dw.cpu(), torch.tensor([[64.0, 0.0], [0.0, 0.0], [64.0, 64.0]]))


def test_combine_strides():
    g = gen(9)
    slot, offsets, P, n = slots(g, 20, 4, 0.1)
    base, w = randn(g, P, 200, dtype=F16), randn(g, 20, 4)
    for a, H in ((0, 128), (1, 100), (8, 64), (3, 33)):
        y = base[:, a:a + H].contiguous().cuda()
        view = base.cuda()[:, a:a + H]
        assert torch.equal(qb.combine(view, w.cuda(), slot.cuda()), qb.combine(y, w.cuda(), slot.cuda()))
        dout = qb.combine(y, w.cuda(), slot.cuda())
        got, dw = qb.combine_backward(dout, view, w.cuda(), slot.cuda(), offsets.cuda())
        want, dw2 = qb.combine_backward(dout, y, w.cuda(), slot.cuda(), offsets.cuda())
        assert torch.equal(got, want)
        close(dw, dw2.cpu().double(), 0.01, "dw")  # the columns fall to other lanes


# ------------------------------------------------------------------ 4-bit products

def weights4(g, lead, N, K, format, group):
    q = torch.randint(0, 256, (*lead, N, K // 2), generator=g, dtype=torch.uint8)
    if format == "int4":
        return q, (0.005 + 0.015 * torch.rand(*lead, N, K // group, generator=g)).half()
    return q, torch.randint(115, 130, (*lead, N, K // 32), generator=g, dtype=torch.uint8)


FORMATS = [("int4", 32), ("int4", 64), ("int4", 128), ("mxfp4", 32)]


@pytest.mark.parametrize("format,group", FORMATS)
@pytest.mark.parametrize("T,N,K", [(1, 1, 128), (1, 2816, 2048), (2, 15, 256), (3, 16, 384), (7, 33, 640), (8, 129, 2176), (9, 64, 4096), (16, 100, 4224),
                                   (13, 40, 2048), (11, 17, 2304), (16, 48, 6144), (3, 24, 16384), (1, 24, 16384), (5, 20, 9216), (4, 70, 512), (2, 300, 768)])
def test_w4_linear(T, N, K, format, group):
    g = gen(T * 7 + N + K + group)
    dtype = (BF16, F16)[(T + N) % 2]
    x = randn(g, T, K, dtype=dtype)
    q, s = weights4(g, (), N, K, format, group)
    w = ref.codes4(q, s)
    for out in (None, F32):
        y = qb.w4_linear(dev(x), dev(q), dev(s), out_dtype=out)
        assert y.dtype == (out or dtype) and y.shape == (T, N)
        close(y, x.double() @ w.t(), ref.w4_slack(x.double(), w, s, K), "y")
    assert status() == 0


@pytest.mark.parametrize("format,group", FORMATS)
@pytest.mark.parametrize("T,N,K", [(17, 40, 2048), (32, 48, 6144), (33, 40, 128), (64, 129, 256), (200, 264, 640), (300, 7, 1152)])
def test_w4_linear_many(T, N, K, format, group):
    g = gen(T + N + K + group)
    dtype = (BF16, F16)[(T + N) % 2]
    x, dy = randn(g, T, K, dtype=dtype), randn(g, T, N, dtype=dtype)
    q, s = weights4(g, (), N, K, format, group)
    w = ref.codes4(q, s)
    # the weights are rounded to 16 bits once (E2M1 times a power of two is not rounded)
    r = (ROUND[dtype] * 1.01 if format == "int4" else 0.0)
    y = qb.w4_linear(dev(x), dev(q), dev(s))
    close(y, x.double() @ w.t(), (x.double().abs() @ w.abs().t()) * (ref.sums(K) + r), "y")
    dx = qb.w4_linear_backward(dev(dy), dev(q), dev(s))
    close(dx, dy.double() @ w, (dy.double().abs() @ w.abs()) * (ref.sums(N) + r), "dx")


@pytest.mark.parametrize("T,N,K", [(1, 40, 128), (4, 9, 256), (19, 64, 384)])
def test_w4_linear_backward_few(T, N, K):
    g = gen(T)
    q, s = weights4(g, (), N, K, "int4", 64)
    w, dy = ref.codes4(q, s), randn(g, T, N, dtype=F16)
    dx = qb.w4_linear_backward(dev(dy), dev(q), dev(s))
    close(dx, dy.double() @ w, (dy.double().abs() @ w.abs()) * (ref.sums(N) + ROUND[F16] * 1.01), "dx")


@pytest.mark.parametrize("format,group", FORMATS)
@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 128, 64, 256), (4, 10, 16, 33, 640), (3, 1, 5, 16, 4352), (40, 2, 4, 20, 128), (150, 2, 3, 20, 128), (64, 4, 30, 17, 256),
                                       (16, 8, 8, 40, 512), (33, 1, 1, 130, 1152), (5, 3, 9, 300, 384), (7, 6, 14, 24, 2304)])
def test_w4_experts(T, k, E, N, K, format, group):
    g = gen(T + k + E + group)
    dtype = (BF16, F16)[T % 2]
    x = randn(g, T, K, dtype=dtype)
    q, s = weights4(g, (E,), N, K, format, group)
    ids = torch.randint(0, E, (T, k), generator=g).int()
    ids[0, 0] = E if T % 2 else -1
    y = qb.w4_linear(dev(x), dev(q), dev(s), ids=dev(ids))
    assert y.shape == (T * k, N)
    w = ref.codes4(q, s)
    for p in range(T * k):
        e = int(ids.view(-1)[p])
        row = x[p // k].double()[None]
        if not 0 <= e < E:
            assert (y[p] == 0).all()
        else:
            close(y[p:p + 1], row @ w[e].t(), ref.w4_slack(row, w[e], s[e], K), f"pair {p}")


@pytest.mark.parametrize("format", ["int4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(1, 40, 96), (4, 24, 160), (7, 33, 32), (16, 17, 288), (20, 16, 96)])
def test_w4_linear_odd_groups(T, N, K, format):
    """Reductions of an odd number of groups: no two scales in one word, a last block that is short."""
    g = gen(T + K)
    x = randn(g, T, K, dtype=BF16)
    q, s = weights4(g, (), N, K, format, 32)
    w = ref.codes4(q, s)
    slack = ref.w4_slack(x.double(), w, s, K) if T <= 16 else (x.double().abs() @ w.abs().t()) * (ref.sums(K) + ROUND[BF16] * 1.01)
    close(qb.w4_linear(dev(x), dev(q), dev(s)), x.double() @ w.t(), slack, "y")


def test_w4_linear_special_values():
    """Extreme scales, and NaN and infinities that stay in their token."""
    g = gen(40)
    x = randn(g, 3, 128, dtype=F16)
    q, s = weights4(g, (), 20, 128, "mxfp4", 32)
    s[0, 0], s[1, 1], s[2, :] = 0, 30, 140
    w = ref.codes4(q, s)
    close(qb.w4_linear(dev(x), dev(q), dev(s), out_dtype=F32), x.double() @ w.t(), ref.w4_slack(x.double(), w, s, 128), "y")
    s[5, 2] = 255
    x[1, 7], x[2, 100] = float("inf"), float("nan")
    for scales in (s, (s.float() * 0 + 0.01).half()):
        y = qb.w4_linear(dev(x), dev(q), dev(scales), out_dtype=F32).cpu()
        assert not y[1:].isfinite().any() or scales.dtype == torch.uint8
        assert y[2].isnan().all() and y[0].isfinite().sum() >= 19


def test_w4_linear_strides():
    g = gen(4)
    q, s = weights4(g, (), 40, 256, "int4", 32)
    base = randn(g, 50, 300, dtype=BF16)
    for rows in (1, 6, 50):
        for a in (0, 1, 8, 13):
            x = base[:rows, a:a + 256]
            view = base.cuda()[:rows, a:a + 256]
            assert torch.equal(qb.w4_linear(view, dev(q), dev(s)), qb.w4_linear(x.contiguous().cuda(), dev(q), dev(s)))


# ------------------------------------------------------------------ together

def step(x, ids, wr, w1, w2, dout):
    """A training step of the routed experts: output, gradients of x, the routing weights and both expert weights."""
    T, k = ids.shape
    offsets, pairs, pair_slot = qb.align_sort(ids, w1.shape[0])
    gu = qb.expert_linear(x, w1, offsets, pairs=pairs, k=k)
    h = qb.swiglu(gu)
    y = qb.expert_linear(h, w2, offsets)
    out = qb.combine(y, wr, pair_slot)
    dy, dwr = qb.combine_backward(dout, y, wr, pair_slot, offsets)
    dh, dw2 = qb.expert_linear_backward(dy, h, w2, offsets)
    dgu, _ = qb.swiglu_backward(dh, gu)
    dxs, dw1 = qb.expert_linear_backward(dgu, x, w1, offsets, pairs=pairs, k=k)
    return out, qb.combine(dxs, None, pair_slot), dwr, dw1, dw2


def plain_step(x, ids, wr, w1, w2, dout):
    x, wr, w1, w2 = (t.double().requires_grad_() for t in (x, wr, w1, w2))
    out = torch.zeros(x.shape[0], w2.shape[1], dtype=torch.float64)
    rows = []
    for t in range(ids.shape[0]):
        r = torch.zeros(w2.shape[1], dtype=torch.float64)
        for j, e in enumerate(ids[t].tolist()):
            if 0 <= e < w1.shape[0]:
                r = r + wr[t, j] * (ref.swiglu((x[t] @ w1[e].t())[None])[0] @ w2[e].t())
        rows.append(r)
    out = torch.stack(rows)
    return [out.detach()] + list(torch.autograd.grad(out, (x, wr, w1, w2), dout.double()))


def layer(seed, T=37, k=3, E=6, H=136, I=72):
    g = gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[1, 2], ids[4] = -1, -1
    return (randn(g, T, H, dtype=BF16), ids, torch.softmax(randn(g, T, k), 1), randn(g, E, 2 * I, H, dtype=BF16, scale=H ** -0.5),
            randn(g, E, H, I, dtype=BF16, scale=I ** -0.5), randn(g, T, H, dtype=BF16))


def test_training_step():
    args = layer(1)
    got, want = step(*map(dev, args)), plain_step(*args)
    for name, a, b in zip(("out", "dx", "dwr", "dw1", "dw2"), got, want):
        # roundings to bf16 on the way, each at most 2^-8 of the value it rounds: 5 of them in out, 9 in a gradient
        rel = float((a.cpu().double() - b).norm() / b.norm())
        assert rel < 9 * 2.0 ** -8, (name, rel)
    assert status() == 0


def test_training_step_in_graphs():
    """Two captured steps of different inputs, replayed in turn, give what the calls give."""
    sets = [tuple(map(dev, layer(s, T=t))) for s, t in ((2, 20), (3, 61))]
    eager = [step(*a) for a in sets]
    words = [torch.zeros(1, dtype=torch.int32, device="cuda")]
    del words
    graphs = []
    for a in sets:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(*a)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*a)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, out), want in zip(graphs, eager):
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_streams():
    """Calls on two streams at once, and on the stream that a call names."""
    a, b = tuple(map(dev, layer(5, T=50))), tuple(map(dev, layer(6, T=70)))
    want = step(*a), step(*b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, args in zip(streams, (a, b)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(*args))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    offsets, pairs, _ = qb.align_sort(a[1], 6)
    torch.cuda.synchronize()
    y = qb.expert_linear(a[0], a[3], offsets, pairs=pairs, k=3, stream=streams[0])
    h = qb.swiglu(y, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(h, qb.swiglu(qb.expert_linear(a[0], a[3], offsets, pairs=pairs, k=3)))


def test_decode_with_4_bit_experts():
    """A token through its experts in 4 bits and a shared expert beside them, as the pieces are used in decoding."""
    g = gen(11)
    T, k, E, H, I = 2, 3, 8, 256, 128
    x, wr = randn(g, T, H, dtype=BF16), torch.softmax(randn(g, T, k), 1)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    (q1, s1), (q2, s2), (q3, s3), (q4, s4) = (weights4(g, lead, n, m, f, 32) for lead, n, m, f in (
        ((E,), 2 * I, H, "mxfp4"), ((E,), H, I, "int4"), ((), 2 * I, H, "int4"), ((), H, I, "mxfp4")))
    s1, s4 = s1 // 8 + 104, s4 // 8 + 104  # scales about 2^-8
    y = qb.w4_linear(qb.swiglu(qb.w4_linear(dev(x), dev(q1), dev(s1), ids=dev(ids))), dev(q2), dev(s2), ids=dev(ids.view(-1, 1)))
    slot = torch.arange(T * k, dtype=torch.int32).view(T, k)
    out = qb.combine(y, dev(wr), dev(slot)).float() + qb.w4_linear(qb.swiglu(qb.w4_linear(dev(x), dev(q3), dev(s3))), dev(q4), dev(s4)).float()
    w1, w2, w3, w4 = (ref.codes4(q, s) for q, s in ((q1, s1), (q2, s2), (q3, s3), (q4, s4)))
    X = x.double()
    want = ref.swiglu(X @ w3.t()) @ w4.t()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            want[t] += wr[t, j].double() * (ref.swiglu((X[t] @ w1[e].t())[None])[0] @ w2[e].t())
    assert float((out.cpu().double() - want).norm() / want.norm()) < 5 * 2.0 ** -8


def test_same_bits():
    args = tuple(map(dev, layer(9, T=200, E=6, H=264, I=136)))
    first = step(*args)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step(*args)))


def test_first_call_in_a_capture_is_refused_without_a_status():
    held = dict(qb._status_words)
    qb._status_words.clear()
    try:
        x, w, off = torch.ones(4, 64, device="cuda", dtype=BF16), torch.ones(1, 64, 64, device="cuda", dtype=BF16), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        qb.expert_linear(x, w, off, dev_status=word)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(qb.QmoeError):
                qb.expert_linear(x, w, off)
            y = qb.expert_linear(x, w, off, dev_status=word)
        graph.replay()
        torch.cuda.synchronize()
        assert (y == 64).all()
    finally:
        qb._status_words.update(held)


def test_trained_experts_example():
    """examples/moe_block.py's trained experts: gradients against the 64-bit step, with tokens that are not routed."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    x, ids, wr, _, _, dout = layer(21, T=30, k=3, E=5, H=128, I=64)
    experts = m.TrainedExperts(H=128, I=64, E=5, seed=2)
    out, kept = experts.forward(dev(x), dev(ids), dev(wr))
    got = (out,) + experts.backward(dev(dout), kept)
    want = plain_step(x, ids, wr, experts.w1.cpu(), experts.w2.cpu(), dout)
    for name, a, b in zip(("out", "dn", "dw", "dw1", "dw2"), got, want):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        assert rel < 9 * 2.0 ** -8, (name, rel)  # as in test_training_step
    assert status() == 0


# ------------------------------------------------------------------ what the binding refuses

def test_binding_refuses():
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    x, w = z(8, 64), z(2, 32, 64)
    for f in (lambda: qb.expert_linear(x, z(2, 32, 63), off), lambda: qb.expert_linear(x, w, off[:2]), lambda: qb.expert_linear(x, w.half(), off),
              lambda: qb.expert_linear(x.float(), w.float(), off), lambda: qb.expert_linear(x, w, off.long()), lambda: qb.expert_linear(x, w[0], off),
              lambda: qb.expert_linear(x[0], w, off), lambda: qb.expert_linear(x, w, off, pairs=off.float()), lambda: qb.expert_linear(x, w, off, pairs=off, k=0),
              lambda: qb.expert_linear(x, w, off, out_dtype=torch.int64), lambda: qb.expert_linear_backward(z(7, 32), x, w, off),
              lambda: qb.expert_linear_backward(z(8, 33), x, w, off), lambda: qb.expert_linear_backward(z(8, 32).half(), x, w, off),
              lambda: qb.swiglu(z(4, 7)), lambda: qb.swiglu_backward(z(4, 8), z(4, 15)), lambda: qb.swiglu_backward(z(4, 8), z(4, 16).half()),
              lambda: qb.combine(x, z(4, 2), off.view(1, 3)), lambda: qb.combine(x, None, off), lambda: qb.combine_backward(z(4, 64), x, None, off.view(1, 3), off),
              lambda: qb.combine_backward(z(1, 64).half(), x, None, off.view(1, 3), off),
              lambda: qb.w4_linear(x, z(16, 32, dtype=torch.uint8), z(16, 3, dtype=F16)), lambda: qb.w4_linear(x, z(16, 32, dtype=torch.uint8), z(16, 2, dtype=F32)),
              lambda: qb.w4_linear(x, z(16, 31, dtype=torch.uint8), z(16, 2, dtype=F16)), lambda: qb.w4_linear(x, z(16, 32, dtype=torch.int8), z(16, 2, dtype=F16)),
              lambda: qb.w4_linear(x.float(), z(16, 32, dtype=torch.uint8), z(16, 2, dtype=F16)),
              lambda: qb.w4_linear(x, z(2, 16, 32, dtype=torch.uint8), z(2, 16, 2, dtype=F16), ids=off), lambda: qb.align_sort(off, 4)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: qb.expert_linear(x.t(), z(2, 32, 8), off), lambda: qb.expert_linear(x, w.transpose(1, 2).contiguous().transpose(1, 2), off),
              lambda: qb.expert_linear(x.cpu(), w, off), lambda: qb.expert_linear(x, w, off, out_dtype=F16), lambda: qb.expert_linear(z(1, 64).expand(8, 64), w, off),
              lambda: qb.w4_linear(z(4, 64), z(16, 32, dtype=torch.uint8), z(16, 4, dtype=F16)),
              lambda: qb.w4_linear(z(4, 64), z(32, 16, dtype=torch.uint8).t(), z(16, 2, dtype=F16)),
              lambda: qb.expert_linear(x, w, off, ws=torch.empty(1, dtype=torch.uint8).cuda()) if qb.lib().qmoe_expert_workspace_bytes(8, 2, 32, 64, 0, 0)
              else (_ for _ in ()).throw(qb.QmoeError()),
              lambda: qb.w4_linear(z(20, 64), z(16, 32, dtype=torch.uint8), z(16, 2, dtype=F16), ws=torch.empty(256, dtype=torch.uint8).cuda())):
        with pytest.raises(qb.QmoeError):
            f()
    assert status() == 0


def test_align_sort():
    ids = torch.tensor([[2, 0], [1, 2], [-1, 5], [2, 1]], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets, pairs, slot = qb.align_sort(ids, 3, dev_status=word)
    assert offsets.tolist() == [0, 1, 3, 6] and pairs.tolist() == [1, 2, 7, 0, 3, 6, -1, -1]
    assert slot.tolist() == [[3, 0], [1, 4], [-1, -1], [5, 2]] and int(word) == qb.DEV_BAD_EXPERT_ID
    offsets, pairs, slot = qb.align_sort(ids[:0], 3)
    assert offsets.tolist() == [0, 0, 0, 0] and pairs.numel() == 0 == slot.numel()
