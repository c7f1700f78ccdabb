"""GPU tests of the operators around the experts (norms, routing with the balance loss, FP8 products) against plain 64-bit
forms.  Tolerances: one rounding of the output's type, and the fp32 arithmetic before it, bounded by the number of its
roundings times 2^-24 of the magnitudes that are added."""

import ctypes
import math

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from tests import block_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24
EPS = 1e-6
TYPES = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def f64(t):
    return None if t is None else t.double()


# ------------------------------------------------------------------ norms

NORM_SIZES = [(1, 1), (3, 7), (5, 64), (1, 256), (17, 255), (9, 257), (6, 1024), (33, 1000), (2, 4096), (129, 4104), (7, 4097),
              (5, 8192), (3, 8193), (2, 16384), (2, 16383), (700, 512), (1300, 136), (0, 64)]


def _gate(g, mode, T, H, block):
    return {"none": None, "row": torch.rand(T, 1, generator=g), "col": randn(g, H), "full": torch.rand(T, H, generator=g).to(block)}[mode]


def _norm_slack(x, w, H):
    # the sum of squares takes at most H / 128 + 40 additions in a row, half of which reach rstd; five more operations
    return (H / 128 + 48) * U * (x * w).abs()


@pytest.mark.parametrize("i,size", list(enumerate(NORM_SIZES)))
def test_norm_pre(i, size):
    T, H = size
    for j in range(2):
        st, bt = TYPES[(i + j) % 5]
        g = gen(100 + i)
        x, w = randn(g, T, H, dtype=st, scale=3.0), 1 + randn(g, H, scale=0.2)
        if T > 2:
            x[1] = 0  # an empty row: n = 0, rstd = 1 / sqrt(eps)
        n, rstd = qb.norm_pre(dev(x), dev(w), eps=EPS, out_dtype=bt)
        rn, rr = ref.norm(f64(x), f64(w), EPS)
        assert n.dtype == bt and n.shape == (T, H)
        ref.close(n, rn, _norm_slack(rn, torch.ones(()), H), "n")
        ref.close(rstd, rr, (H / 128 + 48) * U * rr, "rstd")


@pytest.mark.parametrize("gate_mode", ["none", "row", "col", "full"])
@pytest.mark.parametrize("i,size", list(enumerate(NORM_SIZES)))
def test_norm_post(i, size, gate_mode):
    T, H = size
    st, bt = TYPES[i % 5]
    g = gen(200 + i)
    r, y = randn(g, T, H, dtype=st), randn(g, T, H, dtype=bt, scale=0.3)
    gate = _gate(g, gate_mode, T, H, bt)
    w, w_next = (1 + randn(g, H, scale=0.2) for _ in range(2))
    if (i + len(gate_mode)) % 3 == 0:
        w = None
    if (i + len(gate_mode)) % 4 == 0:
        w_next = None
    out, n, rstd, rstd_next = qb.norm_post(dev(r), dev(y), w=dev(w), gate=dev(gate), alpha=-0.6, w_next=dev(w_next), eps=EPS)
    ro, rn = ref.post(f64(r), f64(y), f64(w), f64(gate), -0.6, f64(w_next), EPS)
    c = (H / 128 + 56) * U
    size_out = f64(r).abs() + (ro - f64(r)).abs()
    ref.close(out, ro, c * size_out, "out")
    assert (rstd is None) == (w is None) and (n is None) == (w_next is None) == (rstd_next is None)
    if w is not None:
        ry = ref.norm(f64(y), 1.0, EPS)[1]
        ref.close(rstd, ry, c * ry, "rstd")
    if w_next is not None:
        rr = ref.norm(ro, f64(w_next), EPS)[1]
        ref.close(n, rn, c * (rn.abs() + size_out * rr[:, None] * f64(w_next).abs()), "n")
        ref.close(rstd_next, rr, 2 * c * rr * (1 + size_out.square().mean(-1) * rr.square()), "rstd_next")


def _norm_bwd_slack(x, w, dn, rstd, H):
    xhat, d = (x * rstd[:, None]).abs(), (dn * w).abs()
    return (H / 128 + 64) * U * rstd[:, None] * (d + xhat * (d * xhat).mean(-1, keepdim=True))


def _directional(f, args, grads, seed):
    """Central differences of f (64 bits, a scalar) along a random direction, and the gradients' product with it."""
    g = gen(seed)
    ds = [torch.randn(a.shape, generator=g).double() for a in args]
    h = 1e-5
    up, down = f(*[a + h * d for a, d in zip(args, ds)]), f(*[a - h * d for a, d in zip(args, ds)])
    return float((up - down) / (2 * h)), float(sum((gr.double().cpu() * d).sum() for gr, d in zip(grads, ds))), ds


@pytest.mark.parametrize("i,size", list(enumerate(NORM_SIZES)))
def test_norm_pre_backward(i, size):
    T, H = size
    st, bt = TYPES[i % 5]
    g = gen(300 + i)
    x, dn, w = randn(g, T, H, dtype=st, scale=2.0), randn(g, T, H, dtype=bt), 1 + randn(g, H, scale=0.2)
    dres = randn(g, T, H, dtype=st) if i % 2 else None
    rstd = ref.norm(f64(x), 1.0, EPS)[1].float()
    dx, dw = qb.norm_pre_backward(dev(dn), dev(x), dev(rstd), dev(w), dres=dev(dres))
    assert dx.dtype == st and dw.dtype == F32
    lx, lw = f64(x).requires_grad_(), f64(w).requires_grad_()
    rx, rw = torch.autograd.grad(ref.norm(lx, lw, EPS)[0], (lx, lw), f64(dn))
    slack = _norm_bwd_slack(f64(x), f64(w), f64(dn), rstd.double(), H)
    if dres is not None:
        rx = rx + f64(dres)
        slack = slack + 2 * U * f64(dres).abs()
    ref.close(dx, rx, slack, "dx")
    ref.close(dw, rw, (T + 48) * U * (f64(dn) * f64(x) * rstd.double()[:, None]).abs().sum(0), "dw")


@pytest.mark.parametrize("gate_mode", ["none", "row", "col", "full"])
@pytest.mark.parametrize("i,size", list(enumerate(NORM_SIZES)))
def test_norm_post_backward(i, size, gate_mode):
    T, H = size
    st, bt = TYPES[(i + 1) % 5]
    g = gen(400 + i)
    alpha = 0.8
    y, out, dout, dn = randn(g, T, H, dtype=bt, scale=0.5), randn(g, T, H, dtype=st), randn(g, T, H, dtype=st), randn(g, T, H, dtype=bt)
    gate = _gate(g, gate_mode, T, H, bt)
    w, w_next = (1 + randn(g, H, scale=0.2) for _ in range(2))
    variant = (i + len(gate_mode)) % 4
    if variant == 1:
        w = None
    if variant == 2:
        dn = out = w_next = None
    if variant == 3:
        dout = None
    rstd = None if w is None else ref.norm(f64(y), 1.0, EPS)[1].float()
    rstd_next = None if dn is None else ref.norm(f64(out), 1.0, EPS)[1].float()
    dr, dy, dw, dgate, dw_next = qb.norm_post_backward(dev(dout), dev(y), w=dev(w), rstd=dev(rstd), gate=dev(gate), alpha=alpha,
                                                       dn=dev(dn), out=dev(out), w_next=dev(w_next), rstd_next=dev(rstd_next))
    d, d_slack = (f64(dout), 0.0) if dout is not None else (torch.zeros(T, H).double(), 0.0)
    if dn is not None:
        lo, lw = f64(out).requires_grad_(), f64(w_next).requires_grad_()
        through, rw = torch.autograd.grad(ref.norm(lo, lw, EPS)[0], (lo, lw), f64(dn))
        d = d + through
        d_slack = _norm_bwd_slack(f64(out), f64(w_next), f64(dn), rstd_next.double(), H)
        ref.close(dw_next, rw, (T + 48) * U * (f64(dn) * f64(out) * rstd_next.double()[:, None]).abs().sum(0), "dw_next")
    else:
        assert dw_next is None
    d_slack = d_slack + 2 * U * d.abs()
    ref.close(dr, d, d_slack, "dr")
    leaves = [t for t in (f64(y), f64(w), f64(gate)) if t is not None]
    for t in leaves:
        t.requires_grad_()
    it = iter(leaves)
    ly, lw, lg = next(it), None if w is None else next(it), None if gate is None else next(it)
    zero = torch.zeros(T, H).double()
    grads = list(torch.autograd.grad(ref.post(zero, ly, lw, lg, alpha, None, EPS)[0], leaves, d))
    ga = torch.ones(()).double() if gate is None else f64(gate)
    rs = torch.ones(T).double() if w is None else rstd.double()
    ww = torch.ones(H).double() if w is None else f64(w)
    dz_slack = (alpha * ga).abs() * (d_slack + 4 * U * d.abs())
    xhat = (f64(y) * rs[:, None]).abs()
    if w is None:
        slack = dz_slack
    else:
        slack = _norm_bwd_slack(f64(y), ww, alpha * ga * d, rs, H) + rs[:, None] * (dz_slack * ww.abs() + xhat * (dz_slack * ww.abs() * xhat).mean(-1, keepdim=True))
    ref.close(dy, grads.pop(0), slack, "dy")
    z = (xhat * ww.abs())
    if w is not None:
        ref.close(dw, grads.pop(0), (dz_slack * xhat).sum(0) + (T + 48) * U * ((alpha * ga * d).abs() * xhat).sum(0), "dw")
    else:
        assert dw is None
    if gate is None:
        assert dgate is None
        return
    each = alpha * (d_slack * z + 8 * U * d.abs() * z)
    all_ = alpha * d.abs() * z
    assert dgate.shape == gate.shape and dgate.dtype == gate.dtype
    if gate_mode == "row":
        each, all_ = each.sum(1, keepdim=True), (H / 128 + 48) * U * all_.sum(1, keepdim=True)
    elif gate_mode == "col":
        each, all_ = each.sum(0), (T + 48) * U * all_.sum(0)
    else:
        all_ = 0.0
    ref.close(dgate, grads.pop(0), each + all_, "dgate")


def test_norm_gate_shapes_of_as_many_rows_as_columns():
    # [T] is one for each row even where T == H; [1, H] is always one for each column
    g = gen(9)
    n = 24
    r, y, gate = randn(g, n, n), randn(g, n, n), randn(g, n)
    c = (n / 128 + 56) * U
    for given, wide in [(gate, gate[:, None]), (gate[:, None], gate[:, None]), (gate[None], gate[None])]:
        want = ref.post(f64(r), f64(y), None, f64(wide), 1.0, None, EPS)[0]
        got = qb.norm_post(dev(r), dev(y), gate=dev(given))[0]
        ref.close(got, want, c * (f64(r).abs() + (want - f64(r)).abs()), "out")
        dgate = qb.norm_post_backward(dev(r), dev(y), gate=dev(given))[3]
        each = f64(r) * f64(y)
        by = 1 if wide.shape[1] == 1 else 0
        assert dgate.shape == given.shape
        ref.close(dgate.flatten(), each.sum(by), (n + 48) * U * each.abs().sum(by), "dgate")
    one = qb.norm_post(dev(r[:1]), dev(y[:1]), gate=dev(gate[None]))[0]  # one row: [1, H]
    ref.close(one, f64(r[:1]) + f64(gate) * f64(y[:1]), c * (f64(r[:1]).abs() + (f64(gate) * f64(y[:1])).abs()), "out")


def test_norm_gradients_against_differences():
    T, H, alpha = 6, 40, 0.9
    g = gen(7)
    r, y, dout, dn = (randn(g, T, H) for _ in range(4))
    w, w_next, gate = 1 + randn(g, H, scale=0.2), 1 + randn(g, H, scale=0.2), torch.rand(T, 1, generator=g)
    out, n, rstd, rstd_next = qb.norm_post(dev(r), dev(y), w=dev(w), gate=dev(gate), alpha=alpha, w_next=dev(w_next), eps=EPS)
    dr, dy, dw, dgate, dw_next = qb.norm_post_backward(dev(dout), dev(y), w=dev(w), rstd=rstd, gate=dev(gate), alpha=alpha,
                                                       dn=dev(dn), out=out, w_next=dev(w_next), rstd_next=rstd_next)

    def f(r_, y_, w_, g_, wn_):
        o, n_ = ref.post(r_, y_, w_, g_, alpha, wn_, EPS)
        return (o * f64(dout)).sum() + (n_ * f64(dn)).sum()

    args = [f64(t) for t in (r, y, w, gate, w_next)]
    grads = [dr, dy, dw, dgate, dw_next]
    a, b, ds = _directional(f, args, grads, 8)
    # fp32 gradients: 64 roundings of the magnitudes, differences: h^2
    size = sum(float((gr.double().cpu() * d).abs().sum()) for gr, d in zip(grads, ds))
    assert abs(a - b) <= 256 * U * size + 1e-6


# rows that begin at every place of a 16-byte access, several for each CTA; weights off the boundaries
@pytest.mark.parametrize("i,size", list(enumerate([(1300, 6), (700, 1021), (400, 4095), (340, 4099), (320, 6001), (170, 8195)])))
def test_norm_odd_rows(i, size):
    T, H = size
    for j in range(2):
        st, bt = TYPES[(2 * i + j) % 5]
        g = gen(700 + i)
        r, y, w, w_next = randn(g, T, H, dtype=st), randn(g, T, H, dtype=bt, scale=0.3), randn(g, H + 1)[1:], randn(g, H + 1)[1:]
        gate, dout, dn = torch.rand(T, H, generator=g).to(bt), randn(g, T, H, dtype=st), randn(g, T, H, dtype=bt)
        c = (H / 128 + 56) * U
        on = [dev(torch.cat([torch.zeros(1), v]))[1:] for v in (w, w_next)]
        out, n, rstd, rstd_next = qb.norm_post(dev(r), dev(y), w=on[0], gate=dev(gate), w_next=on[1], eps=EPS)
        ro, rn = ref.post(f64(r), f64(y), f64(w), f64(gate), 1.0, f64(w_next), EPS)
        size_out, rr = f64(r).abs() + (ro - f64(r)).abs(), ref.norm(ro, 1.0, EPS)[1]
        ref.close(out, ro, c * size_out, "out")
        ref.close(n, rn, c * (rn.abs() + size_out * rr[:, None] * f64(w_next).abs()), "n")
        rstd = ref.norm(f64(y), 1.0, EPS)[1].float()
        o = ro.to(st)
        rstd_next = ref.norm(f64(o), 1.0, EPS)[1].float()
        dr, dy, dw, dgate, dw_next = qb.norm_post_backward(dev(dout), dev(y), w=on[0], rstd=dev(rstd), gate=dev(gate), dn=dev(dn),
                                                           out=dev(o), w_next=on[1], rstd_next=dev(rstd_next))
        lo, lw = f64(o).requires_grad_(), f64(w_next).requires_grad_()
        through, rw = torch.autograd.grad(ref.norm(lo, lw, EPS)[0], (lo, lw), f64(dn))
        d = f64(dout) + through
        d_slack = _norm_bwd_slack(f64(o), f64(w_next), f64(dn), rstd_next.double(), H) + 2 * U * d.abs()
        ref.close(dr, d, d_slack, "dr")
        ref.close(dw_next, rw, (T + 48) * U * (f64(dn) * f64(o) * rstd_next.double()[:, None]).abs().sum(0), "dw_next")
        leaves = [v.requires_grad_() for v in (f64(y), f64(w), f64(gate))]
        ry, rw, rg = torch.autograd.grad(ref.post(torch.zeros(T, H).double(), *leaves, 1.0, None, EPS)[0], leaves, d)
        rs, ga, ww = rstd.double()[:, None], f64(gate), f64(w)
        xhat, dz = (f64(y) * rs).abs(), ga * (d_slack + 4 * U * d.abs())
        lost = rs * (dz * ww.abs() + xhat * (dz * ww.abs() * xhat).mean(-1, keepdim=True))
        ref.close(dy, ry, _norm_bwd_slack(f64(y), ww, ga * d, rs[:, 0], H) + lost, "dy")
        ref.close(dw, rw, (dz * xhat).sum(0) + (T + 48) * U * ((ga * d).abs() * xhat).sum(0), "dw")
        ref.close(dgate, rg, (d_slack + 8 * U * d.abs()) * xhat * ww.abs(), "dgate")


# the widest rows that go through the ring, five fp32 matrices: a stage, and with it the whole ring, of 164 KB
@pytest.mark.parametrize("T,H", [(3, 8188), (3, 8189), (310, 8191), (310, 8192)])
def test_norm_gradient_of_five_matrices_of_the_widest_rows(T, H):
    g = gen(760)
    y, out, dout, dn = randn(g, T, H, scale=0.5), randn(g, T, H), randn(g, T, H), randn(g, T, H)
    gate, w, w_next = torch.rand(T, H, generator=g), 1 + randn(g, H, scale=0.2), 1 + randn(g, H, scale=0.2)
    rstd, rstd_next = ref.norm(f64(y), 1.0, EPS)[1].float(), ref.norm(f64(out), 1.0, EPS)[1].float()
    dr, dy, dw, dgate, dw_next = qb.norm_post_backward(dev(dout), dev(y), w=dev(w), rstd=dev(rstd), gate=dev(gate), alpha=0.8, dn=dev(dn),
                                                       out=dev(out), w_next=dev(w_next), rstd_next=dev(rstd_next))
    lo, lw = f64(out).requires_grad_(), f64(w_next).requires_grad_()
    through, rw = torch.autograd.grad(ref.norm(lo, lw, EPS)[0], (lo, lw), f64(dn))
    d = f64(dout) + through
    d_slack = _norm_bwd_slack(f64(out), f64(w_next), f64(dn), rstd_next.double(), H) + 2 * U * d.abs()
    ref.close(dr, d, d_slack, "dr")
    ref.close(dw_next, rw, (T + 48) * U * (f64(dn) * f64(out) * rstd_next.double()[:, None]).abs().sum(0), "dw_next")
    leaves = [v.requires_grad_() for v in (f64(y), f64(w), f64(gate))]
    ry, rw, rg = torch.autograd.grad(ref.post(torch.zeros(T, H).double(), *leaves, 0.8, None, EPS)[0], leaves, d)
    rs, ga, ww = rstd.double()[:, None], 0.8 * f64(gate), f64(w)
    xhat, dz = (f64(y) * rs).abs(), ga * (d_slack + 4 * U * d.abs())
    lost = rs * (dz * ww.abs() + xhat * (dz * ww.abs() * xhat).mean(-1, keepdim=True))
    ref.close(dy, ry, _norm_bwd_slack(f64(y), ww, ga * d, rs[:, 0], H) + lost, "dy")
    ref.close(dw, rw, (dz * xhat).sum(0) + (T + 48) * U * ((ga * d).abs() * xhat).sum(0), "dw")
    ref.close(dgate, rg, 0.8 * (d_slack + 8 * U * d.abs()) * xhat * ww.abs(), "dgate")


def test_norm_odd_rows_beside_an_infinite_gate():
    # a row gate that is infinite makes its own row infinite (1 / rms = 0), whatever lies past the ends of the row
    g = gen(91)
    T, H = 9, 1021
    r, y, gate, w = randn(g, T, H), randn(g, T, H).abs() + 0.1, torch.rand(T, 1, generator=g), torch.ones(H)
    gate[4] = math.inf
    out, n, _, rstd_next = qb.norm_post(dev(r), dev(y), w=dev(w), gate=dev(gate), w_next=dev(w), eps=EPS)
    assert torch.isinf(out[4]).all() and float(rstd_next[4].cpu()) == 0
    others = [i for i in range(T) if i != 4]
    assert torch.isfinite(out[others]).all() and torch.isfinite(n[others]).all() and (rstd_next[others] > 0).all()


def test_norm_strides_and_alignment():
    # rows with a stride, a base off the 16-byte boundary, and outputs whose padding stays as it was
    T, H = 5, 96
    for off, ld in [(0, 104), (1, 104), (0, 97), (8, 112)]:
        g = gen(11)
        buf_x, buf_n = randn(g, T * ld + 16, dtype=BF16).cuda(), torch.full((T * ld + 16,), 7.0, dtype=BF16).cuda()
        x = torch.as_strided(buf_x, (T, H), (ld, 1), off)
        n = torch.as_strided(buf_n, (T, H), (ld, 1), off)
        w = torch.ones(H).cuda()
        assert qb.lib().qmoe_norm_pre(T, H, 1, 1, x.data_ptr(), ld, w.data_ptr(), EPS, n.data_ptr(), ld, None, None) == 0
        torch.cuda.synchronize()
        rn, _ = ref.norm(x.cpu().double(), torch.ones(H).double(), EPS)
        ref.close(n, rn, _norm_slack(rn, torch.ones(()), H), "n")
        keep = torch.ones(T * ld + 16, dtype=torch.bool)
        torch.as_strided(keep, (T, H), (ld, 1), off).fill_(False)
        assert (buf_n.cpu()[keep] == 7.0).all()
        n2, _ = qb.norm_pre(x, w, eps=EPS)
        ref.close(n2, rn, _norm_slack(rn, torch.ones(()), H), "n")


def test_norm_in_place_and_repeatable():
    g = gen(12)
    r, y, w = randn(g, 300, 512).cuda(), randn(g, 300, 512).cuda(), torch.ones(512).cuda()
    out = qb.norm_post(r, y, w=w, alpha=0.5, eps=EPS)[0]
    same = r.clone()
    rc = qb.lib().qmoe_norm_post(300, 512, 0, 0, same.data_ptr(), 512, y.data_ptr(), 512, w.data_ptr(), 0, None, 0, 0.5, None, EPS,
                                 same.data_ptr(), 512, None, 0, None, None, None)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(same, out)
    rstd = qb.norm_pre(y, w, eps=EPS)[1]
    one, two = (qb.norm_pre_backward(r, y, rstd, w) for _ in range(2))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_norm_values_that_are_not_finite():
    g = gen(13)
    x, w = randn(g, 6, 200), torch.ones(200)
    x[1, 5], x[3, 7], x[4, 8] = math.nan, math.inf, -math.inf
    n, _ = qb.norm_pre(x.cuda(), w.cuda(), eps=EPS)
    n = n.cpu()
    assert n[1].isnan().all() and n[3, 7].isnan() and n[4, 8].isnan()  # inf * 0
    assert (n[3][torch.arange(200) != 7] == 0).all()
    for t in (0, 2, 5):
        assert n[t].isfinite().all()  # rows do not touch each other


# ------------------------------------------------------------------ routing

ROUTE_SIZES = [(1, 1, 1), (1, 512, 10), (5, 2, 2), (7, 31, 3), (64, 32, 4), (33, 33, 33 - 1), (300, 64, 8), (40, 100, 7), (129, 128, 1),
               (50, 255, 16), (1000, 512, 10), (17, 513, 9), (9, 1024, 32), (0, 16, 2)]


def _logits(g, T, E, dtype, kind):
    lg = randn(g, T, E, scale=1.5)
    if kind == "ties":
        lg = (lg * 2).round() / 2
        lg[lg == 0] *= torch.where(torch.rand(int((lg == 0).sum()), generator=g) < 0.5, -1.0, 1.0)  # both zeros
    if kind == "holes":
        lg = lg.masked_fill(torch.rand(T, E, generator=g) < 0.5, -math.inf)
        lg[::3] = -math.inf
    if kind == "lowest":
        lg = lg.masked_fill(torch.rand(T, E, generator=g) < 0.5, torch.finfo(dtype).min)
        if T:
            lg[0] = torch.finfo(dtype).min  # a row of the lowest value alone: all equal
    return lg.to(dtype)


def _route_slack(r, lg, E):
    # exp of a difference d has a relative error of about 2 |d| 2^-24 and a few more; sums of E terms
    low = torch.where(lg > -1e30, lg, torch.zeros_like(lg))
    return (2 * (low.abs().amax() if low.numel() else 0.0) * 2 + E / 32 + 32) * U


@pytest.mark.parametrize("kind", ["plain", "ties", "holes", "lowest"])
@pytest.mark.parametrize("i,size", list(enumerate(ROUTE_SIZES)))
def test_route_topk(i, size, kind):
    T, E, k = size
    dtype = [F32, BF16, F16][(i + len(kind)) % 3]
    g = gen(500 + i)
    lg = _logits(g, T, E, dtype, kind)
    bias = randn(g, E, scale=0.3) if i % 2 else None
    mask = torch.rand(T, generator=g) < 0.8 if i % 3 else None
    renorm, scale, coef = bool(i % 2), 1.0 if i % 4 else 2.5, 0.02
    got = qb.route_topk(dev(lg), k, bias=dev(bias), mask=dev(mask), renorm=renorm, scale=scale, coef=coef)
    want = ref.route(f64(lg), k, bias, mask, renorm, scale, coef)
    assert torch.equal(got.ids.cpu(), want["ids"])
    assert torch.equal(got.counts.cpu(), want["counts"])
    c = _route_slack(want, f64(lg), E)
    ref.close(got.w, want["w"], c * want["w"], "w")
    gone = torch.isinf(want["lse"])
    assert torch.equal(torch.isinf(got.lse.cpu()), gone)
    ref.close(got.lse[dev(~gone)], want["lse"][~gone], 2 * U * f64(lg)[~gone].abs().amax(1) + c, "lse")
    ref.close(got.probs, want["probs"], (c + (T + 48) * U) * want["probs"], "probs")
    ref.close(got.loss, want["loss"][None], (c + (T + E + 64) * U) * want["loss"].abs(), "loss")
    bare = qb.route_topk(dev(lg), k, bias=dev(bias), mask=dev(mask), renorm=renorm, scale=scale)
    assert torch.equal(bare.ids, got.ids) and torch.equal(bare.w, got.w) and bare.loss is None


@pytest.mark.parametrize("kind", ["plain", "ties", "holes", "lowest"])
@pytest.mark.parametrize("i,size", list(enumerate(ROUTE_SIZES)))
def test_route_topk_backward(i, size, kind):
    T, E, k = size
    dtype = [F32, BF16, F16][i % 3]
    g = gen(600 + i)
    lg = _logits(g, T, E, dtype, kind)
    mask = torch.rand(T, generator=g) < 0.8 if i % 2 else None
    dw, dloss = randn(g, T, k), torch.tensor([1.7])
    coef = 0.5
    for renorm, use in [(True, "both"), (False, "both"), (bool(i % 2), "dw"), (bool(i % 2), "loss")]:
        r = qb.route_topk(dev(lg), k, mask=dev(mask), renorm=renorm, scale=1.5, coef=coef)
        got = qb.route_topk_backward(dev(lg), r, dw=dev(dw) if use != "loss" else None, dloss=dev(dloss) if use != "dw" else None)
        leaf = f64(lg).requires_grad_()
        want = ref.route(leaf, k, None, mask, renorm, 1.5, coef)
        total = want["w"].sum() * 0
        if use != "loss":
            total = total + (want["w"] * f64(dw)).sum()
        if use != "dw":
            total = total + want["loss"] * 1.7
        grad = torch.nan_to_num(torch.autograd.grad(total, leaf)[0])
        p, w = want["p"].detach(), want["w"].detach()
        n = max(int(want["counts"][-1]), 1)
        a = 1.7 * coef * E * want["counts"][:-1].double() / (n * k) / n if use != "dw" else torch.zeros(E).double()
        s = (w * f64(dw).abs()).sum(1, keepdim=True) if use != "loss" else torch.zeros(T, 1).double()
        size_ = p * (a + (p * a).sum(1, keepdim=True) + s)
        if use != "loss":
            at = want["ids"].clamp(min=0).long()
            size_ = size_.scatter_add(1, at, w * (f64(dw).abs() + s))
        lse = want["lse"].detach()
        lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
        c = 4 * _route_slack(want, f64(lg), E) + 4 * U * (lse.abs().amax() if T else 0.0)
        ref.close(got, grad, c * size_, f"dlogits {renorm} {use}")


def test_route_gradient_against_differences():
    T, E, k = 6, 20, 3
    g = gen(21)
    lg, dw, dloss = randn(g, T, E), randn(g, T, k), torch.tensor([0.8])
    for renorm in (True, False):
        r = qb.route_topk(dev(lg), k, renorm=renorm, coef=0.3)
        got = qb.route_topk_backward(dev(lg), r, dw=dev(dw), dloss=dev(dloss))

        def f(x):  # the choice of experts does not move over 1e-5
            v = ref.route(x, k, None, None, renorm, 1.0, 0.3)
            return (v["w"] * f64(dw)).sum() + 0.8 * v["loss"]

        a, b, ds = _directional(f, [f64(lg)], [got], 22)
        assert abs(a - b) <= 256 * U * float((got.cpu().double() * ds[0]).abs().sum() + f64(dw).abs().sum()) + 1e-7


@pytest.mark.parametrize("E", [5, 64, 300, 512, 1024])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_scores_that_differ_in_their_last_bits(E, dtype):
    # the choice goes by whole 32-bit scores, ties by the lower expert, among neighbouring floats too
    g = gen(60 + E)
    T, k = 40, min(E, 7)
    step = torch.randint(0, 3 * E, (T, E), generator=g).float()
    if dtype == F32:
        lg, bias = 1.0 + step * 2.0 ** -23, None
        lg[::4] = -lg[::4]
        lg[1::4, E // 2:] += 3.0
    else:
        lg, bias = (1.0 + step / 128).to(BF16), torch.randint(0, 4, (E,), generator=g).float() * 2.0 ** -20
    score = lg.float() if bias is None else lg.float() + bias
    got = qb.route_topk(dev(lg), k, bias=dev(bias))
    want = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(got.ids.cpu().long(), want)
    p = torch.softmax(f64(lg), 1).gather(1, want)
    w = p / p.sum(1, keepdim=True)
    ref.close(got.w, w, _route_slack(got, f64(lg), E) * w, "w")


@pytest.mark.parametrize("E", [6, 64, 512, 1000])
def test_route_bias_off_its_boundaries_and_not_finite(E):
    # -inf and NaN in the bias take an expert out, +inf puts it first; weights are of the logits alone
    g = gen(80 + E)
    T, k = 33, 3
    lg, whole = randn(g, T, E, dtype=BF16), randn(g, E + 1)
    whole[[1, 4]], whole[2], whole[5] = -math.inf, math.nan, math.inf
    got = qb.route_topk(dev(lg), k, bias=dev(whole)[1:])
    score = lg.float() + whole[1:].nan_to_num(nan=-math.inf, posinf=1e30)
    want = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(got.ids.cpu().long(), want) and (want[:, 0] == 4).all()
    w = torch.softmax(f64(lg).gather(1, want), 1)
    ref.close(got.w, w, _route_slack(got, f64(lg), E) * w, "w")


def test_route_values_that_are_not_numbers():
    lg = torch.zeros(4, 8)
    lg[0] = torch.arange(8.0)
    lg[0, 7], lg[0, 6] = math.nan, math.inf
    lg[1] = math.nan
    lg[2, 3] = lg[2, 5] = math.inf
    r = qb.route_topk(lg.cuda(), 3, renorm=False, coef=1.0)
    ids, w = r.ids.cpu(), r.w.cpu()
    assert ids[0].tolist() == [6, 5, 4] and w[0].tolist() == [1.0, 0.0, 0.0]
    assert ids[1].tolist() == [-1, -1, -1] and w[1].tolist() == [0.0, 0.0, 0.0]
    assert ids[2].tolist() == [3, 5, 0] and w[2].tolist() == [0.5, 0.5, 0.0]
    assert ids[3].tolist() == [0, 1, 2]
    assert int(r.counts[-1]) == 3 and bool(torch.isfinite(r.loss).all())


def _infinite_rows(E, dtype):
    """Rows with one, two and four logits of +inf, beside the type's largest finite value, NaN and -inf; the experts with
    +inf by row."""
    top = torch.finfo(dtype).max
    lg = torch.linspace(-2.0, 2.0, E).repeat(4, 1)
    lg[0, 5] = math.inf
    lg[1, [1, E - 1]] = math.inf
    lg[2, [0, 2, 3, 6]] = math.inf
    lg[3, 4], lg[3, 0], lg[3, 1], lg[3, 2] = math.inf, top, math.nan, -math.inf
    return lg.to(dtype), [[5], [1, E - 1], [0, 2, 3, 6], [0, 4] if dtype == F32 else [4]]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("E", [8, 65, 512, 1024])
def test_route_infinite_logits_take_all_the_weight(E, dtype, renorm):
    # +inf counts as the largest finite value: equal shares for the experts that have it, and exactly 0 for all others
    lg, there = _infinite_rows(E, dtype)
    k, scale = 6, 2.0
    dw = torch.full((4, k), 3.0)
    dw[:, 0], dw[:, 1] = 0.25, -0.5
    for wide in (False, True):  # contiguous rows, and rows off the 16-byte boundaries
        on = torch.zeros(4, E + 3, dtype=dtype).cuda()[:, 1:E + 1] if wide else torch.zeros(4, E, dtype=dtype).cuda()
        on.copy_(lg)
        r = qb.route_topk(on, k, renorm=renorm, scale=scale, coef=1.0)
        bare = qb.route_topk(on, k, renorm=renorm, scale=scale)
        dl = qb.route_topk_backward(on, r, dw=dw.cuda()).cpu().float()
        ids, w = r.ids.cpu(), r.w.cpu()
        assert torch.equal(bare.ids, r.ids) and torch.equal(bare.w, r.w)
        probs = torch.zeros(E)
        for t, at in enumerate(there):
            n = len(at)
            assert ids[t, :n].tolist() == at
            assert w[t].tolist() == [scale / n] * n + [0.0] * (k - n)
            probs[at] += 1.0 / n / 4
            # w_j (dw_j - sum_i w_i dw_i / scale), exact in every type; 0 for the experts without weight
            mean = sum(dw[t, :n].tolist()) / n
            want = torch.zeros(E)
            want[at] = scale / n * (dw[t, :n] - mean)
            assert torch.equal(dl[t], want), (t, dl[t][at], want[at])
        assert torch.equal(r.probs.cpu(), probs) and int(r.counts[-1]) == 4
        largest = torch.finfo(F32).max
        assert (r.lse.cpu() == largest).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("i,size", list(enumerate([(3, 8, 3), (40, 60, 7), (700, 128, 8), (33, 512, 10), (20, 1000, 32)])))
def test_route_weights_by_type_bias_and_renorm(i, size, dtype, biased, renorm):
    T, E, k = size
    g = gen(900 + i)
    lg = _logits(g, T, E, dtype, "holes" if i % 2 else "plain")
    bias, mask = randn(g, E, scale=0.3) if biased else None, torch.rand(T, generator=g) < 0.8
    got = qb.route_topk(dev(lg), k, bias=dev(bias), mask=dev(mask), renorm=renorm, scale=1.5, coef=0.1)
    want = ref.route(f64(lg), k, bias, mask, renorm, 1.5, 0.1)
    assert torch.equal(got.ids.cpu(), want["ids"]) and torch.equal(got.counts.cpu(), want["counts"])
    c = _route_slack(want, f64(lg), E)
    ref.close(got.w, want["w"], c * want["w"], "w")
    ref.close(got.probs, want["probs"], (c + (T + 48) * U) * want["probs"], "probs")
    ref.close(got.loss, want["loss"][None], (c + (T + E + 64) * U) * want["loss"].abs(), "loss")


def test_route_feeds_the_routing_sort():
    # ids of -1 (masked tokens) take no slot
    g = gen(31)
    lg, mask = randn(g, 50, 16), torch.rand(50, generator=g) < 0.7
    r = qb.route_topk(lg.cuda(), 4, mask=mask.cuda(), coef=1.0)
    d = qb.dims(50, 4, 256, 128, 16)
    o = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in [("c", 16), ("o", 17), ("s", 200), ("p", 200)]}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb.qmoe_align_sort(d, r.ids, o["c"], o["o"], o["s"], o["p"], st, qb.alloc_workspace(qb.workspace_bytes(d)))
    assert torch.equal(o["c"], r.counts[:-1]) and int(o["o"][-1]) == int(mask.sum()) * 4
    assert (o["p"].view(50, 4)[~mask.cuda()] == -1).all()


def test_route_repeatable():
    g = gen(32)
    lg = randn(g, 5000, 200).cuda()
    one, two = (qb.route_topk(lg, 6, coef=1.0) for _ in range(2))
    for name in ("ids", "w", "lse", "counts", "probs", "loss"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name


# ------------------------------------------------------------------ FP8

QUANT_SIZES = [(1, 1), (1, 128), (3, 100), (5, 129), (130, 8), (128, 128), (127, 257), (300, 136), (64, 1000), (257, 512)]


def _wild(g, R, C, dtype):
    """Values over a wide range, zero blocks, and magnitudes whose codes are halfway between two."""
    x = randn(g, R, C) * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g).float())
    x[:, : C // 2] = torch.where(torch.rand(R, C // 2, generator=g) < 0.3, 0.0, x[:, : C // 2])
    x[R // 2] = 0
    x = x.to(dtype)
    if C > 3:
        x[0, 1], x[0, 2], x[0, 3] = 3.5, 0.1328125, -0.1484375  # with 3.5 the largest: halves of code steps
        x[0, 4:] = x[0, 4:].clamp(-3.5, 3.5)
        x[0, 0] = 0
    return x


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("i,size", list(enumerate(QUANT_SIZES)))
def test_fp8_quant(i, size, dtype):
    R, C = size
    x = _wild(gen(700 + i), R, C, dtype)
    xd = x.cuda()
    q, s = qb.fp8_quant_rows(xd)
    rq, rs = ref.quant(x, 1)
    assert torch.equal(bits(q.cpu()), bits(rq)) and torch.equal(s.cpu(), rs)
    cq, cs = ref.quant(x.t(), 1)
    qt, st, q2, s2 = qb.fp8_quant_cols(xd, rows_too=True)
    assert torch.equal(bits(qt.cpu()), bits(cq)) and torch.equal(st.cpu(), cs)
    assert torch.equal(bits(q2.cpu()), bits(rq)) and torch.equal(s2.cpu(), rs)
    qt, st = qb.fp8_quant_cols(xd)
    assert torch.equal(bits(qt.cpu()), bits(cq)) and torch.equal(st.cpu(), cs)
    bq, bs = ref.quant(x, 128)
    q, s, qt = qb.fp8_quant_blocks(xd, transposed=True)
    assert torch.equal(bits(q.cpu()), bits(bq)) and torch.equal(s.cpu(), bs) and torch.equal(bits(qt.cpu()), bits(bq.t()))
    q, s = qb.fp8_quant_blocks(xd)
    assert torch.equal(bits(q.cpu()), bits(bq)) and torch.equal(s.cpu(), bs)


def test_fp8_quant_strides_and_specials():
    g = gen(41)
    big = randn(g, 20, 400).cuda()
    for x in (big[:, 3:300], big[::2, :256], big[5:6, 1:2]):
        q, s = qb.fp8_quant_rows(x)
        rq, rs = ref.quant(x.cpu(), 1)
        assert torch.equal(bits(q.cpu()), bits(rq)) and torch.equal(s.cpu(), rs)
    x = torch.full((3, 256), 1e-38)
    x[0, 5], x[1, 7], x[1, 200] = math.nan, math.inf, 2.0
    q, s = qb.fp8_quant_rows(x.cuda())
    v = q.cpu().float()
    assert v[0, 5].isnan() and (v[0][torch.arange(256) != 5] == 0).all()  # too small for the least scale
    assert v[1, 7].isnan() and (v[1, :128][torch.arange(128) != 7] == 0).all() and v[1, 200] == 448
    assert (v[2] == 0).all() and torch.equal(s[2].cpu(), torch.full((2,), 2.0 ** -100) / torch.tensor(448.0))


MATMUL_SIZES = [(1, 1, 1), (1, 128, 128), (1, 512, 2048), (2, 200, 300), (15, 129, 100), (16, 384, 1024), (17, 127, 257), (33, 1000, 512),
                (60, 8, 2040), (64, 640, 640), (65, 130, 129), (128, 256, 1536), (129, 384, 16), (200, 1, 4096), (256, 129, 384),
                (257, 300, 200), (513, 260, 256), (2000, 2816, 320), (700, 4096, 130), (2050, 2501, 200), (10001, 300, 1290), (256, 9800, 128)]


def _mats(g, M, N, K, b_tall):
    a, a_s = ref.quant(randn(g, M, K) * torch.exp2(torch.randint(-6, 6, (M, 1), generator=g).float()), 1)
    b, b_s = ref.quant(randn(g, N, K) * torch.exp2(torch.randint(-6, 6, (N, 1), generator=g).float()), b_tall)
    return a, a_s, b, b_s


def _padded(q):
    """The same codes on the GPU with rows on 16-byte boundaries."""
    out = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")[:, :q.shape[1]]
    out.copy_(q.cuda())
    return out


def _mat(q, s):
    return qb.Fp8Mat(q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0), s.stride(1), 1 if s.shape[0] == q.shape[0] else 128, 0)


@pytest.mark.parametrize("b_tall", [1, 128])
@pytest.mark.parametrize("i,size", list(enumerate(MATMUL_SIZES)))
def test_fp8_matmul(i, size, b_tall):
    M, N, K = size
    a, a_s, b, b_s = _mats(gen(800 + i), M, N, K, b_tall)
    want, slack = ref.product(ref.dequant(a, a_s), ref.dequant(b, b_s))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out_dtype in (F32, [BF16, F16][i % 2]):
        if out_dtype == F16 and want.abs().max() > 60000:
            continue
        c = qb.fp8_matmul(_padded(a), a_s.cuda(), _padded(b), b_s.cuda(), out_dtype=out_dtype, dev_status=status)
        ref.close(c, want, slack, "c")
        # scales in the other order of strides
        d = qb.fp8_matmul(_padded(a), a_s.cuda().t().contiguous().t(), _padded(b), b_s.cuda().t().contiguous().t(), out_dtype=out_dtype)
        assert torch.equal(c, d)
    assert int(status) == 0 and int(qb.status_word("cuda")) == 0


def test_fp8_matmul_block_scales_on_both_sides():
    g = gen(51)
    a, a_s = ref.quant(randn(g, 300, 260), 128)
    b, b_s = ref.quant(randn(g, 140, 260), 128)
    want, slack = ref.product(ref.dequant(a, a_s), ref.dequant(b, b_s))
    ref.close(qb.fp8_matmul(_padded(a), a_s.cuda(), _padded(b), b_s.cuda(), out_dtype=F32), want, slack, "c")


def test_fp8_matmul_strided_output_and_codes():
    # c with a row stride: what lies between its rows stays; codes that are part of a wider matrix
    g = gen(52)
    a, a_s, b, b_s = _mats(g, 70, 200, 256, 1)
    wide = torch.zeros(70, 512, dtype=torch.uint8, device="cuda")
    wide[:, 128:384] = bits(a).cuda()
    want, slack = ref.product(ref.dequant(a, a_s), ref.dequant(b, b_s))
    ref.close(qb.fp8_matmul(wide[:, 128:384], a_s.cuda(), _padded(b), b_s.cuda(), out_dtype=F32), want, slack, "c")
    c = torch.full((70, 211), 9.0, device="cuda")
    bq, bs, as_ = _padded(b), b_s.cuda(), a_s.cuda()
    ma, mb = _mat(wide[:, 128:384], as_), _mat(bq, bs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert qb.lib().qmoe_fp8_matmul(70, 200, 256, ctypes.byref(ma), ctypes.byref(mb), c.data_ptr(), 0, 211, st.data_ptr(), None) == 0
    torch.cuda.synchronize()
    ref.close(c[:, :200], want, slack, "c")
    assert (c[:, 200:] == 9.0).all()


def test_fp8_matmul_values_that_are_not_finite():
    g = gen(53)
    a, a_s, b, b_s = _mats(g, 40, 150, 256, 1)
    av = bits(a).clone()
    av[7, 3] = 0x7F  # NaN
    c = qb.fp8_matmul(_padded(av.view(torch.float8_e4m3fn)), a_s.cuda(), _padded(b), b_s.cuda(), out_dtype=F32).cpu()
    assert c[7].isnan().all() and c[torch.arange(40) != 7].isfinite().all()


@pytest.mark.parametrize("size", [(1, 2048, 4096), (60, 1407, 2040), (130, 256, 100), (300, 640, 512), (0, 128, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_fp8_linear_and_backward(size, dtype):
    T, N, K = size
    g = gen(61)
    x, w, dy = randn(g, T, K, dtype=dtype), randn(g, N, K, dtype=dtype, scale=K ** -0.5), randn(g, T, N, dtype=dtype, scale=0.1)
    w_q, w_s, wt_q = qb.fp8_quant_blocks(w.cuda(), transposed=True)
    y = qb.fp8_linear(x.cuda(), w_q, w_s)
    dx, dw = qb.fp8_linear_backward(dy.cuda(), x.cuda(), wt_q, w_s)
    wd = ref.dequant(*ref.quant(w, 128))
    if T == 0:
        assert y.shape == (0, N) and dx.shape == (0, K) and dw.shape == (N, K) and not dw.any()
        return
    ref.close(y, *ref.product(ref.dequant(*ref.quant(x, 1)), wd), "y")
    ref.close(dx, *ref.product(ref.dequant(*ref.quant(dy, 1)), wd.t().contiguous()), "dx")
    ref.close(dw, *ref.product(ref.dequant(*ref.quant(dy.t().contiguous(), 1)), ref.dequant(*ref.quant(x.t().contiguous(), 1))), "dw")


@pytest.mark.parametrize("T,N,K", [(1, 2048, 4096), (1, 128, 256), (40, 1500, 512), (300, 640, 1024)])
def test_fp8_linear_with_weights_written_by_the_calls_around_it(T, N, K):
    # products read weight tiles before the kernel ahead of them has ended: codes and scales that are written anew between
    # two products on one stream are those of the call's own turn
    g = gen(74)
    x, ws = randn(g, T, K, dtype=BF16).cuda(), [randn(g, N, K, dtype=BF16).cuda() for _ in range(6)]
    want = []
    for w in ws:
        want.append(qb.fp8_linear(x, *qb.fp8_quant_blocks(w), out_dtype=F32))
        torch.cuda.synchronize()
    q, s = qb.fp8_quant_blocks(ws[0])
    for _ in range(10):
        got = []
        for w in ws:
            assert qb.lib().qmoe_fp8_quant_blocks(N, K, 1, w.data_ptr(), K, q.data_ptr(), K, None, 0, s.data_ptr(),
                                                  torch.cuda.current_stream().cuda_stream) == 0
            got.append(qb.fp8_linear(x, q, s, out_dtype=F32))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_fp8_linear_gradient_against_differences():
    # the product of what the codes stand for, along a direction of it: quantisation itself has no gradient
    g = gen(62)
    T, N, K = 24, 40, 72
    x, w, dy = randn(g, T, K), randn(g, N, K, scale=0.1), randn(g, T, N)
    w_q, w_s, wt_q = qb.fp8_quant_blocks(w.cuda(), transposed=True)
    dx, dw = qb.fp8_linear_backward(dy.cuda(), x.cuda(), wt_q, w_s)
    wd, dyr = ref.dequant(*ref.quant(w, 128)), ref.dequant(*ref.quant(dy, 1))
    a, b, _ = _directional(lambda v: ((v @ wd.t()) * dyr).sum(), [f64(x)], [dx], 63)
    assert abs(a - b) <= 1e-4 * float(dx.double().norm().cpu()) * 8
    dyc, xc = ref.dequant(*ref.quant(dy.t().contiguous(), 1)).t(), ref.dequant(*ref.quant(x.t().contiguous(), 1)).t()
    a, b, _ = _directional(lambda v: ((xc @ v.t()) * dyc).sum(), [f64(w)], [dw], 64)
    assert abs(a - b) <= 1e-4 * float(dw.double().norm().cpu()) * 8


# ------------------------------------------------------------------ streams and refusals that need tensors

def test_calls_on_another_stream():
    g = gen(71)
    x, w = randn(g, 64, 256).cuda(), torch.ones(256).cuda()
    w_q, w_s = qb.fp8_quant_blocks(randn(g, 128, 256).cuda())
    want = qb.fp8_linear(qb.norm_pre(x, w)[0], w_q, w_s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n, _ = qb.norm_pre(x, w, stream=side)
    y = qb.fp8_linear(n, w_q, w_s, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_graph_capture():
    g = gen(72)
    x, w, lg = randn(g, 16, 256).cuda(), torch.ones(256).cuda(), randn(g, 16, 64).cuda()
    w_q, w_s = qb.fp8_quant_blocks(randn(g, 256, 256).cuda())

    def step():
        n, _ = qb.norm_pre(x, w)
        r = qb.route_topk(lg, 4, coef=1.0)
        return qb.norm_post(x, qb.fp8_linear(n, w_q, w_s), w=w, w_next=w)[1], r.loss

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_first_fp8_call_in_a_graph_capture_is_refused(monkeypatch):
    # the word where a product reports is made by the first call outside a capture, or by status_word; a capture goes on
    # after the refusal
    g = gen(73)
    x, w = randn(g, 16, 256).cuda(), torch.ones(256).cuda()
    w_q, w_s = qb.fp8_quant_blocks(randn(g, 128, 256).cuda())
    x_q, x_s = qb.fp8_quant_rows(x)
    want, n_want = qb.fp8_linear(x, w_q, w_s), qb.norm_pre(x, w)[0]
    own = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(qb, "_status_words", {})
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            n, _ = qb.norm_pre(x, w)
            with pytest.raises(qb.QmoeError, match="status_word"):
                qb.fp8_linear(x, w_q, w_s)
            with pytest.raises(qb.QmoeError, match="status_word"):
                qb.fp8_matmul(x_q, x_s, w_q, w_s)
            with pytest.raises(qb.QmoeError, match="status_word"):
                qb.status_word("cuda")
            y = qb.fp8_linear(x, w_q, w_s, dev_status=own)  # with a word of its own a call is captured
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, n_want) and torch.equal(y, want) and int(own) == 0
        qb.status_word("cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = qb.fp8_linear(x, w_q, w_s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_refusals_of_tensors():
    x, w = torch.zeros(4, 64).cuda(), torch.ones(64).cuda()
    with pytest.raises(ValueError):
        qb.norm_pre(x, w[:-1])
    with pytest.raises(ValueError):
        qb.norm_pre(x.double(), w)
    with pytest.raises(qb.QmoeError):
        qb.norm_pre(x.t(), torch.ones(4).cuda())
    with pytest.raises(qb.QmoeError):
        qb.norm_pre(x.cpu(), w)
    with pytest.raises(qb.QmoeError, match="-1"):
        qb.norm_pre(x.to(BF16), w, out_dtype=F32)  # a 32-bit block in a 16-bit stream
    with pytest.raises(ValueError):
        qb.norm_post(x, x, gate=torch.ones(3).cuda())
    with pytest.raises(ValueError):
        qb.norm_post_backward(None, x)
    with pytest.raises(qb.QmoeError, match="-1"):
        qb.route_topk(x, 65)
    with pytest.raises(qb.QmoeError, match="-2"):
        qb.route_topk(torch.zeros(2, 1025).cuda(), 2)
    r = qb.route_topk(x, 2)
    with pytest.raises(ValueError):
        qb.route_topk_backward(x, r)
    with pytest.raises(ValueError):
        qb.route_topk_backward(x, r, dloss=torch.ones(1).cuda())
    q, s = qb.fp8_quant_rows(x)
    with pytest.raises(ValueError):
        qb.fp8_matmul(q, s, q[:, :32], s)
    with pytest.raises(ValueError):
        qb.fp8_matmul(q, s[:3], q, s)
    with pytest.raises(ValueError):
        qb.fp8_matmul(x, s, q, s)
    with pytest.raises(qb.QmoeError, match="-1"):  # codes off the 16-byte boundary
        qb.fp8_matmul(torch.zeros(4, 80, dtype=torch.uint8).cuda()[:, 1:65], s, q, s)
    with pytest.raises(qb.QmoeError, match="-1"):
        qb.fp8_matmul(torch.zeros(4, 72, dtype=torch.uint8).cuda()[:, :64], s, q, s)


# ------------------------------------------------------------------ together

def test_block_example_gradients():
    """examples/moe_block.py: the operators together.  A small step along the gradients changes the loss as they say; the
    routed experts' output and the codes' rounding stay as they are along it, so the step goes through the norms, the gate
    and the balance loss, whose gradients do not pass through them."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    block = m.MoeBlock(H=256, I=128, E=8, k=2, seed=3)
    g = gen(91)
    r = randn(g, 40, 256, dtype=BF16).cuda()
    mask = (torch.rand(40, generator=g) < 0.8).cuda()
    dout, dn = randn(g, 40, 256, dtype=BF16, scale=0.1).cuda(), randn(g, 40, 256, dtype=BF16, scale=0.1).cuda()
    out, n_next, s = block.forward(r, mask=mask, coef=0.5)
    dx, grads, route = block.train_step(r, dout, dn, coef=0.5, mask=mask)
    assert dx.shape == r.shape and all(torch.isfinite(t).all() for t in grads.values())
    assert int(route.counts[-1]) == int(mask.sum()) and torch.equal(route.counts, s["route"].counts)
    # the norms and the gate against the 64-bit block end on the same y
    y = f64(s["y"].cpu()).requires_grad_()
    leaves = [f64(t.cpu()).requires_grad_() for t in (block.w_out, block.gate, block.w_next)]
    o, n = ref.post(f64(r.cpu()), y, leaves[0], leaves[1], block.alpha, leaves[2], m.EPS)
    c = (256 / 128 + 56) * U
    ref.close(out, o.detach(), c * (f64(r.cpu()).abs() + (o.detach() - f64(r.cpu())).abs()), "out")
    want = torch.autograd.grad((o * f64(dout.cpu())).sum() + (n * f64(dn.cpu())).sum(), leaves)
    for name, got, w in zip(("w_out", "gate", "w_next"), (grads["w_out"], grads["gate"], grads["w_next"]), want):
        # out is rounded to bf16 before the gradient reads it: 2^-8 of each of the 40 terms, of random signs
        assert float((got.cpu().double() - w).norm() / w.norm()) < 2.0 ** -7, name
    # one token is served as it is in the batch (quantised row by row)
    one = block.forward(r[:1], mask=mask[:1])[0]
    assert torch.allclose(one.float(), out[:1].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    # the shared expert's second product, whose gradient is the formula on what the codes stand for
    dy = qb.norm_post_backward(dout, s["y"], w=block.w_out, rstd=s["rstd"], gate=block.gate, alpha=block.alpha, dn=dn, out=out,
                               w_next=block.w_next, rstd_next=s["rstd_next"])[1].cpu()
    a = s["a"].cpu()
    want, slack = ref.product(ref.dequant(*ref.quant(dy.t().contiguous(), 1)), ref.dequant(*ref.quant(a.t().contiguous(), 1)))
    ref.close(grads["w2"], want, slack, "w2")
    assert int(qb.status_word("cuda")) == 0
