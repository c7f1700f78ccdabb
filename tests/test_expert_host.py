"""CPU checks of the experts' products, SwiGLU, the weighted sum and the 4-bit products: what their C entry points refuse
before any launch (no GPU is touched), their workspace sizes, and that the tests' 64-bit forms notice a planted mistake."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from quantized_mixture_experts_moe_gb300 import build as qbuild
from tests import expert_ref as ref

ARG, UNSUPPORTED, OK = -1, -2, 0
A = 1 << 20  # an aligned address that is never read: every call here ends before a launch
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qb.lib()


def with_(base, **changes):
    d = dict(base)
    d.update(changes)
    return tuple(d.values())


LINEAR = dict(P=40, E=4, N=64, K=128, dt=1, x=A, ldx=128, x_rows=40, pairs=None, k=1, w=A, ldw=128, w_e=64 * 128, off=A, y=A, yt=1, ldy=64,
              st=A, ws=A, wsn=1 << 30, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(P=-1), ARG), (dict(E=0), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(dt=0), ARG), (dict(dt=3), ARG), (dict(yt=2), ARG),
    (dict(yt=7), ARG), (dict(x=None), ARG), (dict(x=A + 1), ARG), (dict(ldx=127), ARG), (dict(w=None), ARG), (dict(ldw=127), ARG),
    (dict(w_e=64 * 128 - 1), ARG), (dict(off=None), ARG), (dict(off=A + 2), ARG), (dict(y=None), ARG), (dict(y=A + 1), ARG),
    (dict(ldy=63), ARG), (dict(st=None), ARG), (dict(st=A + 2), ARG), (dict(yt=0, y=A + 2), ARG), (dict(pairs=A, k=0), ARG),
    (dict(pairs=A, x_rows=-1), ARG), (dict(pairs=A + 1), ARG), (dict(pairs=A, x_rows=0), ARG), (dict(P=BIG), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(N=BIG, ldy=BIG, w_e=BIG * 128), UNSUPPORTED), (dict(K=BIG, ldx=BIG, ldw=BIG, w_e=BIG * 64), UNSUPPORTED),
    (dict(pairs=A, x_rows=BIG), UNSUPPORTED), (dict(P=0, x=None, y=None), OK)])
def test_expert_linear_refuses(lib, change, want):
    assert lib.qmoe_expert_linear(*with_(LINEAR, **change)) == want


def test_expert_linear_needs_its_workspace(lib):
    # many rows an expert: x laid out in expert order; a w off the 16-byte boundaries: its copy
    many = dict(LINEAR, P=4000, x_rows=1000, pairs=A, k=4)
    need = lib.qmoe_expert_workspace_bytes(4000, 4, 64, 128, 0, 1)
    assert need == lib.qmoe_expert_copy_bytes(4000, 128) == 4000 * 128 * 2
    for change in (dict(ws=None), dict(wsn=need - 1), dict(ws=A + 16)):
        assert lib.qmoe_expert_linear(*with_(many, **change)) == ARG
    odd = dict(LINEAR, P=4000, ldw=129, w_e=64 * 129)
    assert lib.qmoe_expert_workspace_bytes(4000, 4, 64, 128, 0, 0) == 0
    for change in (dict(ws=None), dict(wsn=lib.qmoe_expert_copy_bytes(256, 128) - 1), dict(ws=A + 8)):
        assert lib.qmoe_expert_linear(*with_(odd, **change)) == ARG
    # few tiles: the sums of those that several CTAs share
    assert lib.qmoe_expert_workspace_bytes(1, 1, 4096, 4096, 0, 0) > 0
    assert lib.qmoe_expert_linear(*with_(LINEAR, P=1, E=1, N=4096, K=4096, ldx=4096, ldw=4096, w_e=4096 * 4096, ldy=4096, ws=None, wsn=0)) == ARG


def test_expert_workspace_sizes(lib):
    f = lib.qmoe_expert_workspace_bytes
    for bad in ((0, 1, 1, 1, 0, 0), (1, 0, 1, 1, 0, 0), (1, 1, 0, 1, 0, 0), (1, 1, 1, 0, 0, 0), (1, 1, 1, 1, 3, 0), (1, 1, 1, 1, -1, 0), (BIG, 1, 1, 1, 0, 1)):
        assert f(*bad) == 0
    assert f(100, 1, 64, 65, 2, 0) == 0 and f(100, 1, 64, 65, 2, 1) == lib.qmoe_expert_copy_bytes(100, 65) == (100 * 72 * 2 + 255) // 256 * 256
    assert f(4000, 4, 64, 128, 1, 0) == 0
    assert lib.qmoe_expert_copy_bytes(0, 8) == 0 == lib.qmoe_expert_copy_bytes(8, -1)


def test_expert_gradients_refuse(lib):
    dx = dict(P=40, E=4, N=64, K=128, dt=1, dy=A, lddy=64, w=A, ldw=128, w_e=64 * 128, off=A, dx=A, dxt=1, lddx=128, st=A, ws=None, wsn=0,
              stream=None)
    for change in (dict(P=-1), dict(dt=0), dict(dxt=2), dict(dy=None), dict(lddy=63), dict(w=None), dict(ldw=1), dict(off=None), dict(dx=None),
                   dict(lddx=127), dict(st=None), dict(dy=A + 1), dict(dxt=0, dx=A + 2)):
        assert lib.qmoe_expert_linear_dx(*with_(dx, **change)) == ARG, change
    assert lib.qmoe_expert_linear_dx(*with_(dx, E=2000)) == UNSUPPORTED
    assert lib.qmoe_expert_linear_dx(*with_(dx, P=0, dy=None, dx=None)) == OK
    dw = dict(P=40, E=4, N=64, K=128, dt=1, dy=A, lddy=64, x=A, ldx=128, x_rows=40, pairs=None, k=1, off=A, dw=A, dwt=0, st=A, ws=None, wsn=0,
              stream=None)
    for change in (dict(P=-1), dict(dt=0), dict(dwt=2), dict(dy=None), dict(lddy=63), dict(x=None), dict(ldx=1), dict(off=None), dict(dw=None),
                   dict(st=None), dict(dw=A + 2), dict(pairs=A, k=-1), dict(pairs=A, k=2, ws=None), dict(pairs=A, k=2, x_rows=0)):
        assert lib.qmoe_expert_linear_dw(*with_(dw, **change)) == ARG, change
    assert lib.qmoe_expert_linear_dw(*with_(dw, E=1025)) == UNSUPPORTED


def test_swiglu_refuses(lib):
    f = dict(rows=4, I=64, dt=1, gu=A, ldgu=128, h=A, ldh=64, stream=None)
    for change in (dict(rows=-1), dict(I=0), dict(dt=4), dict(gu=None), dict(ldgu=127), dict(h=None), dict(ldh=63), dict(gu=A + 1), dict(dt=0, h=A + 2)):
        assert lib.qmoe_swiglu(*with_(f, **change)) == ARG, change
    assert lib.qmoe_swiglu(*with_(f, rows=0, gu=None, h=None)) == OK and lib.qmoe_swiglu(*with_(f, rows=BIG)) == UNSUPPORTED
    b = dict(rows=4, I=64, dt=1, dh=A, lddh=64, gu=A, ldgu=128, dgu=A, lddgu=128, h=None, ldh=0, stream=None)
    for change in (dict(rows=-1), dict(I=0), dict(dt=-1), dict(dh=None), dict(lddh=63), dict(gu=None), dict(ldgu=64), dict(dgu=None), dict(lddgu=1),
                   dict(h=A, ldh=63), dict(h=A + 1, ldh=64)):
        assert lib.qmoe_swiglu_backward(*with_(b, **change)) == ARG, change
    assert lib.qmoe_swiglu_backward(*with_(b, rows=0)) == OK


def test_weighted_sum_refuses(lib):
    f = dict(T=4, k=2, P=8, H=64, dt=1, y=A, ldy=64, w=A, slot=A, out=A, ldo=64, stream=None)
    for change in (dict(T=-1), dict(k=0), dict(P=-1), dict(H=0), dict(dt=3), dict(y=None), dict(ldy=63), dict(slot=None), dict(slot=A + 2), dict(out=None),
                   dict(ldo=63), dict(w=A + 1)):
        assert lib.qmoe_weighted_sum(*with_(f, **change)) == ARG, change
    assert lib.qmoe_weighted_sum(*with_(f, T=0, y=None, out=None, slot=None)) == OK
    for change in (dict(P=BIG), dict(T=1 << 30, k=2), dict(H=BIG, ldy=BIG, ldo=BIG)):
        assert lib.qmoe_weighted_sum(*with_(f, **change)) == UNSUPPORTED, change
    b = dict(T=4, k=2, P=8, H=64, dt=1, dout=A, lddout=64, y=A, ldy=64, w=A, slot=A, routed=A, dy=A, lddy=64, dw=A, stream=None)
    for change in (dict(T=-1), dict(dout=None), dict(lddout=1), dict(y=None), dict(dw=None), dict(ldy=63), dict(slot=None), dict(routed=None),
                   dict(routed=A + 1), dict(dy=None), dict(lddy=63), dict(dw=A + 2)):
        assert lib.qmoe_weighted_sum_backward(*with_(b, **change)) == ARG, change
    assert lib.qmoe_weighted_sum_backward(*with_(b, T=0, P=0, dy=None)) == OK


W4 = dict(T=4, k=1, E=1, N=64, K=128, fmt=0, group=32, dt=1, x=A, ldx=128, w=A, s=A, ids=None, y=A, yt=1, ldy=64, st=A, ws=None, wsn=0, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(K=96, group=64), ARG), (dict(K=100), ARG), (dict(fmt=2), ARG), (dict(group=16), ARG),
    (dict(fmt=1, group=64), ARG), (dict(dt=0), ARG), (dict(yt=2), ARG), (dict(ldy=63), ARG), (dict(k=2), ARG), (dict(E=2), ARG), (dict(x=None), ARG),
    (dict(x=A + 1), ARG), (dict(ldx=127), ARG), (dict(w=None), ARG), (dict(w=A + 8), ARG), (dict(s=None), ARG), (dict(s=A + 1), ARG), (dict(y=None), ARG),
    (dict(st=None), ARG), (dict(T=17), ARG), (dict(ids=A + 2, k=2, E=8), ARG), (dict(ids=A, k=0, E=8), ARG), (dict(ids=A, k=20000, E=8), UNSUPPORTED),
    (dict(T=BIG), UNSUPPORTED), (dict(T=0, x=None, y=None), OK)])
def test_w4_linear_refuses(lib, change, want):
    assert lib.qmoe_w4_linear(*with_(W4, **change)) == want


def test_w4_workspace_and_gradient(lib):
    f = lib.qmoe_w4_workspace_bytes
    assert f(16, 64, 128, 0) == 0 == f(0, 64, 128, 1) and f(17, 64, 128, 0) >= 64 * 128 * 2 and f(1, 64, 128, 1) >= 64 * 128 * 2
    need = f(20, 64, 128, 0)
    for change in (dict(ws=A, wsn=need - 1), dict(ws=A + 16, wsn=need), dict(ws=None, wsn=need)):
        assert lib.qmoe_w4_linear(*with_(W4, T=20, **change)) == ARG
    need = f(4, 64, 128, 1)
    dx = dict(T=4, N=64, K=128, fmt=0, group=32, dt=1, dy=A, lddy=64, w=A, s=A, dx=A, dxt=1, lddx=128, st=A, ws=A, wsn=need, stream=None)
    for change in (dict(T=-1), dict(group=31), dict(dt=0), dict(dxt=2), dict(dy=None), dict(lddy=63), dict(w=None), dict(s=None), dict(dx=None), dict(lddx=127),
                   dict(st=None), dict(ws=None), dict(wsn=need - 1), dict(ws=A + 128)):
        assert lib.qmoe_w4_linear_dx(*with_(dx, **change)) == ARG, change
    assert lib.qmoe_w4_linear_dx(*with_(dx, T=0)) == OK


# ------------------------------------------------------------------ the 64-bit forms

def case():
    g = torch.Generator().manual_seed(0)
    off = torch.tensor([0, 3, 3, 8], dtype=torch.int32)
    return (torch.randn(9, 5, generator=g, dtype=torch.float64), torch.randn(3, 4, 5, generator=g, dtype=torch.float64),
            torch.randn(9, 4, generator=g, dtype=torch.float64), off)


def test_forms_agree_with_autograd():
    x, w, dy, off = case()
    x.requires_grad_(), w.requires_grad_()
    y = torch.stack([w[e] @ x[s] if s < 8 else torch.zeros(4, dtype=torch.float64) for s, e in enumerate([0, 0, 0, 2, 2, 2, 2, 2, 0])])
    assert torch.allclose(ref.linear(x, w, off)[0], y, rtol=1e-12, atol=0)
    gx, gw = torch.autograd.grad(y, (x, w), dy)
    assert torch.allclose(ref.linear_dx(dy, w, off)[0], gx, rtol=1e-12, atol=0) and torch.allclose(ref.linear_dw(dy, x, off)[0], gw, rtol=1e-12, atol=0)


@pytest.mark.parametrize("plant", ["an expert late", "a row of none", "the other nibble", "an offset of 7", "up and gate exchanged"])
def test_planted_mistakes_are_noticed(plant):
    x, w, dy, off = case()
    y, slack = ref.linear(x, w, off)
    bound = slack + 2.0 ** -8 * y.abs()
    if plant == "an expert late":
        wrong = ref.linear(x, w, torch.tensor([0, 4, 4, 8], dtype=torch.int32))[0]
    elif plant == "a row of none":
        wrong = ref.linear(x, w, torch.tensor([0, 3, 3, 9], dtype=torch.int32))[0]
    elif plant == "up and gate exchanged":
        gu = torch.cat([x, dy[:, :1].expand(9, 5)], 1)
        y, wrong, bound = ref.swiglu(gu), ref.swiglu(torch.cat([gu[:, 5:], gu[:, :5]], 1)), 1e-3
    else:
        g = torch.Generator().manual_seed(1)
        q = torch.randint(0, 256, (4, 32), generator=g, dtype=torch.uint8)
        s = torch.full((4, 2), 0.01).half()
        y = ref.codes4(q, s)
        wrong = ref.codes4(q >> 4 | (q & 15) << 4, s) if plant == "the other nibble" else y + 0.01
        bound = 1e-4
    assert ((wrong - y).abs() > bound).any()
