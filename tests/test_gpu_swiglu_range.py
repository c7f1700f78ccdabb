"""GPU tests of SwiGLU and its gradient at the ends of the range: gates whose sigmoid is among fp32's least values, and products
whose factors do not fit together though they do.  Against 64 bits; the bound of fp32's steps is test_swiglu's."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from tests import expert_ref as ref
from tests.block_ref import close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def rows(gates, up, I, dtype):
    """[g, u] with the gates by turns and u of that size."""
    g = torch.Generator().manual_seed(I)
    gate = torch.tensor(gates)[torch.arange(3 * I) % len(gates)].view(3, I)
    u = (torch.randn(3, I, generator=g).sign() * (0.5 + torch.rand(3, I, generator=g))) * up
    return torch.cat([gate, u], 1).to(dtype)


def err(gu, I, dtype):
    v = gu[:, :I].double().abs()
    return (10 + 3 * v + (0.0 if dtype == F32 else 4.0)) * U


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("I", [64, 65, 66])
def test_gates_about_the_least_sigmoid(I, dtype):
    """Gates from -89 to -86, up values that bring the result back among ordinary numbers: 1 + e^88 is above 2^126."""
    gu = rows([-86.0, -87.0, -87.25, -87.5, -88.0, -88.5, -88.75, -89.0], 1e30, I, dtype)
    want = ref.swiglu(gu.double())
    e = err(gu, I, dtype) + 2.0 ** -18  # a sigmoid of 2^-129 has 20 bits left, the last two of them in doubt
    h = qb.swiglu(gu.cuda())
    close(h, want, e * want.abs(), "h")
    dh = torch.ones(3, I).to(dtype)
    dgu, again = qb.swiglu_backward(dh.cuda(), gu.cuda(), h_too=True)
    assert torch.equal(again, h)
    leaf = gu.double().requires_grad_()
    grad, = torch.autograd.grad(ref.swiglu(leaf), leaf, dh.double())
    close(dgu, grad, 2 * torch.cat([e, e], 1) * grad.abs() + 2.0 ** -149, "dgu")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("I", [64, 65, 66])
def test_large_gradients_of_closed_gates(I, dtype):
    """dh u is 10^50, the gate's factor brings it back."""
    gu = rows([-60.0, -70.0, -80.0, -86.0], 1e25, I, dtype)
    dh = (torch.ones(3, I) * 1e25).to(dtype)
    dgu, _ = qb.swiglu_backward(dh.cuda(), gu.cuda())
    leaf = gu.double().requires_grad_()
    grad, = torch.autograd.grad(ref.swiglu(leaf), leaf, dh.double())
    assert grad.abs().max() < 1e38
    e = err(gu, I, dtype)
    close(dgu, grad, 2 * torch.cat([e, e], 1) * grad.abs(), "dgu")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_infinite_gates(dtype):
    """silu(+inf) is +inf; -inf times 0 is NaN, as by the formula; NaN stays NaN."""
    gu = torch.tensor([[float("inf"), float("-inf"), float("nan"), 200.0, -200.0, 0.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0]]).to(dtype)
    h = qb.swiglu(gu.cuda()).cpu()[0]
    assert h[0] == float("inf") and h[1].isnan() and h[2].isnan() and h[3] == 1000.0 and h[4] == 0 and h[5] == 0
