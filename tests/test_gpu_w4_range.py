"""GPU tests of 4-bit products that widen their weights (more than 16 tokens, and the gradient) beside those that do not: scales
anywhere in their type, weights that leave fp16's range, infinities and NaN.  Against 64 bits, with tests/expert_ref.py's bounds."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from tests import expert_ref as ref
from tests.block_ref import close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g).to(dtype)


def e2m1(g, N, K, low, high):
    return torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8), torch.randint(low, high + 1, (N, K // 32), generator=g, dtype=torch.uint8)


def slack_of(x, s, w, K):
    """Of y: sums of groups for few tokens (some more than 16 for int4); else of the products, for int4 of two matrices'."""
    few, many = ref.w4_slack(x.double(), w, s, K), (x.double().abs() @ w.abs().t()) * ref.sums(2 * K)
    return few if x.shape[0] <= 16 else torch.maximum(few, many) if x.shape[0] <= 32 else many


def product(x, q, s, w, K):
    """y in 32 bits against 64."""
    y = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32)
    close(y, x.double() @ w.t(), slack_of(x, s, w, K), "y")


def gradient(dy, q, s, w, N):
    """The gradient, which has dy's type: dy is as small as keeps it there.  What fp16 loses below 2^-25 is no error."""
    dx = qb.w4_linear_backward(dy.cuda(), q.cuda(), s.cuda())
    close(dx, dy.double() @ w, (dy.double().abs() @ w.abs()) * ref.sums(2 * N), "dx")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [17, 60, 300])
@pytest.mark.parametrize("low,high", [(85, 95), (140, 146), (98, 106), (119, 123)])
def test_e2m1_scales_beyond_fp16(T, low, high, dtype):
    """Scales whose values leave fp16 upwards, vanish in it, or lie among its subnormals."""
    g = gen(T + low)
    N, K = 72, 320
    q, s = e2m1(g, N, K, low, high)
    w, x = ref.codes4(q, s), randn(g, T, K, dtype=dtype)
    product(x, q, s, w, K)
    few = qb.w4_linear(x[:16].cuda(), q.cuda(), s.cuda(), out_dtype=F32).cpu().double()
    many = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32)[:16].cpu().double()
    assert float((few - many).norm() / many.norm()) < 1e-5  # the same product, whatever else is in the batch
    if high <= 123:
        dy = randn(g, T, N, dtype=dtype) * (2.0 ** 8 if high < 110 else 1.0)
    else:
        dy = (randn(g, T, N) * 2.0 ** -12).to(dtype)
    gradient(dy, q, s, w, N)


@pytest.mark.parametrize("T", [17, 200])
def test_e2m1_rows_and_columns_of_different_size(T):
    """Each row's, and for the gradient each column's, weights keep their bits beside those of 2^50 times their size."""
    g = gen(T)
    N, K = 96, 256
    q, s = e2m1(g, N, K, 120, 124)
    x, dy = randn(g, T, K, dtype=F16), randn(g, T, N, dtype=F16)
    by_row = s.int() + torch.tensor([-50, 0, 30, -20])[torch.arange(N) % 4][:, None]
    by_col = s.int() + torch.tensor([-8, 0, 9, 3])[torch.arange(K // 32) % 4][None]
    rows, cols = by_row.to(torch.uint8), by_col.to(torch.uint8)
    product(x, q, rows, ref.codes4(q, rows), K)
    product(x, q, cols, ref.codes4(q, cols), K)
    gradient(dy, q, cols, ref.codes4(q, cols), N)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("low,high", [(8191.0, 65504.0), (2.0 ** -24, 2.0 ** -15), (1e-3, 60000.0)])
def test_int4_scales_of_any_size(low, high, group, dtype):
    """Scales up to fp16's largest (8 times which fp16 does not hold) and among its subnormals."""
    g = gen(group)
    T, N, K = 40, 48, 384
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.exp(torch.empty(N, K // group).uniform_(generator=g) * (torch.tensor(high).log() - torch.tensor(low).log()) + torch.tensor(low).log()).half()
    assert s.isfinite().all() and (s > 0).all()
    w, x = ref.codes4(q, s), randn(g, T, K, dtype=dtype)
    product(x, q, s, w, K)
    dy = (randn(g, T, N) * (2.0 ** -16 if high > 1 else 1.0)).to(dtype)
    gradient(dy, q, s, w, N)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,N,K,group", [(17, 40, 2048, 32), (24, 264, 128, 128), (25, 40, 2112, 64), (33, 72, 96, 32), (64, 129, 4096, 128),
                                         (90, 1100, 192, 64), (97, 16, 32, 32), (300, 264, 640, 64), (513, 520, 2304, 128)])
def test_int4_weights_are_not_rounded(T, N, K, group, dtype):
    """Weights of 14 bits rounded to x's type would be up to 2^-9 (bf16) or 2^-12 (fp16) off: outputs in 32 bits show it.  A
    row is the same by itself but for the sums' roundings, and the gradient has no other rounding than its type's."""
    g = gen(T + N)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (0.005 + 0.015 * torch.rand(N, K // group, generator=g)).half()
    w, x, dy = ref.codes4(q, s), randn(g, T, K, dtype=dtype), randn(g, T, N, dtype=dtype)
    product(x, q, s, w, K)
    y = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32).cpu().double()
    one = qb.w4_linear(x[:1].cuda(), q.cuda(), s.cuda(), out_dtype=F32).cpu().double()
    assert float((y[:1] - one).norm() / one.norm()) < 1e-5
    gradient(dy, q, s, w, N)


@pytest.mark.parametrize("T", [17, 20, 24, 25, 32])
def test_rows_of_several_launches(T):
    """Views of x, 17 to 32 tokens: each row is its own."""
    g = gen(T)
    q = torch.randint(0, 256, (48, 64), generator=g, dtype=torch.uint8).cuda()
    s = (0.005 + 0.015 * torch.rand(48, 4, generator=g)).half().cuda()
    base = randn(g, T, 150, dtype=BF16).cuda()
    w = ref.codes4(q.cpu(), s.cpu())
    for a in (0, 1, 8):
        x = base[:, a:a + 128]
        y = qb.w4_linear(x, q, s, out_dtype=F32)
        close(y, x.cpu().double() @ w.t(), slack_of(x.cpu(), s.cpu(), w, 128), "y")
        rows = qb.w4_linear(x[:16], q, s, out_dtype=F32)
        assert float((y[:16] - rows).norm() / rows.norm()) < 1e-5


@pytest.mark.parametrize("T", [3, 16, 17, 100])
def test_e2m1_ends_of_the_scale(T):
    """Bytes 0 and 254 in bf16, which holds all that fp32 does: the least scale's values and 6 x 2^127, by way of a small x."""
    g = gen(T)
    N, K = 24, 128
    q, s = e2m1(g, N, K, 0, 1)
    x = (randn(g, T, K) * 2.0 ** 100).to(BF16)
    w = ref.codes4(q, s)
    product(x, q, s, w, K)
    s = s + 253
    x = (randn(g, T, K) * 2.0 ** -40).to(BF16)
    w = ref.codes4(q, s)
    product(x, q, s, w, K)
    dy = (randn(g, T, N) * 2.0 ** -40).to(BF16)
    gradient(dy, q, s, w, N)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("format", ["int4", "mxfp4"])
@pytest.mark.parametrize("T", [3, 9, 16, 17, 90])
def test_infinities_and_nan_stay_in_their_token(T, format, dtype):
    """A token with an infinity or a NaN has no finite value, in either format and on either side of 16 tokens; the others'
    are what they are without it."""
    g = gen(T)
    N, K = 40, 256
    q, s = e2m1(g, N, K, 119, 125)
    if format == "int4":
        s = (torch.rand(N, K // 32, generator=g) * 0.01 + 0.001).half()
    x = randn(g, T, K, dtype=dtype)
    clean = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32)
    x[1, 7], x[2, 100] = float("inf"), float("nan")
    y = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32)
    assert not y[1].isfinite().any() and y[2].isnan().all()
    rest = torch.tensor([t for t in range(T) if t not in (1, 2)], device="cuda")
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("T", [3, 40])
def test_scales_that_are_no_numbers_stay_in_their_row(T):
    g = gen(T)
    N, K = 20, 128
    q, s = e2m1(g, N, K, 110, 140)
    x = randn(g, T, K, dtype=F16)
    want = ref.codes4(q, s)
    slack = slack_of(x, s, want, K)
    s[5, 2] = 255
    y = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), out_dtype=F32).cpu()
    assert y[:, 5].isnan().all()
    keep = [n for n in range(N) if n != 5]
    close(y[:, keep], (x.double() @ want.t())[:, keep], slack[:, keep], "y")
    h = (torch.rand(N, K // 64, generator=g) * 0.01).half()
    want = ref.codes4(q, h)
    slack = slack_of(x, h, want, K)
    h[3, 1], h[7, 0] = float("inf"), float("nan")
    y = qb.w4_linear(x.cuda(), q.cuda(), h.cuda(), out_dtype=F32).cpu()
    assert not y[:, 3].isfinite().any() and y[:, 7].isnan().all()
    keep = [n for n in range(N) if n not in (3, 7)]
    close(y[:, keep], (x.double() @ want.t())[:, keep], slack[:, keep], "y")


@pytest.mark.parametrize("format", ["int4", "mxfp4"])
@pytest.mark.parametrize("T,k,E", [(33, 8, 8), (64, 8, 20), (257, 1, 5), (100, 5, 3), (2, 300, 8), (5, 256, 4), (7, 129, 9)])
def test_more_pairs_than_a_launch_sorts(T, k, E, format):
    """Tokens by 256 pairs, and pair by pair where a token has more than that: every pair's row is what its token's call by
    itself gives, whatever stands beside it."""
    g = gen(T + k)
    N, K = 72, 288
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = (0.005 + 0.015 * torch.rand(E, N, K // 32, generator=g)).half() if format == "int4" else torch.randint(118, 124, (E, N, K // 32), generator=g, dtype=torch.uint8)
    x = randn(g, T, K, dtype=BF16)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).int()
    y = qb.w4_linear(x.cuda(), q.cuda(), s.cuda(), ids=ids.cuda(), out_dtype=F32).cpu()
    assert y.shape == (T * k, N)
    w = ref.codes4(q, s)
    token = torch.arange(T * k) // k
    for e in range(E):
        mine = (ids.view(-1) == e).nonzero().view(-1)
        rows = x[token[mine]].double()
        close(y[mine], rows @ w[e].t(), ref.w4_slack(rows, w[e], s[e], K), f"expert {e}")
    assert (y[(ids.view(-1) < 0) | (ids.view(-1) >= E)] == 0).all()
