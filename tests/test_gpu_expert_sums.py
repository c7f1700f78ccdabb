"""GPU tests of long sums in the experts' products: the tensor core cuts a sum off where fp32 would round it, always
downwards, so sums are made in pieces of at most 2048 values that are added with fp32's rounding.

Tolerance, of the sum of the magnitudes: a piece is cut off once for each 16 values, by 2^-23 at most each time, and a few
times more where the products of a step are aligned; then half a step of fp32 for each piece that is added (`adds` of them at
most).  It does not grow with the pieces' own length, so that two sums of 16384 positive values, which lose 5e-5, fail."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def bound(adds):
    return (2048 / 16 + 8) * 2.0 ** -23 + adds * 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def positive(g, *shape, dtype=BF16):
    return torch.rand(*shape, generator=g, device="cuda", dtype=dtype) + 0.5


def offsets_of(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).int()


def near(got, want, size, adds, what):
    off = ((got.double() - want).abs() / size.clamp(min=1e-30)).max().item()
    assert off <= bound(adds), f"{what}: {off:.3g} of the magnitudes off, {bound(adds):.3g} allowed"


def status():
    return int(qb.status_word("cuda").item())


# rows, outputs, length of the sum, fp32 additions: tiles of two CTAs; of one, whole and shared by the SMs, for up to 96 rows
# and for up to 16
LONG = [(300, 64, 65536, 40), (50, 39168, 32768, 40), (5, 39168, 32768, 40), (50, 128, 1 << 20, 200), (5, 128, 1 << 20, 200)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("P,N,K,adds", LONG)
def test_long_sums_of_y(P, N, K, adds, gather):
    g = gen(P + N)
    x, w = positive(g, P, K), positive(g, 1, N, K)
    pairs = torch.randperm(P, generator=g, device="cuda").int() if gather else None
    y = qb.expert_linear(x, w, offsets_of([P]), pairs=pairs, k=1, out_dtype=F32)
    some = torch.randint(0, N, (48,), generator=g, device="cuda")
    want = (x if pairs is None else x[pairs.long()]).double() @ w[0, some].double().t()
    near(y[:, some], want, want, adds, "y")
    assert status() == 0


@pytest.mark.parametrize("P,K,N,adds", LONG)
def test_long_sums_of_dx(P, K, N, adds):
    """The gradient has the products' type, which rounds more than its sum is off: the mean over its values has not."""
    g = gen(P + N + 1)
    dy, w = positive(g, P, N, dtype=F16) / N, positive(g, 1, N, K, dtype=F16)
    dx, _ = qb.expert_linear_backward(dy, torch.empty(P, K, device="cuda", dtype=F16), w, offsets_of([P]), need_dw=False)
    some = torch.randperm(K, generator=g, device="cuda")[:2000]
    want = dy.double() @ w[0][:, some].double()
    # a rounding to 11 bits, by up to 2^-11, has no sign: the mean of n of them is off by 2^-11 / sqrt(3 n) in the mean square,
    # and by five times that at most
    n = want.numel()
    off = ((dx[:, some].double() - want) / want).mean().abs().item()
    assert off <= bound(adds) + 5 * 2.0 ** -11 / (3 * n) ** 0.5, f"dx: {off:.3g} off in the mean"
    assert status() == 0


@pytest.mark.parametrize("P,N,K", [(2, 16, 131073), (1, 7, 131071)])
def test_long_sums_of_odd_rows(P, N, K):
    """Weights off the 16-byte boundaries, read as they lie."""
    g = gen(K)
    x, w = positive(g, P, K), positive(g, 1, N, K)
    y = qb.expert_linear(x, w, offsets_of([P]), out_dtype=F32)
    want = x.double() @ w[0].double().t()
    near(y, want, want, 160, "y")


@pytest.mark.parametrize("counts", [[65536], [3, 70001, 0, 900], [30900] + [1] * 1000, [9] * 300 + [22001] + [0] * 600])
@pytest.mark.parametrize("gather", [False, True])
def test_long_sums_of_dw(counts, gather):
    """One expert has almost all rows; the last two are stored by TMA, as most experts have few."""
    g = gen(len(counts))
    P, N, K, offsets = sum(counts), 64, 72, offsets_of(counts)
    dy, x = positive(g, P, N), positive(g, P, K)
    pairs = torch.randperm(P, generator=g, device="cuda").int() if gather else None
    _, dw = qb.expert_linear_backward(dy, x, torch.empty(len(counts), N, K, device="cuda", dtype=BF16), offsets, pairs=pairs, k=1, need_dx=False)
    rows = x if pairs is None else x[pairs.long()]
    o = offsets.tolist()
    for e in sorted(range(len(counts)), key=lambda e: -counts[e])[:3]:
        want = dy[o[e]:o[e + 1]].double().t() @ rows[o[e]:o[e + 1]].double()
        near(dw[e], want, want, 40, f"dw of expert {e}")
    assert status() == 0


# ------------------------------------------------------------------ many tiles, each of several pieces

def by_expert(f, *tensors, offsets):
    o = offsets.tolist()
    return [f(e, *(t[o[e]:o[e + 1]].double() for t in tensors)) for e in range(len(o) - 1)]


@pytest.mark.parametrize("steps", [31, 32, 33, 64, 65, 97, 130])
@pytest.mark.parametrize("E,least,most", [(60, 97, 400), (100, 17, 96), (300, 1, 16), (150, 1, 60)])
def test_pieces_of_many_tiles(E, least, most, steps):
    """Rows of many experts, more tiles than SMs, and sums of one piece, of whole ones, and with a short last one."""
    g = gen(E + steps)
    counts = torch.randint(least, most + 1, (E,), generator=torch.Generator().manual_seed(steps)).tolist()
    counts[3] = 0
    P, L, M, offsets = sum(counts), 64 * steps - 24, 264, offsets_of(counts)
    x = torch.randn(P, L, generator=g, device="cuda").to(BF16)
    w = torch.randn(E, M, L, generator=g, device="cuda").to(BF16)
    pairs = torch.randperm(P, generator=g, device="cuda").int()
    rows = x[pairs.long()]
    for got, xs in ((qb.expert_linear(x, w, offsets, out_dtype=F32), x), (qb.expert_linear(x, w, offsets, pairs=pairs, k=1, out_dtype=F32), rows)):
        want = torch.cat(by_expert(lambda e, a: a @ w[e].double().t(), xs, offsets=offsets))
        size = torch.cat(by_expert(lambda e, a: a.abs() @ w[e].double().abs().t(), xs, offsets=offsets))
        near(got, want, size, 16, "y")
    wt = w.transpose(1, 2).contiguous()  # [E, L, M]: the same sums, as a gradient
    dx, _ = qb.expert_linear_backward(x, torch.empty(P, M, device="cuda", dtype=BF16), wt, offsets, need_dw=False)
    want = torch.cat(by_expert(lambda e, a: a @ w[e].double().t(), x, offsets=offsets))
    size = torch.cat(by_expert(lambda e, a: a.abs() @ w[e].double().abs().t(), x, offsets=offsets))
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + bound(16) * size).all()
    assert status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,most", [(12, 6000), (40, 1500), (500, 40)])
def test_pieces_of_dw(E, most, dtype):
    """Experts of no row, of one, of whole steps and pieces, and of any number; several tiles a pair of CTAs."""
    g = gen(E)
    counts = torch.randint(0, most + 1, (E,), generator=torch.Generator().manual_seed(E)).tolist()
    counts[:6] = [0, 1, 2048, 4096, 64, 2049]
    P, N, K, offsets = sum(counts), 328, 520, offsets_of(counts)
    dy, x = (torch.randn(P, n, generator=g, device="cuda").to(F16 if dtype == F32 else BF16) for n in (N, K))
    w = torch.empty(E, N, K, device="cuda", dtype=x.dtype)
    _, dw = qb.expert_linear_backward(dy, x, w, offsets, need_dx=False, dw_dtype=dtype)
    wants = by_expert(lambda e, a, b: (a.t() @ b, a.abs().t() @ b.abs()), dy, x, offsets=offsets)
    for e, (want, size) in enumerate(wants):
        assert ((dw[e].double() - want).abs() <= (2.0 ** -24 if dtype == F32 else 2.0 ** -8 * 1.01) * want.abs() + bound(16) * size).all(), e
    assert status() == 0


@pytest.mark.parametrize("P", [32, 33, 64, 65, 100, 128, 129, 192, 193])
@pytest.mark.parametrize("N,K", [(264, 2120), (20040, 320)])
def test_one_matrix(P, N, K):
    """Rows of one matrix about the tiles' widths, its few tiles shared by the SMs or more tiles than SMs."""
    g = gen(P + N)
    x, w = (torch.randn(*s, generator=g, device="cuda").to(BF16) for s in ((P, K), (1, N, K)))
    offsets = offsets_of([P])
    pairs = torch.randperm(P, generator=g, device="cuda").int()
    for got, rows in ((qb.expert_linear(x, w, offsets, out_dtype=F32), x), (qb.expert_linear(x, w, offsets, pairs=pairs, k=1, out_dtype=F32), x[pairs.long()])):
        near(got, rows.double() @ w[0].double().t(), rows.double().abs() @ w[0].double().abs().t(), 16, "y")
    wt = w.transpose(1, 2).contiguous()
    dx, _ = qb.expert_linear_backward(x, None, wt, offsets, need_dw=False)
    want, size = x.double() @ w[0].double().t(), x.double().abs() @ w[0].double().abs().t()
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + bound(16) * size).all()
    assert status() == 0
