"""GPU tests of what the calls around the experts' products ask for: workspaces, operands that one gradient does not need,
refusals."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from tests import expert_ref as ref
from tests.block_ref import close

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def offsets_of(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).int()


def randn(seed, *shape, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_few_rows_beside_odd_weights_take_no_copy_of_them():
    """One token on all experts' odd weights, which are read as they lie: 66 MB would be the copy that nobody writes."""
    E, N, K = 32, 511, 2047
    w, x = randn(1, E, N, K), randn(2, 2, K)
    offsets = offsets_of([0] * 7 + [1] + [0] * 20 + [1] + [0] * 3)
    assert qb.lib().qmoe_expert_linear_in_place(2, E, N, K) == 1
    qb.expert_linear(x, w, offsets)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = qb.expert_linear(x, w, offsets)
    assert torch.cuda.max_memory_allocated() - held < 1 << 20
    close(y, *ref.linear(x.cpu().double(), w.cpu().double(), offsets.cpu()), "y")


def test_workspaces_that_are_too_small_are_refused():
    x, w, off = randn(3, 1, 4096), randn(4, 1, 4096, 4096), offsets_of([1])
    need = qb.lib().qmoe_expert_workspace_bytes(1, 1, 4096, 4096, 0, 0)
    assert need > 0
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    for n in (1, need - 1):
        with pytest.raises(qb.QmoeError):
            qb.expert_linear(x, w, off, ws=byte(n))
    want = qb.expert_linear(x, w, off)
    assert torch.equal(qb.expert_linear(x, w, off, ws=byte(need)), want)
    odd, rows = randn(5, 2, 64, 65), randn(6, 600, 65)
    offsets, copies = offsets_of([300, 300]), qb.lib().qmoe_expert_copy_bytes(128, 65) + qb.lib().qmoe_expert_copy_bytes(600, 65)
    assert not qb.lib().qmoe_expert_linear_in_place(600, 2, 64, 65)
    with pytest.raises(qb.QmoeError):
        qb.expert_linear(rows, odd, offsets, ws=byte(copies - 256))
    assert torch.equal(qb.expert_linear(rows, odd, offsets, ws=byte(copies)), qb.expert_linear(rows, odd, offsets))


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("gather", [False, True])
def test_each_gradient_without_what_the_other_takes(gather, odd):
    counts, N, K, k = [40, 0, 300, 7], 136 - odd, 72 + odd, 2
    P, offsets = sum(counts) + 3, offsets_of(counts)
    w, dy = randn(7, 4, N, K), randn(8, P, N)
    x = randn(9, P // k if gather else P, K)
    pairs = torch.randperm(P, device="cuda").int() % (P // k * k) if gather else None
    dx, dw = qb.expert_linear_backward(dy, x, w, offsets, pairs=pairs, k=k)
    one, none = qb.expert_linear_backward(dy, None, w, offsets, pairs=pairs, k=k, need_dw=False)
    assert none is None and torch.equal(one, dx)
    none, one = qb.expert_linear_backward(dy, x, None, offsets, pairs=pairs, k=k, need_dx=False)
    assert none is None and torch.equal(one, dw)
    assert qb.expert_linear_backward(dy, None, None, offsets, need_dx=False, need_dw=False) == (None, None)
    back = lambda *args, **kw: qb.expert_linear_backward(*args, pairs=pairs, k=k, **kw)
    for f in (lambda: back(dy, None, w, offsets), lambda: back(dy, x, None, offsets), lambda: back(dy, x, None, offsets[:0], need_dx=False),
              lambda: back(dy, x.half(), None, offsets, need_dx=False), lambda: back(dy[:, :-1], None, w, offsets, need_dw=False),
              lambda: back(dy.float(), None, w.float(), offsets, need_dw=False), lambda: back(dy, None, w, offsets[1:], need_dw=False)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(qb.QmoeError):
        back(dy, x, None, offsets[:1], need_dx=False)  # no experts


@pytest.mark.parametrize("T", [40, 3000])
def test_align_sort_reports_bad_ids(T):
    """To the device's word, as the other calls; an id of -1 is no error, and the sort is the same."""
    k, E = 2, 7
    ids = torch.randint(-1, E, (T, k), device="cuda").int()
    word = qb.status_word("cuda")
    before = int(word)
    offsets, pairs, slot = qb.align_sort(ids, E)
    assert int(word) == before
    d, new = qb.dims(T, k, 32, 32, E), lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    own, out = torch.zeros(1, dtype=torch.int32, device="cuda"), (new(E), new(E + 1), new(T * k), new(T, k))
    qb.qmoe_align_sort(d, ids, *out, own, qb.alloc_workspace(qb.workspace_bytes(d)))
    assert all(torch.equal(a, b) for a, b in zip(out[1:], (offsets, pairs, slot))) and int(own) == qb.DEV_BAD_EXPERT_ID
    try:
        for wrong in (E, -2, 2 ** 31 - 1, -2 ** 31):
            ids[T // 2, 1] = wrong
            word.zero_()
            qb.align_sort(ids, E)
            assert int(word) == qb.DEV_BAD_EXPERT_ID
            mine = torch.zeros(1, dtype=torch.int32, device="cuda")
            word.zero_()
            qb.align_sort(ids, E, dev_status=mine)
            assert int(mine) == qb.DEV_BAD_EXPERT_ID and int(word) == 0
    finally:
        word.fill_(before)


def test_align_sort_is_captured_without_a_status_word():
    ids = torch.tensor([[2, 0], [1, 2], [-1, 7]], dtype=torch.int32, device="cuda")
    want = qb.align_sort(ids, 3, dev_status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    held = dict(qb._status_words)
    qb._status_words.clear()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = qb.align_sort(ids, 3)
        graph.replay()
        torch.cuda.synchronize()
        assert not qb._status_words and all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        qb._status_words.update(held)
