"""GPU tests of gathered rows in tiles of few rows, where some of the warps that gather have nothing to bring: many launches, none
of which may wait in vain (the status word) or give other bits than the first."""

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def offsets_of(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.as_tensor(counts).cumsum(0)]).int().cuda()


# rows of the experts: tiles of up to 32 rows (16 an expert on average), and of up to 128 (96), with few rows in most
CASES = {"one row": [1] * 300, "four": [4] * 200, "eight": [8] * 128, "twelve": [12] * 128, "up to 13": [1 + i % 13 for i in range(250)],
         "few beside many": [96 if i % 4 == 0 else 1 + i % 12 for i in range(160)], "eight beside one": [2000] + [8] * 63}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("N,K", [(264, 2048), (1024, 192)])
def test_tiles_of_few_gathered_rows(name, N, K):
    counts = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(len(counts) + N)
    E, P, k = len(counts), sum(counts), 2
    x = torch.randn(-(-P // k), K, generator=g, device="cuda").to(BF16)
    w = torch.randn(E, N, K, generator=g, device="cuda").to(BF16)
    pairs = torch.randperm(P, generator=g, device="cuda").int()
    offsets, word = offsets_of(counts), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = x[(pairs // k).long()]
    first = qb.expert_linear(x, w, offsets, pairs=pairs, k=k, dev_status=word)
    assert torch.equal(first, qb.expert_linear(rows, w, offsets, dev_status=word))
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        other += (qb.expert_linear(x, w, offsets, pairs=pairs, k=k, dev_status=word) != first).any()
    assert int(other) == 0 and int(word) == 0
