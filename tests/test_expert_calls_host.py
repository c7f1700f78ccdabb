"""CPU checks of the rules that the bindings of the experts' products ask of the library."""

import pytest

from quantized_mixture_experts_moe_gb300 import binding as qb
from quantized_mixture_experts_moe_gb300 import build as qbuild


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qb.lib()


def test_odd_weights_are_read_in_place_for_few_rows_only(lib):
    f = lib.qmoe_expert_linear_in_place
    assert f(1, 1, 7, 9) == 1
    # measured: one and two tokens x 8 of 128 experts 22 us for 41 and 53 for 61, one x 10 of 512 69 for 131, four rows 20 for 29
    assert all(f(*c) for c in ((8, 128, 1536, 2047), (16, 128, 1536, 2047), (10, 512, 2047, 4095), (4, 1, 4096, 4095), (2, 8, 2815, 4095)))
    # 242 us for 152, 41 for 29, 29 for 26, 182 for 162
    assert not any(f(*c) for c in ((112, 256, 1408, 1095), (16, 1, 4096, 4095), (32, 128, 767, 513), (54, 64, 2816, 1957)))
    assert f(4000, 128, 1536, 2047) == 0 and f(65536, 1024, 7, 9) == 0  # copied; more rows than a grid's second dimension
    for bad in ((-1, 1, 8, 8), (1, 0, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0)):
        assert f(*bad) == 0
