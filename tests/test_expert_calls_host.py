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
    assert f(4000, 128, 1536, 2047) == 0 and f(65536, 1024, 7, 9) == 0  # copied; more rows than a grid's second dimension
    for bad in ((-1, 1, 8, 8), (1, 0, 8, 8), (1, 1, 0, 8), (1, 1, 8, 0)):
        assert f(*bad) == 0
