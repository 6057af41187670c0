"""Host-side edges of the experts' calls (no GPU: nothing here reaches a launch)."""

import pytest

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return q.lib()


def test_which_calls_of_few_rows_need_a_workspace(L):
    """Those whose rows are too long, or too many: 5 for each expert that could have any."""
    def size(pairs, k, experts=64):
        return L.qlin_expert_linear_workspace_size(pairs, experts, 32, k)

    assert size(8, 8384) == 0 and size(320, 8384) == 0 and size(320, 64) == 0
    for pairs, k in ((1, 8448), (8, 8448), (320, 8448), (321, 64)):
        # the rows in f16, a factor for each and for every row of the weights
        assert size(pairs, k) >= pairs * k * 2 + (pairs + 64 * 32) * 4
