"""Host-side behaviour of the calls between a decoder's linears that needs no GPU: how
work is cut, and what the bindings do before anything is launched."""

import ctypes

import pytest

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return q.lib()


# ------------------------------------------------------------------ sampling
def sample_plan(L, m, v, sms=152):
    got = [ctypes.c_int(-1) for _ in range(3)]
    status = L.qlin_testing_sample_plan(m, v, sms, *map(ctypes.byref, got))
    return status, *(g.value for g in got)


@pytest.mark.parametrize("m", [1, 512])
def test_sample_cuts_every_vocabulary_alike(L, m):
    """All CTAs of a row read each other's histograms, so they have to agree on the
    limbs, and a limb's sum over a part has to stay below 2^32.  Vocabularies whose last
    part is shorter than 16384 elements while the others are not are among these (280,
    between 131009 and 131463)."""
    uneven = 0
    for v in range(1, 262145):
        status, ranks, part, limb = sample_plan(L, m, v)
        assert status == 0 and ranks in (1, 2, 4, 8) and part % 8 == 0
        last = v - (ranks - 1) * part
        assert 0 < last <= part <= 32768, v
        # weights are at most 2^36: two limbs of 18 bits (and the carry), or three of 12
        assert limb in (12, 18) and part * 2 ** (18 if limb == 18 else 12) < 2 ** 32, v
        uneven += last < 16384 <= part
    assert uneven == 280


def test_sample_plan_refusals(L):
    assert sample_plan(L, 0, 10)[0] == 1
    assert sample_plan(L, 1, 0)[0] == 1
    assert sample_plan(L, 1, 262145)[0] == 1
    assert sample_plan(L, 1, 10, 0)[0] == 1
    assert L.qlin_testing_sample_plan(1, 10, 152, None, None, None) == 1
