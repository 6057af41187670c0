"""GPU parity of the calls between a decoder's linears where their work splits unevenly
or their values are far apart, infinite or NaN, against the float64 oracle."""

import pytest
import torch

import int8_qmv_qmm_gb300 as q
from tests.test_gpu_decoder import (F16, F32, Model, check_sample, dev, normal,  # noqa: F401
                                    settings)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ sampling
@pytest.mark.parametrize("v", [8200, 16392, 33000])
def test_sample_small_parts_of_a_row(dev, v):  # noqa: F811
    """Clusters of 2, 4 and 8 CTAs whose first exchange comes soon after their start:
    the same token every time, and the oracle's."""
    row = (2.5 * normal(v, v)).to(F32)
    check_sample(dev, row, m=8, p=0.9)
    x, u = row.to(dev).view(1, v), torch.tensor([0.37], device=dev)
    got = [q.sample(x, u, *settings(dev, 1, p=0.9)) for _ in range(300)]
    assert len({(t.item(), p.item()) for t, p in got}) == 1


@pytest.mark.parametrize("dt", [F32, F16])
@pytest.mark.parametrize("v", [131009, 131071, 131073, 131463, 131464])
def test_sample_where_the_last_part_is_short(dev, v, dt):  # noqa: F811
    """Eight CTAs share a row, the last with fewer than 16384 logits, the others with
    16384 or more: a bound by weight, alone and after top-k."""
    row = (3.0 * normal(v, v)).to(dt)
    for kw in (dict(p=0.9), dict(p=0.3, tau=2.0), dict(k=v // 2, p=0.95), dict(p=0.7, mp=0.01),
               dict(k=50, p=0.9), dict(p=0.999, tau=0.5)):
        check_sample(dev, row, m=16, **kw)


# ------------------------------------------------------------------ attention
def test_parts_of_both_kernels_joined_in_one_call(dev):  # noqa: F811
    """Sequences that decode over caches long enough to be cut, beside prompts whose
    tiles are cut too: both kernels leave parts, and one launch joins them."""
    m = Model(dev, 5, 2, 64, F16, blocks=70)
    m.append([4000, 3000, 200, 2500, 0], 8, None, seed=1)
    new = [1, 2, 150, 1, 90]
    m.append(new, 8, None, seed=2, advance=False)
    m.attend(new, 8, seed=3, q_scale=1.5, only={0, 1, 2, 3, 80, 152, 153, 154, 200, 243})
    assert q.device_status() == 0
