"""Edges of the experts' products, log probabilities and what stands beside them: plans
that leave most of a launch without work, logits at the ends of their types, weights whose
scales are far apart, lengths at a border.

Tolerances are derived beside each test (u = 2^-11 for f16, 2^-8 for bf16, 2^-24 for f32: one
rounding to nearest of a result)."""

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from tests.test_gpu_decoder import normal
from tests.test_gpu_experts import BF16, F16, F32, Layer, dev, routing_of  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ experts' products
@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16)])
def test_expert_linear_launches_that_are_mostly_idle(dev, bits, dt):  # noqa: F811
    """All rows of 64 experts' plan with one of them: the host sizes the launch for 74 tiles
    of tokens, 10 have rows, and the other CTAs, which multiply nothing, make room for those
    of the next call while this one runs.  The same bits from every call."""
    layer = Layer(dev, 64, 200, 256, bits, dt, seed=3)
    x = normal(1, 640, 256).to(dt).to(dev)
    routing = routing_of(np.full((640, 1), 41), 64, dev)
    ref = layer.check(x, routing)
    args = (x, routing, layer.wq, layer.scales, layer.biases, bits)
    outs = [q.expert_linear(*args, overlap_previous=True) for _ in range(40)]
    assert all(torch.equal(o, ref) for o in outs)
    assert q.device_status() == 0
