"""The decoder's steps around captures, and with logits that hold no token."""

import math

import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300.decoder import Decoder
from tests.test_gpu_decode_loop import SHAPE, dev, prompts  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_a_slot_without_a_token(dev, captured):  # noqa: F811
    """Its token is -1, step after step, and the other slots' are as ever."""
    seen = []
    for bad in (False, True):
        d = Decoder(dev, **SHAPE)
        ids = prompts((20, 70, 5))
        ids = [[t if t != 7 else 8 for t in p] for p in ids]
        if bad:
            d.embed[7] = math.nan
            ids[1][66] = 7
        d.prefill(ids)
        got = [d.tokens.clone()]
        if captured:
            d.capture()
        got += [d.decode().clone() for _ in range(4)]
        seen.append(torch.stack(got).tolist())
    clean, bad = seen
    assert all(t[1] >= 0 for t in clean)
    assert [t[1] for t in bad] == [-1] * 5
    # (none of the others' tokens is 7, whose embedding differs)
    assert all(7 not in (t[0], t[2]) for t in clean)
    assert [(t[0], t[2]) for t in bad] == [(t[0], t[2]) for t in clean]
    assert q.device_status() == 0


def test_logits_are_the_last_calls(dev):  # noqa: F811
    """Around a capture, and where prompts come between replays."""
    seen = []
    for captured in (False, True):
        d = Decoder(dev, **SHAPE)
        ids = prompts((63, 5, 120))
        got = []

        def keep():
            got.append((d.tokens.clone(), d.logits.clone()))

        d.prefill(ids)
        keep()
        if captured:
            d.capture()
            keep()
        else:
            got.append(got[-1])
        for more in ([], [[], ids[0][:9], []], [ids[1], [], [3]]):
            if more:
                d.prefill(more)
                keep()
            for _ in range(2):
                d.decode()
                keep()
        seen.append(got)
    for i, ((t0, l0), (t1, l1)) in enumerate(zip(*seen)):
        assert torch.equal(t0, t1) and torch.equal(l0, l1), i
    assert q.device_status() == 0
