"""Host-side edges of the experts' calls (no GPU: nothing here reaches a launch)."""

import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib
from tests.test_decoder_host import NoLaunch, OnDevice


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


# ------------------------------------------------- tensors of a device that is not current
def test_calls_are_refused_where_their_device_is_not_current(monkeypatch):
    """The kernels would run on the current device with another one's pointers."""
    monkeypatch.setattr(q, "lib", NoLaunch)
    monkeypatch.setattr(q, "_raw_stream", lambda index: 0)
    f16, f32, i32 = torch.float16, torch.float32, torch.int32

    def tensors(index):
        def t(shape, dtype=f16):
            return OnDevice(shape, dtype, index)

        routing = q.Routing(t((3, 2), i32), t((3, 2), f32), t((6,), i32), t((5,), i32))
        return [lambda: q.add_rms_norm(t((3, 64)), t((64,)), out=t((3, 64))),
                lambda: q.expert_linear(t((3, 64)), routing, t((4, 32, 8), i32), t((4, 32, 1)),
                                        t((4, 32, 1)), 4, out=t((6, 32))),
                lambda: q.combine_experts(t((6, 32)), routing, out=t((3, 32)))]

    monkeypatch.setattr(NoLaunch, "qlin_expert_linear_workspace_size", lambda *a: 0,
                        raising=False)
    for current in (0, 1):
        monkeypatch.setattr(q, "_current_device", lambda: current)
        for index in (0, 1):
            for call in tensors(index):
                if index == current:
                    with pytest.raises(AssertionError, match="was called"):
                        call()
                else:
                    with pytest.raises(ValueError, match=f"cuda:{index}, which is not the current"):
                        call()


def test_stalled_expert_linear_refusals(L):
    """The test-only entry refuses what qlin_expert_linear does, calls that take the streaming
    kernel, and limits out of range."""
    FAKE, INVALID, MISALIGNED = 0x10000, 1, 3
    need = L.qlin_expert_linear_workspace_size(320, 8, 256, 128)

    def call(x=FAKE, P=320, K=128, ws=FAKE, size=need, stage=3, limit=2000):
        return L.qlin_testing_expert_linear_stalled(x, 128, 1, FAKE, FAKE, P, FAKE, FAKE, FAKE,
                                                    FAKE, 8, 256, K, ws, size, stage, limit, None)

    assert call(x=None) == INVALID and call(x=FAKE + 8) == MISALIGNED
    assert call(K=100) == INVALID and call(ws=None) == INVALID and call(size=need - 1) == INVALID
    assert call(P=8) == INVALID and call(P=0) == INVALID
    assert call(stage=-1) == INVALID
    assert call(limit=999) == INVALID and call(limit=2000001) == INVALID
