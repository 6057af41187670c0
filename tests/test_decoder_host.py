"""Host-side behaviour of the calls between a decoder's linears that needs no GPU: how
work is cut, and what the bindings do before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib
from int8_qmv_qmm_gb300.decoder import Decoder


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


def test_sample_quotient_rounds_as_the_division(L):
    """Over temperatures of every size, distances up to 26 of them, and quotients next to
    the middle between two numbers, where a faithful but not correct step shows.  (A
    distance that is subnormal leaves no exact remainder: quotients below 2^-30, whose
    exponential is 1, only have to stay below it.)"""
    rng = np.random.default_rng(3)
    f32 = np.float32
    n = 200000
    tau = np.concatenate([np.exp(rng.uniform(np.log(1e-2), np.log(1e2), n)),
                          np.exp(rng.uniform(np.log(1.1e-30), np.log(0.9e30), n)),
                          2.0 ** rng.integers(-90, 90, n) * (2 - 2.0 ** -23)]).astype(f32)
    share = np.concatenate([rng.uniform(1e-9, 25.9, 2 * n), 2.0 ** rng.uniform(-60, 4, n)])
    a = -(tau.astype(np.float64) * share).astype(f32)
    # numbers nearest to tau times a middle
    mid = (1 + (2 * rng.integers(0, 2 ** 23, n) + 1) * 2.0 ** -24) * 2.0 ** rng.integers(-8, 4, n)
    a = np.concatenate([a, -(tau[:n].astype(np.float64) * mid).astype(f32)])
    tau = np.concatenate([tau, tau[:n]])
    q = np.empty_like(a)
    assert L.qlin_testing_sample_quotient(a.ctypes.data, tau.ctypes.data, q.ctypes.data, len(a)) == 0
    true = a / tau
    matters = np.abs(true) >= 2.0 ** -30
    assert matters.sum() > 3.4 * n and np.array_equal(q[matters], true[matters])
    assert (np.abs(q[~matters]) <= 2.0 ** -30).all()
    assert L.qlin_testing_sample_quotient(None, None, None, 1) == 1


# ------------------------------------------------------------------ the bindings
class OnDevice:
    """A tensor's face, on a CUDA device that need not be there."""

    def __init__(self, shape, dtype, index=0):
        self.t = torch.zeros(shape, dtype=dtype)
        self.index, self.device, self.is_cuda = index, torch.device("cuda", index), True

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class NoLaunch:
    """A library whose calls all launch: none may be reached."""

    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.mark.parametrize("which", ["weight", "residual", "residual_out", "out"])
def test_norm_refuses_tensors_on_another_device(monkeypatch, which):
    monkeypatch.setattr(q, "lib", NoLaunch)
    monkeypatch.setattr(q, "_current_raw_stream", lambda index: 0)
    f16, f32 = torch.float16, torch.float32
    tensors = dict(x=((3, 64), f16), weight=((64,), f16), residual=((3, 64), f32),
                   residual_out=((3, 64), f32), out=((3, 64), f16))
    good = {name: OnDevice(*v) for name, v in tensors.items()}
    with pytest.raises(AssertionError, match="qlin_add_rms_norm was called"):
        q.add_rms_norm(**good)
    with pytest.raises(ValueError, match=f"^{which} must"):
        q.add_rms_norm(**{**good, which: OnDevice(*tensors[which], index=1)})


def test_a_cache_keeps_its_tensors(monkeypatch):
    """The handle holds their addresses: replacing one would be silently ignored."""
    monkeypatch.setattr(q, "_need_cuda", lambda *ts: None)
    c = q.KVCache.empty(2, 128, 1, 64, device="cpu")
    lens, at = c.lens, c.lens.data_ptr()
    c.lens += 3
    c.lens.copy_(c.lens + 1)
    c.table[1] = 5
    c.table = c.table
    assert c.lens is lens and c.lens.tolist() == [4, 4] and c._struct.lens == at
    for name in ("pages", "scales", "tail", "table", "lens"):
        with pytest.raises(AttributeError, match=f"cache's {name} cannot be replaced"):
            setattr(c, name, getattr(c, name) + 1)
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(c, name, getattr(c, name).clone())
    assert c.lens is lens and c.table.tolist() == [[0, 1], [5, 5]]


# ------------------------------------------------------------------ the decoder
def test_a_decode_step_after_a_row_without_a_token():
    """sample() gives -1 for such a row; looking its embedding up would fault."""
    d = object.__new__(Decoder)
    d.embed = torch.arange(12.0).view(4, 3)
    d.tokens = torch.tensor([2, -1, 3], dtype=torch.int32)
    d._one_each = torch.arange(4, dtype=torch.int32)
    d._forward = lambda tokens, starts, max_new: F.embedding(tokens, d.embed)
    d._sample = lambda logits, tokens: None
    d._step()
    assert torch.equal(d.logits, d.embed[[2, 0, 3]])
    assert d.tokens.tolist() == [2, -1, 3]
