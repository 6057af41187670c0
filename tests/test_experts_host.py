"""Host-side tests of routing, the experts' calls and log probabilities: what is
refused before anything is launched (no GPU: no call here reaches a launch), and the
oracle on cases worked out by hand."""

import ctypes
import math

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib
from oracle import experts_oracle as O
from tests.test_decoder_abi import CACHE_FAULTS, cache

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
FAKE = 0x10000  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return q.lib()


def test_route_refusals(L):
    def route(x=FAKE, xs=64, bias=None, scoring=0, groups=1, top_groups=1, gs=0, k=8, renorm=1,
              scale=1.0, experts=FAKE, weights=FAKE, order=FAKE, offsets=FAKE, T=3, E=64,
              dt=q.QLIN_F32, ws=None, size=0, flags=0):
        return L.qlin_route_experts(x, xs, bias, scoring, groups, top_groups, gs, k, renorm, scale,
                                    experts, weights, order, offsets, T, E, dt, ws, size, flags,
                                    None)

    assert route(k=0) == INVALID
    assert route(k=65) == INVALID
    assert route(k=33) == UNSUPPORTED
    assert route(E=0) == INVALID
    assert route(E=513, xs=513) == UNSUPPORTED
    assert route(T=-1) == INVALID
    assert route(T=1 << 30) == UNSUPPORTED
    assert route(dt=3) == UNSUPPORTED
    assert route(scoring=2) == INVALID
    assert route(gs=2) == INVALID
    assert route(renorm=2) == INVALID
    assert route(groups=0) == INVALID
    assert route(groups=5) == INVALID
    assert route(groups=64) == UNSUPPORTED
    assert route(groups=4, top_groups=5) == INVALID
    assert route(groups=4, top_groups=0) == INVALID
    assert route(scale=float("inf")) == INVALID
    assert route(x=None) == INVALID
    assert route(offsets=None) == INVALID
    assert route(T=0, offsets=None) == INVALID
    assert route(order=None) == INVALID
    assert route(xs=63) == INVALID
    assert route(flags=2) == INVALID
    assert route(x=FAKE + 2) == MISALIGNED
    assert route(x=FAKE + 1, dt=q.QLIN_F16) == MISALIGNED
    assert route(bias=FAKE + 2) == MISALIGNED
    need = L.qlin_route_experts_workspace_size(1000, 64)
    assert need > 0 and L.qlin_route_experts_workspace_size(1, 64) == 0
    assert route(T=1000) == INVALID
    assert route(T=1000, ws=FAKE, size=need - 1) == INVALID
    assert route(T=1000, ws=FAKE + 2, size=need) == MISALIGNED


def linear(L, x=FAKE, xs=128, ppr=2, order=FAKE, offsets=FAKE, P=6, wq=FAKE, sc=FAKE, bi=FAKE,
           y=FAKE, E=4, N=32, K=128, bits=4, group=64, dt=q.QLIN_F16, ydt=q.QLIN_F16, flags=0,
           ws=None, size=0):
    return L.qlin_expert_linear(x, xs, ppr, order, offsets, P, wq, sc, bi, y, E, N, K, bits, group,
                                dt, ydt, ws, size, flags, None)


def test_expert_linear_refusals(L):
    assert linear(L, bits=3) == UNSUPPORTED
    assert linear(L, group=32) == UNSUPPORTED
    assert linear(L, dt=q.QLIN_F32) == UNSUPPORTED
    assert linear(L, ydt=q.QLIN_BF16) == UNSUPPORTED
    assert linear(L, K=96) == INVALID
    assert linear(L, K=0) == INVALID
    assert linear(L, N=0) == INVALID
    assert linear(L, E=0) == INVALID
    assert linear(L, E=513) == UNSUPPORTED
    assert linear(L, N=(1 << 20) + 1) == UNSUPPORTED
    assert linear(L, K=65600, xs=65600) == UNSUPPORTED
    assert linear(L, P=-2) == INVALID
    assert linear(L, P=7) == INVALID
    assert linear(L, ppr=0) == INVALID
    assert linear(L, flags=2) == INVALID
    for name in ("x", "order", "offsets", "wq", "sc", "bi", "y"):
        assert linear(L, **{name: None}) == INVALID, name
    assert linear(L, xs=120) == INVALID
    assert linear(L, xs=132) == MISALIGNED
    assert linear(L, x=FAKE + 8) == MISALIGNED
    assert linear(L, wq=FAKE + 4) == MISALIGNED
    assert linear(L, sc=FAKE + 1) == MISALIGNED
    assert linear(L, y=FAKE + 2, ydt=q.QLIN_F32) == MISALIGNED
    assert linear(L, P=0, x=None, y=None) == OK
    need = L.qlin_expert_linear_workspace_size(4000, 4, 32, 128)
    assert need >= 4000 * 128 * 2 and L.qlin_expert_linear_workspace_size(6, 4, 32, 128) == 0
    assert linear(L, P=4000) == INVALID
    assert linear(L, P=4000, ws=FAKE, size=need - 1) == INVALID
    assert linear(L, P=4000, ws=FAKE + 8, size=need) == MISALIGNED


def test_combine_refusals(L):
    def combine(y=FAKE, experts=FAKE, weights=FAKE, add=None, stride=0, out=FAKE, T=3, k=2, N=64,
                dt=q.QLIN_F16, ydt=q.QLIN_F16, flags=0):
        return L.qlin_combine_experts(y, experts, weights, add, stride, out, T, k, N, dt, ydt,
                                      flags, None)

    assert combine(dt=q.QLIN_F32) == UNSUPPORTED
    assert combine(ydt=q.QLIN_BF16) == UNSUPPORTED
    assert combine(T=-1) == INVALID
    assert combine(k=0) == INVALID
    assert combine(k=33) == UNSUPPORTED
    assert combine(N=0) == INVALID
    assert combine(y=None) == INVALID
    assert combine(weights=None) == INVALID
    assert combine(add=FAKE, stride=63) == INVALID
    assert combine(flags=8) == INVALID
    assert combine(y=FAKE + 1) == MISALIGNED
    assert combine(experts=FAKE + 2) == MISALIGNED
    assert combine(T=0, y=None) == OK


def test_norm_rope_append_refusals(L):
    def append(c=None, qkv=FAKE, qs=8 * 64, qn=FAKE, kn=FAKE, eps=1e-6, T=3, rot=64, flags=0):
        c = c or cache()
        return L.qlin_norm_rope_append(qkv, qs, qn, kn, eps, FAKE, FAKE, 100, rot, 0,
                                       ctypes.byref(c), FAKE, T, 4, flags, None)

    for over, status in CACHE_FAULTS:
        assert append(cache(**over)) == status, over
    assert append(eps=-1.0) == INVALID
    assert append(eps=float("nan")) == INVALID
    assert append(eps=float("inf")) == INVALID
    assert append(qn=None) == INVALID
    assert append(kn=None) == INVALID
    assert append(qn=FAKE + 8) == MISALIGNED
    assert append(kn=FAKE + 2) == MISALIGNED
    assert append(rot=24) == UNSUPPORTED
    assert append(qkv=None) == INVALID
    assert append(flags=4) == INVALID
    assert append(T=0, qn=None, kn=None) == OK


def test_token_logprobs_refusals(L):
    def score(x=FAKE, xs=100, tokens=FAKE, lp=FAKE, ent=FAKE, top=2, tt=FAKE, tl=FAKE, M=2, V=100,
              dt=q.QLIN_F32, flags=0):
        return L.qlin_token_logprobs(x, xs, tokens, lp, ent, top, tt, tl, M, V, dt, flags, None)

    assert score(dt=7) == UNSUPPORTED
    assert score(V=0) == INVALID
    assert score(V=262145, xs=262145) == UNSUPPORTED
    assert score(M=-1) == INVALID
    assert score(top=-1) == INVALID
    assert score(top=33) == UNSUPPORTED
    assert score(x=None) == INVALID
    assert score(tokens=None) == INVALID
    assert score(ent=None) == INVALID
    assert score(tt=None) == INVALID
    assert score(tl=None) == INVALID
    assert score(xs=99) == INVALID
    assert score(flags=2) == INVALID
    assert score(x=FAKE + 2) == MISALIGNED
    assert score(tokens=FAKE + 2) == MISALIGNED
    assert score(M=0, x=None) == OK


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(2, 64)
    ints = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.route_experts(x, 1)
    with pytest.raises(ValueError):
        q.token_logprobs(x, ints[:, 0])
    with pytest.raises(ValueError):
        q.Routing(ints, torch.zeros(2, 1), ints[:, 0], ints[:, 0])


# ------------------------------------------------------------------ the oracle
def test_oracle_route_by_hand():
    x = np.log([1.0, 2.0, 4.0, 1.0])
    e, w, margin = O.route(x, 2)
    assert e.tolist() == [2, 1] and np.allclose(w, [2 / 3, 1 / 3]) and margin > 0.6
    e, w, _ = O.route(x, 2, renormalise=False, scale=8.0)
    assert np.allclose(w, [4.0, 2.0])
    # the bias chooses, the score weighs; equal ones by index
    e, w, _ = O.route(x, 2, bias=[1.0, 0.0, 0.0, 1.0], renormalise=False)
    assert e.tolist() == [0, 3] and np.allclose(w, [1 / 8, 1 / 8])
    # groups {1, 2}, {4, 1}: by the largest the second, by the sum of two as well
    for score in ("max", "top2"):
        e, _, _ = O.route(x, 2, groups=2, top_groups=1, group_score=score)
        assert e.tolist() == [2, 3]
    # sigmoid; a masked expert and too few of them
    e, w, _ = O.route([0.0, -np.inf, np.nan], 2, scoring="sigmoid", renormalise=False)
    assert e.tolist() == [0, -1] and w.tolist() == [0.5, 0.0]
    e, w, _ = O.route([np.nan, -np.inf], 1)
    assert e.tolist() == [-1] and w.tolist() == [0.0]
    order, offsets = O.plan(np.array([[1, 0], [-1, 1], [0, 2]]), 3)
    assert order.tolist() == [1, 4, 0, 3, 5, 2] and offsets.tolist() == [0, 2, 4, 5]


def test_oracle_logprobs_by_hand():
    lp, h, t, v = O.logprobs(np.log([1.0, 1.0, 2.0]), 0, 2)
    assert np.isclose(lp, -math.log(4)) and t.tolist() == [2, 0]
    assert np.isclose(h, 1.5 * math.log(2)) and np.allclose(v, [-math.log(2), -math.log(4)])
    lp, h, t, v = O.logprobs([np.nan, -np.inf, 3.0], 0, 2)
    assert lp == -np.inf and h == 0 and t.tolist() == [2, -1] and v.tolist() == [0.0, -np.inf]
    lp, h, t, _ = O.logprobs([np.inf, 1.0, np.inf], 2, 3)
    assert np.isclose(lp, -math.log(2)) and np.isclose(h, math.log(2)) and t.tolist() == [0, 2, 1]
    assert O.logprobs([-np.inf, np.nan], 0, 1)[0] == -np.inf


def test_oracle_combine_leaves_out_missing_experts():
    y = np.array([[[1.0, 2.0], [np.nan, np.inf]]])
    out, size = O.combine(y, np.array([[3, -1]]), np.array([[0.5, 0.0]]), np.array([[1.0, -4.0]]))
    assert out.tolist() == [[1.5, -3.0]] and size.tolist() == [[1.5, 5.0]]
