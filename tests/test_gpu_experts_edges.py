"""Edges of the experts' products, log probabilities and what stands beside them: plans
that leave most of a launch without work, logits at the ends of their types, weights whose
scales are far apart, lengths at a border.

Tolerances are derived beside each test (u = 2^-11 for f16, 2^-8 for bf16, 2^-24 for f32: one
rounding to nearest of a result)."""

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300.decoder import Decoder
from oracle import experts_oracle as O
from tests.test_gpu_decode_loop import prompts
from tests.test_gpu_decoder import TINY, U, f64, normal
from tests.test_gpu_experts import (BF16, F16, F32, Layer, dev, random_experts,  # noqa: F401
                                    routing_of)
from tests.test_gpu_experts_together import MIXED

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


# ------------------------------------------------------------ log probabilities
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 240])  # (a cluster to a row, and a CTA)
@pytest.mark.parametrize("rest,high", [(0.0, 5e35), (0.0, 1e37), (59.0, 1e13), (59.0, 1e30)])
def test_logprobs_of_a_logit_far_above_all_others(dev, dt, rows, rest, high):  # noqa: F811
    """The others' exponentials are 0, whatever number of them, or sum under a lower reference
    (threads begin at 0, then meet `rest`), stands before them: the entropy is 0 and the log
    probabilities are differences of logits."""
    v, at = 128256, 77777
    x = torch.zeros(rows, v, dtype=dt, device=dev)
    x.view(rows, 8, -1)[:, :, v // 16:] = rest
    x[:, at] = high
    tokens = torch.full((rows,), at, dtype=torch.int32, device=dev)
    tokens[::2] = 4
    lp, entropy, top, top_lp = q.token_logprobs(x, tokens, 3)
    assert (entropy == 0).all()
    assert torch.equal(lp, torch.where(tokens == at, 0.0, -x[:, at].float()))
    assert (top[:, 0] == at).all() and (top_lp[:, 0] == 0).all()
    assert (top[:, 1:] == (x[0] == rest).nonzero()[:2, 0]).all()
    assert torch.equal(top_lp[:, 1], rest - x[:, at].float())


def test_logprobs_are_not_positive(dev):  # noqa: F811
    """A probability is at most 1: no log probability is above 0, and no entropy below, also
    where one token has all but nothing of the share and its exponential is 1 by way of a
    product of two (the reference that a thread began with, 0, and the largest logit, in
    vectors of the same thread)."""
    rows, v = 600, 4096
    high = torch.linspace(1.0, 59.9, rows, dtype=torch.float64)
    x = torch.full((rows, v), -float("inf"))
    x[:, 0] = 0.0
    x[:, 2048] = high.float()
    for dt in (F32, F16, BF16):
        y = x.to(dt)
        h = y[:, 2048].double()
        tokens = torch.full((rows,), 2048, dtype=torch.int32, device=dev)
        lp, entropy, _, top_lp = q.token_logprobs(y.to(dev), tokens, 2)
        assert (lp <= 0).all() and (entropy >= 0).all() and (top_lp <= 0).all()
        ref = -torch.log1p(torch.exp(-h))
        # exponentials are 2 ulp off, as is their product's argument: 2^-20 of z; the entropy's
        # mean is a difference of two numbers up to 60 * log2(e), off by 2^-22 of them
        assert (lp.double().cpu() - ref).abs().max() <= 2.0 ** -20
        ref = -ref + h / (1 + torch.exp(h))
        assert (entropy.double().cpu() - ref).abs().max() <= 2.0 ** -15


# ---------------------------------------------------- what a weight is rounded to
def spread_layer(dev, bits, dt, spread):  # noqa: F811
    """A layer in which half of each row's groups are 2^spread smaller than the others, and its
    scales and biases in float64, for each weight."""
    layer = Layer(dev, 3, 72, 256, bits, dt, seed=11)
    for t in (layer.scales, layer.biases):
        t[..., 1:3] *= 2.0 ** -spread
    s, b = (np.repeat(f64(t), 64, -1) for t in (layer.scales, layer.biases))
    codes = layer.wq.cpu().numpy().view(np.uint32)[..., None] >> np.arange(0, 32, bits,
                                                                           dtype=np.uint32)
    layer.w = (codes & (2 ** bits - 1)).reshape(s.shape).astype(np.float64) * s + b
    return layer, s, b


def one_hot(dev, layer, tokens, bound, first=0):  # noqa: F811
    """Rows of x that hold one element each, at first and on, times every weight of their
    expert, in float32: the largest error in units of `bound` (of each weight) times x."""
    e, n, k = layer.w.shape
    rng = np.random.default_rng(5)
    at = rng.permutation((first + np.arange(tokens)) % k)
    value = torch.from_numpy(rng.uniform(1, 2, tokens)).to(layer.dt)
    x = torch.zeros(tokens, k, dtype=layer.dt)
    x[torch.arange(tokens), torch.from_numpy(at)] = value
    which = rng.integers(0, e, tokens)
    y = q.expert_linear(x.to(dev), routing_of(which[:, None], e, dev), layer.wq, layer.scales,
                        layer.biases, layer.bits, out_dtype=F32)
    v = value.double().numpy()[:, None]
    return (np.abs(f64(y) - v * layer.w[which, :, at]) / (v * bound[which, :, at])).max()


SPREADS = [(F16, 0), (F16, 12), (BF16, 0), (BF16, 20), (BF16, 32), (BF16, 40)]


@pytest.mark.parametrize("dt,spread", SPREADS)
@pytest.mark.parametrize("bits", [4, 8])
def test_expert_linear_rounds_weights_as_it_says(dev, bits, dt, spread):  # noqa: F811
    """With one element of x at a time an output is one weight.  Of many rows' products a weight
    is one rounding to f16: off by 2^-11 of it at most, or by 2^-25 (f16's least numbers).

    bfloat16 weights are in a unit that puts the row's largest at 2^14 or more.  Scale, bias
    and weight are multiples of 2^-24 there, the first two off by 2^-25 at most, so that the
    weight is off by (largest code + 1) * 2^-25 before its own rounding, which is exact where
    it is below f16's normal numbers: 2^-31 of the row's largest at 8 bits, 2^-35 at 4."""
    layer, s, b = spread_layer(dev, bits, dt, spread)
    largest = np.maximum(np.abs(b), np.abs(b + (2 ** bits - 1) * s)).max(-1, keepdims=True)
    least = 2.0 ** -25 if dt is F16 else 2.0 ** (bits - 39) * largest
    # (the rounding of a weight that is off already: 2^-11 more of that)
    worst = one_hot(dev, layer, 768, np.abs(layer.w) * 2.0 ** -11 + least)
    assert worst <= 1 + 2.0 ** -10, worst


@pytest.mark.parametrize("dt,spread", SPREADS)
@pytest.mark.parametrize("bits", [4, 8])
def test_expert_linear_of_few_rows_rounds_no_weight(dev, bits, dt, spread):  # noqa: F811
    """x and (1024 + code) * x are exact.  bias - 1024 * scale is rounded once, its product with
    x once more, their sum with scale times the other once more, all in float32: a weight that
    was rounded to f16 (2^-12 of it off, on the whole) would be far outside."""
    layer, s, b = spread_layer(dev, bits, dt, spread)
    bound = np.abs(b - 1024 * s) * 2.0 ** -23 + np.abs(layer.w) * 2.0 ** -24
    rounded = np.abs(layer.w - layer.w.astype(np.float16)) if dt is F16 or not spread else None
    assert rounded is None or (rounded / bound).max() > 4
    for first in range(0, 256, 12):  # (12 rows of 3 experts: few)
        worst = one_hot(dev, layer, 12, bound, first)
        assert worst <= 1 + 2.0 ** -10, (first, worst)


# ---------------------------------------------------------------- lengths at a border
@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16)])
@pytest.mark.parametrize("k", [8384, 8448])
def test_expert_linear_at_the_longest_streamed_row(dev, bits, dt, k):  # noqa: F811
    """The last length whose tokens fit beside the weights on their way, and the first that
    goes to the tensor cores."""
    layer = Layer(dev, 3, 40, k, bits, dt, seed=k)
    for tokens in (1, 7):
        layer.check(normal(1, tokens, k).to(dt).to(dev),
                    routing_of(random_experts(3, tokens, 2, 3), 3, dev))
    assert q.device_status() == 0


# --------------------------------------------------------------------- the decoder
def test_decoder_log_probabilities_stay_with_their_tokens(dev):  # noqa: F811
    """A call that gives a slot no tokens leaves its last token, and that token's log
    probabilities with it: the next slot's prompt does not take their place."""
    d = Decoder(dev, **MIXED)
    d.temperature.fill_(0.8)
    torch.manual_seed(3)
    d.prefill(prompts((5, 70, 9)))
    names = ("logprobs", "entropy", "top_tokens", "top_logprobs")
    for captured in (False, True):
        if captured:
            d.capture()
        d.decode()
        before = {name: getattr(d, name).clone() for name in names}
        token = d.tokens.clone()
        d.prefill([[], [1, 2, 3], []])
        for name in names:
            now = getattr(d, name)
            assert torch.equal(now[[0, 2]], before[name][[0, 2]]), name
        assert torch.equal(d.tokens[[0, 2]], token[[0, 2]])
        ref = O.logprobs(f64(d.logits)[1], int(d.tokens[1]), 5)
        assert abs(float(d.logprobs[1]) - ref[0]) <= 2.0 ** -16
        assert np.array_equal(d.top_tokens[1].cpu().numpy(), ref[2])
    assert q.device_status() == 0


# --------------------------------------------------- a device that is not the current one
def test_every_call_is_refused_where_its_device_is_not_current(dev, monkeypatch):  # noqa: F811
    layer = Layer(dev, 2, 8, 64, 8, F16)
    w = normal(1, 8, 64).float().to(dev)
    packed = q.quantize_affine(w, 8)
    x, z = normal(2, 3, 64).to(F16).to(dev), torch.zeros(3, 10, device=dev)
    qkv = normal(3, 3, 3 * 64).to(F16).to(dev)
    norm = torch.ones(64, dtype=F16, device=dev)
    routing = q.route_experts(z, 2)
    row, none = torch.ones(3, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    cache = q.KVCache.empty(1, 128, 1, 64, device=dev)
    starts = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    ws = q.attention_workspace(64)
    expert = (routing_of([[0], [1], [1]], 2, dev), layer.wq, layer.scales, layer.biases, 8)
    calls = [lambda: q.quantize_affine(w, 8), lambda: q.dequant(*packed, 8),
             lambda: q.qmv(x[:1], *packed, 8), lambda: q.qmm(x, *packed, 8),
             lambda: q.linear(x, *packed, 8), lambda: q.add_rms_norm(x, norm),
             lambda: q.rope_table(8, 64), lambda: q.rope_append(qkv, None, cache, starts, 1),
             lambda: q.rope_append(qkv, None, cache, starts, 1, q_norm=norm, k_norm=norm),
             lambda: q.cache_attention(x.view(3, 1, 64), cache, starts, 3, ws),
             lambda: q.cache_dequant(cache, none[:1]),
             lambda: q.sample(z, row, row, none, row, 0 * row),
             lambda: q.token_logprobs(z, none, 2), lambda: q.route_experts(z, 2),
             lambda: q.expert_linear(x, *expert),
             lambda: q.combine_experts(normal(4, 6, 64).to(F16).to(dev), routing)]
    for call in calls:
        call()
    assert q.device_status() == 0
    monkeypatch.setattr(q, "_current_device", lambda: 1)
    for i, call in enumerate(calls):
        if i == 6:
            continue  # (it makes its table on the current device)
        with pytest.raises(ValueError, match="not the current device"):
            call()


# ---------------------------------------------------------- waits that run out
@pytest.mark.parametrize("n,k,stages", [(4096, 256, (0, 2, 5, 8)), (200, 1536, (1, 7, 8, 19, 24))])
def test_expert_linear_whose_copies_stop(dev, n, k, stages):  # noqa: F811
    """The packed weights of each CTA stop at some stage of its tiles: every role's wait runs
    out, the call ends with its status bit, tiles that were complete are right and others not
    written, and the next call finds everything as ever."""
    experts, tokens = 8, 320
    layer = Layer(dev, experts, n, k, 4, F16, seed=k)
    x = normal(1, tokens, k).to(F16).to(dev)
    which = np.arange(tokens) % experts
    routing = routing_of(which[:, None], experts, dev)
    args = (x, routing, layer.wq, layer.scales, layer.biases, 4)
    ref = q.expert_linear(*args)
    size = q.lib().qlin_expert_linear_workspace_size(tokens, experts, n, k)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    blocks = (n + 127) // 128
    tile = which[:, None] * blocks + np.arange(n)[None, :] // 128  # of each output
    for stage in stages:
        out = torch.full_like(ref, 5.0)
        status = q.lib().qlin_testing_expert_linear_stalled(
            x.data_ptr(), k, 1, routing.order.data_ptr(), routing.offsets.data_ptr(), tokens,
            layer.wq.data_ptr(), layer.scales.data_ptr(), layer.biases.data_ptr(), out.data_ptr(),
            experts, n, k, ws.data_ptr(), size, stage, 2000,
            torch.cuda.current_stream().cuda_stream)
        assert status == 0
        complete = torch.from_numpy(tile < sms * (stage * 64 // k)).to(dev)
        assert q.device_status() == (0 if complete.all() else 1 << 30)
        assert torch.equal(out[complete], ref[complete]) and (out[~complete] == 5).all()
        assert torch.equal(q.expert_linear(*args, overlap_previous=True), ref)
        assert q.device_status() == 0


@pytest.mark.parametrize("dt,experts,rows,n,k", [(F16, 64, 11800, 680, 3712), (BF16, 16, 1688, 3000, 3392),
                                                 (F16, 8, 545, 4078, 3520), (BF16, 128, 8388, 310, 3712)])
@pytest.mark.parametrize("bits", [4, 8])
def test_expert_linear_of_long_rows_at_full_speed(dev, bits, dt, experts, rows, n, k):  # noqa: F811
    """Many tiles of long rows, whose scales no longer stay in L1: no packed tile is overwritten
    before it was read.  Ten calls, every output against products in 32 bits."""
    gen = torch.Generator(device=dev).manual_seed(k)
    w = torch.randn(experts * n, k, generator=gen, device=dev) / k ** 0.5
    wq, sc, bi = q.quantize_affine(w, bits, sdtype=dt)
    del w
    which = torch.randint(0, experts, (rows,), generator=gen, device=dev)
    routing = routing_of(which[:, None].cpu().numpy(), experts, dev)
    x = torch.randn(rows, k, generator=gen, device=dev).to(dt)
    hat = q.dequant(wq, sc, bi, bits, out_dtype=F32).view(experts, n, k)
    ref, size = torch.empty(rows, n, device=dev), torch.empty(rows, n, device=dev)
    for e in range(experts):
        at = which == e
        ref[at], size[at] = x[at].float() @ hat[e].T, x[at].float().abs() @ hat[e].abs().T
    # the weight's rounding to f16 (bf16: and 2^-31 of its row's largest, nothing here), float32
    # sums of k products in each of two (an outer bound: each addition off by 2^-24 of the sum
    # of magnitudes), the output's rounding
    bound = (2.0 ** -11 + 2 * k * 2.0 ** -24) * size + U[dt] * ref.abs() + TINY[dt]
    packed = [t.view(experts, n, -1) for t in (wq, sc, bi)]
    for call in range(10):
        out = q.expert_linear(x, routing, *packed, bits).float()
        bad = ~((out - ref).abs() <= bound)
        assert not bad.any(), (call, int(bad.sum()), bad.nonzero()[:3].tolist())
    assert q.device_status() == 0


# ------------------------------------- rings that bulk copies fill while warps read them
@pytest.mark.parametrize("bits,dt", [(4, BF16), (8, F16)])
@pytest.mark.parametrize("n,k,m", [(20000, 8256, 1), (9000, 3712, 3), (30000, 2048, 2)])
def test_linear_is_the_same_at_full_speed(dev, bits, dt, n, k, m):  # noqa: F811
    """Rows with and without a tile's scales beside them: thirty calls in a row, one result, and
    that within float32 sums of the dequantised product."""
    gen = torch.Generator(device=dev).manual_seed(k)
    packed = q.quantize_affine(torch.randn(n, k, generator=gen, device=dev) / k ** 0.5, bits,
                               sdtype=dt)
    x = torch.randn(m, k, generator=gen, device=dev).to(dt)
    outs = [q.linear(x, *packed, bits) for _ in range(30)]
    assert all(torch.equal(o, outs[0]) for o in outs)
    hat, xf = q.dequant(*packed, bits, out_dtype=F32).double(), x.double()
    ref, size = xf @ hat.T, xf.abs() @ hat.abs().T
    # sums of (magic + code) * x: up to 2^9 steps of the group's scale beside the code, k float32
    # additions of what is at most that; the output's rounding
    step = xf.abs() @ packed[1].double().abs().repeat_interleave(64, 1).T
    bound = U[dt] * ref.abs() + k * 2.0 ** -24 * size + 2.0 ** 9 * 2.0 ** -18 * step + TINY[dt]
    assert ((outs[0].double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("context,slots", [(30000, 2), (900, 24)])
def test_cache_attention_is_the_same_at_full_speed(dev, context, slots):  # noqa: F811
    cache = q.KVCache.empty(slots, context + 64, 8, 64, device=dev)
    ws = q.attention_workspace(64)
    starts = torch.arange(slots + 1, dtype=torch.int32, device=dev)
    filled = starts * context
    qkv = normal(3, slots * context, 48 * 64).to(F16).to(dev)
    q.rope_append(qkv, None, cache, filled, 32)
    cache.lens += context
    new = normal(4, slots, 48 * 64).to(F16).to(dev)
    query = q.rope_append(new, None, cache, starts, 32)
    outs = [q.cache_attention(query, cache, starts, 1, ws) for _ in range(30)]
    assert all(torch.equal(o, outs[0]) for o in outs) and outs[0].isfinite().all()
    assert q.device_status() == 0
