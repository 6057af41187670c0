"""GPU parity of routing, the experts' products and their sum, norms of query and key
heads, and log probabilities against the float64 oracle.

Tolerances count the roundings that the definitions name (u = 2^-11 for f16, 2^-8 for
bf16: one rounding to nearest of a result) plus the float32 operations behind them;
each test says how."""

import math

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from oracle import experts_oracle as O
from tests.test_gpu_decoder import Model, U, TINY, close, f64, normal, table_for

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_qmv_qmm_gb300 import build_lib
    build_lib.build()
    q.lib()
    yield torch.device("cuda:0")
    assert q.device_status() == 0


def strided(t, pad):
    """t's values in rows pad elements further apart."""
    buf = torch.empty(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf[:, : t.shape[1]]


# ------------------------------------------------------------------- routing
def check_route(x, top_k, bias=None, **kw):
    r = q.route_experts(x, top_k, bias=bias, **kw)
    rows, n = x.shape
    got_e, got_w = r.experts.cpu().numpy(), f64(r.weights)
    xs, b = f64(x), None if bias is None else f64(bias)
    near = 0
    for t in range(rows):
        e, w, margin = O.route(xs[t], top_k, bias=b, **kw)
        # Choices are float32: a sigmoid, a share or a sum of two is off by at most 2^-21 of
        # its size, which is at most 2 + the bias; closer ones can fall either way.
        if margin <= 2.0 ** -20 * (2 + (0 if b is None else np.abs(b).max())):
            near += 1
            continue
        assert np.array_equal(got_e[t], e), t
        # weights: a score and a sum of at most 512 scores, each off by at most 8 float32
        # steps (exp of an argument up to 100 rounded once: 2^-24 * 100 more), and two
        # operations
        err = np.abs(got_w[t] - w)
        assert (err <= (2.0 ** -19 + 2.0 ** -21) * np.abs(w) + 1e-37).all(), (t, err.max())
    assert near <= rows // 20 + 1, "the inputs have too many near ties to say anything"
    order, offsets = O.plan(got_e, n)
    assert np.array_equal(r.order.cpu().numpy(), order), "order"
    assert np.array_equal(r.offsets.cpu().numpy(), offsets), "offsets"
    return r


@pytest.mark.parametrize("rows", [1, 2, 16, 63, 64, 65, 300, 2500])
def test_route_rows(dev, rows):
    check_route((normal(rows, rows, 64) * 2).to(F32).to(dev), 8)


@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 2), (31, 4), (32, 32), (33, 5), (60, 6),
                                           (128, 1), (129, 8), (256, 8), (257, 9), (512, 32)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_route_experts_and_types(dev, experts, top_k, dt):
    for rows in (5, 200):
        x = strided((normal(experts, rows, experts) * 2).to(dt).to(dev), 3)
        check_route(x, top_k)
        check_route(x, top_k, scoring="sigmoid", renormalise=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("experts,groups,top_groups", [(64, 1, 1), (64, 8, 3), (60, 4, 1),
                                                       (256, 8, 4), (96, 32, 5), (32, 32, 9),
                                                       (510, 3, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups_and_bias(dev, scoring, group_score, experts, groups, top_groups, biased):
    x = (normal(3, 150, experts) * 1.5).to(F32).to(dev)
    bias = (0.3 * normal(4, experts)).float().to(dev) if biased else None
    for renormalise in (True, False):
        check_route(x, min(6, experts // groups * top_groups), bias=bias, scoring=scoring,
                    groups=groups, top_groups=top_groups, group_score=group_score,
                    renormalise=renormalise, scale=1.5)


def test_route_masked_and_special_rows(dev):
    inf, nan = math.inf, math.nan
    x = torch.zeros(8, 40, device=dev)
    x[0] = -inf                       # nothing
    x[1] = nan
    x[2] = -inf
    x[2, 7] = -3.0                    # fewer than top_k
    x[3, 5] = inf                     # only the infinite ones have a share
    x[3, 9] = inf
    x[4] = 1.0                        # all equal: by index
    x[5, ::2] = nan
    x[6] = torch.arange(40.) * 1e30   # exponentials of 0
    x[7, 3] = -0.0                    # as 0
    r = check_route(x, 4)
    e, w = r.experts.cpu(), r.weights.cpu()
    assert (e[0] == -1).all() and (e[1] == -1).all() and (w[:2] == 0).all()
    assert e[2].tolist() == [7, -1, -1, -1] and w[2].tolist() == [1, 0, 0, 0]
    assert e[3, :2].tolist() == [5, 9] and w[3].tolist() == [0.5, 0.5, 0, 0]
    assert e[4].tolist() == [0, 1, 2, 3] and e[5].tolist() == [1, 3, 5, 7]
    assert e[7].tolist() == [0, 1, 2, 3]
    assert int(r.offsets[-1]) == int((e >= 0).sum())
    check_route(x, 4, groups=4, top_groups=2)
    check_route(x, 4, groups=4, top_groups=2, group_score="top2", scoring="sigmoid")
    # a bias that is no number takes its expert out
    bias = torch.zeros(40, device=dev)
    bias[0] = nan
    r = q.route_experts(x[4:5], 2, bias=bias)
    assert r.experts.tolist() == [[1, 2]]
    assert q.route_experts(x[:0], 4).offsets.tolist() == [0] * 41


def test_route_is_the_same_again_and_in_a_graph(dev):
    x = normal(9, 700, 128).float().to(dev)
    first = q.route_experts(x, 8, scoring="sigmoid", groups=8, top_groups=4, group_score="top2")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.route_experts(x, 8)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = q.route_experts(x, 8, scoring="sigmoid", groups=8, top_groups=4,
                                group_score="top2", overlap_previous=True)
    y = x.clone()
    x.copy_(normal(10, 700, 128))
    g.replay()
    x.copy_(y)
    g.replay()
    for name in ("experts", "weights", "order", "offsets"):
        assert torch.equal(getattr(first, name), getattr(again, name)), name


def test_routing_tensors_cannot_be_replaced(dev):
    """Its calls read the memory that it was made with; writing into it works."""
    r = q.route_experts(normal(1, 4, 8).float().to(dev), 2)
    for routing in (r, q.Routing(r.experts, r.weights, r.order, r.offsets)):
        with pytest.raises(AttributeError):
            routing.weights = r.weights * 2
        before = routing.weights.clone()
        routing.weights *= 2
        y = torch.ones(8, 16, dtype=F16, device=dev)
        out = q.combine_experts(y, routing)
        assert torch.allclose(out[:, 0].float(), 2 * before.sum(1), rtol=1e-3)
        routing.weights.copy_(before)
    for bad in (dict(experts=r.experts.long()), dict(weights=r.weights.half()),
                dict(order=r.order[:7]), dict(offsets=r.offsets[:, None]),
                dict(order=r.order.cpu())):
        with pytest.raises(ValueError):
            q.Routing(**{**dict(experts=r.experts, weights=r.weights, order=r.order,
                                offsets=r.offsets), **bad})


# ------------------------------------------------------------ experts' products
class Layer:
    """Packed weights of experts on the GPU beside their float64 values."""

    def __init__(self, dev, experts, n, k, bits, dt, seed=0):
        rng = np.random.default_rng(seed)
        w = torch.from_numpy(rng.standard_normal((experts * n, k)).astype(np.float32) / k ** 0.5)
        wq, sc, bi = q.quantize_affine(w.to(dev), bits, sdtype=dt)
        self.bits, self.dt, self.dev = bits, dt, dev
        self.wq, self.scales, self.biases = (t.view(experts, n, -1) for t in (wq, sc, bi))
        code = wq.cpu().numpy().view(np.uint32)[..., None] >> np.arange(0, 32, bits, dtype=np.uint32)
        code = (code & (2 ** bits - 1)).reshape(experts, n, k // 64, 64).astype(np.float64)
        s, b = (f64(t)[..., None] for t in (self.scales, self.biases))
        self.w = (code * s + b).reshape(experts, n, k)
        self.step = np.broadcast_to(s, code.shape).reshape(experts, n, k)

    def check(self, x, routing, out_dtype=None, out=None, overlap=False):
        got = q.expert_linear(x, routing, self.wq, self.scales, self.biases, self.bits, out=out,
                              out_dtype=out_dtype, overlap_previous=overlap)
        xs, y = f64(x), f64(got)
        experts = routing.experts.cpu().numpy().reshape(-1)
        per_pair = len(xs) == len(experts)
        u = U[got.dtype]
        for e in np.unique(experts[experts >= 0]):
            p = np.flatnonzero(experts == e)
            rows = xs[p if per_pair else p // routing.top_k]
            ref = rows @ self.w[e].T
            size = np.abs(rows) @ np.abs(self.w[e]).T
            step = np.abs(rows) @ self.step[e].T
            # The output's rounding; a weight's rounding to f16 where it is an operand (2^-11
            # of it; bf16 keeps 2^-15); and float32 sums over codes of 4 or 8 bits under the
            # unit 1024 or 32768 of what they are placed in, which costs 1024 steps times a
            # few 2^-22 (32768 times a few 2^-24 with a float32 unit).
            bound = u * np.abs(ref) + 2.0 ** -11 * size + 2.0 ** -9 * step + 1e-7 * size
            bound += TINY[got.dtype]
            err = np.abs(y[p] - ref)
            assert (err <= bound).all(), (e, len(p), float((err / bound).max()))
        return got


def routing_of(experts, n, dev, seed=0):
    experts = np.asarray(experts, np.int32)
    order, offsets = O.plan(experts, n)
    w = np.random.default_rng(seed).random(experts.shape, np.float32)
    return q.Routing(*(torch.from_numpy(np.ascontiguousarray(t)).to(dev) for t in
                       (experts, w, order.astype(np.int32), offsets.astype(np.int32))))


def random_experts(seed, tokens, top_k, n, skew=0.0):
    rng = np.random.default_rng(seed)
    like = rng.standard_normal((tokens, n)) + skew * rng.standard_normal(n)
    return np.argsort(-like, 1)[:, :top_k]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("n,k", [(1, 64), (7, 128), (64, 192), (130, 320), (129, 1088), (256, 512),
                                 (16, 2048), (40, 4160)])
def test_expert_linear_sizes(dev, bits, dt, n, k):
    layer = Layer(dev, 6, n, k, bits, dt, seed=n)
    for tokens, top_k in ((1, 2), (9, 3), (70, 4)):
        routing = routing_of(random_experts(tokens, tokens, top_k, 6), 6, dev)
        layer.check(normal(1, tokens, k).to(dt).to(dev), routing)
        x = strided(normal(2, tokens * top_k, k).to(dt).to(dev), 8)
        layer.check(x, routing, out_dtype=F32)


@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16), (8, F16), (4, BF16)])
@pytest.mark.parametrize("counts", [(0, 0, 1), (1, 0, 8), (9, 16, 17), (33, 0, 31), (64, 65, 1),
                                    (129, 127, 255), (256, 257, 3), (600, 0, 0), (1, 1, 1300)])
def test_expert_linear_rows_of_every_number(dev, bits, dt, counts):
    """Experts with these numbers of rows, among others that have none."""
    layer = Layer(dev, 8, 200, 256, bits, dt, seed=7)
    rng = np.random.default_rng(sum(counts))
    experts = np.concatenate([np.full(c, e) for e, c in zip((1, 4, 7), counts)])
    experts = rng.permutation(experts)[:, None]
    layer.check(normal(3, len(experts), 256).to(dt).to(dev), routing_of(experts, 8, dev))


def test_expert_linear_many_rows(dev):
    """Thousands of rows on few experts; the plan from route_experts."""
    layer = Layer(dev, 4, 384, 512, 4, F16)
    x = normal(4, 3000, 512).to(F16).to(dev)
    routing = q.route_experts(normal(5, 3000, 4).float().to(dev), 2)
    layer.check(x, routing)
    layer = Layer(dev, 4, 96, 128, 8, BF16)
    layer.check(normal(4, 3000, 128).to(BF16).to(dev), routing)


@pytest.mark.parametrize("tokens", [3, 200, 1500])
def test_expert_linear_leaves_rows_without_an_expert(dev, tokens):
    layer = Layer(dev, 5, 72, 128, 8, F16)
    experts = random_experts(1, tokens, 2, 5)
    experts[1] = -1
    experts[::4, 1] = -1
    routing = routing_of(experts, 5, dev)
    out = torch.full((tokens * 2, 72), 77.0, dtype=F16, device=dev)
    x = normal(1, tokens, 128).to(F16).to(dev)
    x[1] = math.nan  # a token without experts is not read
    layer.check(x, routing, out=out)
    none = torch.from_numpy(experts.reshape(-1) < 0).to(dev)
    assert (out[none] == 77).all() and not (out[~none] == 77).all()
    # no token at all, and tokens without any expert
    out.fill_(77)
    q.expert_linear(x, routing_of(np.full((tokens, 2), -1), 5, dev), layer.wq, layer.scales,
                    layer.biases, 8, out=out)
    assert (out == 77).all()
    got = q.expert_linear(x[:0], routing_of(np.zeros((0, 2)), 5, dev), layer.wq, layer.scales,
                          layer.biases, 8)
    assert got.shape == (0, 72)


@pytest.mark.parametrize("tokens", [4, 300])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_expert_linear_rows_do_not_touch_each_other(dev, tokens, dt):
    """A row of NaN or infinity reaches its own outputs only; a row of zeros gives zeros."""
    layer = Layer(dev, 3, 130, 192, 4, dt)
    experts = random_experts(2, tokens, 1, 3)
    routing = routing_of(experts, 3, dev)
    x = normal(1, tokens, 192).to(dt).to(dev)
    ref = q.expert_linear(x, routing, layer.wq, layer.scales, layer.biases, 4)
    x[1], x[2], x[3, 5] = math.nan, 0.0, math.inf
    got = q.expert_linear(x, routing, layer.wq, layer.scales, layer.biases, 4)
    assert got[1].isnan().all() and (got[2] == 0).all() and not got[3].isfinite().any()
    keep = [i for i in range(tokens) if i not in (1, 2, 3)]
    assert torch.equal(got[keep], ref[keep])


def test_expert_linear_bad_plans_are_left_out(dev):
    layer = Layer(dev, 4, 40, 64, 8, F16)
    for tokens in (6, 600):
        routing = routing_of(random_experts(1, tokens, 1, 4), 4, dev)
        x = normal(1, tokens, 64).to(F16).to(dev)
        good = layer.check(x, routing)
        assert q.device_status() == 0
        keep = routing.offsets.clone()
        for bad in (-5, 1 << 30):
            routing.offsets[1] = bad
            out = torch.full_like(good, 5.0)
            q.expert_linear(x, routing, layer.wq, layer.scales, layer.biases, 8, out=out)
            assert q.device_status() == 1 << 30
            own = torch.from_numpy(np.isin(routing.experts.cpu().numpy()[:, 0], (2, 3))).to(dev)
            assert torch.equal(out[own], good[own]) and (out[~own] == 5).all()
            routing.offsets.copy_(keep)
        first = int(routing.order[0])
        for bad in (-1, tokens, 1 << 30):
            routing.order[0] = bad
            out = torch.full_like(good, 5.0)
            q.expert_linear(x, routing, layer.wq, layer.scales, layer.biases, 8, out=out)
            assert q.device_status() == 1 << 30
            rest = [i for i in range(tokens) if i != first]
            assert torch.equal(out[rest], good[rest]) and (out[first] == 5).all()
            routing.order[0] = first


def test_expert_linear_binding_refusals(dev):
    layer = Layer(dev, 4, 40, 64, 8, F16)
    routing = routing_of(random_experts(1, 6, 2, 4), 4, dev)
    x = normal(1, 6, 64).to(F16).to(dev)
    good = dict(x=x, routing=routing, wq=layer.wq, scales=layer.scales, biases=layer.biases, bits=8)
    q.expert_linear(**good)
    for bad in (dict(x=x[:5]), dict(x=x.float()), dict(x=x[:, :32]), dict(bits=4),
                dict(wq=layer.wq[:3]), dict(scales=layer.scales.float()),
                dict(biases=layer.biases[:, :20]), dict(out_dtype=BF16),
                dict(out=torch.zeros(6, 40, dtype=F16, device=dev)),
                dict(wq=layer.wq.cpu()), dict(scales=layer.scales.cpu())):
        with pytest.raises(ValueError):
            q.expert_linear(**{**good, **bad})
    with pytest.raises(q.QlinError):  # rows of x that start off 16 bytes
        q.expert_linear(**{**good, "x": strided(x, 3)})


# ------------------------------------------------------------------ their sum
@pytest.mark.parametrize("dt,ydt", [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("tokens,top_k,n", [(1, 1, 1), (3, 8, 2048), (5, 9, 100), (2, 32, 63),
                                            (300, 4, 512), (7, 2, 8200)])
def test_combine(dev, dt, ydt, tokens, top_k, n):
    experts = random_experts(1, tokens, top_k, 40)
    experts[0, top_k // 2:] = -1
    routing = routing_of(experts, 40, dev)
    y = (3 * normal(1, tokens * top_k, n)).to(ydt).to(dev)
    y.view(tokens, top_k, n)[0, top_k // 2:] = math.nan  # rows that nothing has written
    w = f64(routing.weights)
    for add in (None, strided(normal(2, tokens, n).to(dt).to(dev), 8),
                strided(normal(2, tokens, n).to(dt).to(dev), 3)):
        ref, size = O.combine(f64(y).reshape(tokens, top_k, n), experts, w,
                              None if add is None else f64(add))
        out = q.combine_experts(y, routing, add=add, out_dtype=dt)
        # one rounding, and top_k + 1 float32 operations on the sum of magnitudes
        close(out, ref, U[dt] * np.abs(ref) + (top_k + 1) * 2.0 ** -24 * size + TINY[dt])
    add = normal(2, tokens, n).to(dt).to(dev)
    ref = q.combine_experts(y, routing, add=add)
    assert torch.equal(q.combine_experts(y, routing, add=add, out=add), ref)


def test_combine_binding_refusals(dev):
    routing = routing_of(random_experts(1, 6, 2, 4), 4, dev)
    y = torch.zeros(12, 64, dtype=F16, device=dev)
    for bad in (dict(y=y[:6]), dict(y=y.float()), dict(y=y.cpu()), dict(y=y[:, ::2]),
                dict(add=y[:5]), dict(add=y[:6].float()), dict(out=y[:5]),
                dict(out_dtype=BF16)):
        with pytest.raises(ValueError):
            q.combine_experts(**{"y": y, "routing": routing, **bad})
    assert q.combine_experts(y[:0], routing_of(np.zeros((0, 2)), 4, dev)).shape == (0, 64)


# --------------------------------------------- norms of heads with the rotation
class NormedModel(Model):
    """A cache that is filled through the norms."""

    def __init__(self, dev, slots, kv_heads, d, dt, eps=1e-6, **kw):
        super().__init__(dev, slots, kv_heads, d, dt, **kw)
        self.q_norm = (1 + 0.3 * normal(91, d)).to(dt).to(dev)
        self.k_norm = (1 + 0.3 * normal(92, d)).to(dt).to(dev)
        self.eps = eps

    def append(self, new, heads, table, interleaved=False, seed=0, pad=0, scale=1.0,
               overlap=False):
        rows, width = sum(new), (heads + 2 * self.kvh) * self.d
        buf = torch.zeros(rows, width + pad, dtype=self.dt, device=self.dev)
        qkv = buf[:, :width]
        qkv.copy_((normal(seed, rows, width) * scale).to(self.dt))
        out = q.rope_append(qkv, table, self.cache, self.starts(new), heads, interleaved,
                            q_norm=self.q_norm, k_norm=self.k_norm, eps=self.eps,
                            overlap_previous=overlap)
        x = f64(qkv).reshape(rows, -1, self.d)
        pos = np.concatenate([len(self.k[b]) + np.arange(n) for b, n in enumerate(new)]).astype(int)
        qk = np.concatenate((O.head_norm(x[:, :heads], f64(self.q_norm), self.eps),
                             O.head_norm(x[:, heads:heads + self.kvh], f64(self.k_norm),
                                         self.eps)), 1)
        size = np.abs(qk)
        if table is not None:
            t = f64(table)[pos]
            half = t.shape[1]
            a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                    else (slice(0, half), slice(half, 2 * half)))
            c, s = t[:, None, :, 0], t[:, None, :, 1]
            xa, xb = qk[..., a].copy(), qk[..., b].copy()
            qk[..., a], qk[..., b] = xa * c - xb * s, xb * c + xa * s
            size[..., a] = size[..., b] = np.abs(xa) + np.abs(xb)
        # one rounding; behind it the sum of squares (2^-20 with its root and quotient) and
        # five float32 operations on magnitudes up to size
        self.bound = U[self.dt] * np.abs(qk) + 2.0 ** -19 * size + TINY[self.dt]
        self.close = close(out, qk[:, :heads], self.bound[:, :heads], "queries")
        at = 0
        for b, n in enumerate(new):
            self.k[b] = np.concatenate([self.k[b], qk[at:at + n, heads:]])
            self.v[b] = np.concatenate([self.v[b], x[at:at + n, heads + self.kvh:]])
            at += n
        self.cache.lens += torch.tensor(new, dtype=torch.int32, device=self.dev)
        return out

    def check(self):
        """Tails are the normed keys and the values; blocks hold them to a step: a key's
        rounding to dtype can move its code by one, the scale by that rounding."""
        c, d = self.cache, self.d
        pages, scales, table = f64(c.pages), f64(c.scales), c.table.cpu().numpy()
        tail = f64(c.tail)
        u = 2 * U[self.dt] + 2.0 ** -18
        for b in range(self.slots):
            n = len(self.k[b])
            for j in range(n // 64):
                at = slice(j * 64, (j + 1) * 64)
                for h in range(self.kvh):
                    for i, block in enumerate((self.k[b][at, h], self.v[b][at, h].T)):
                        scale = scales[table[b, j], h, i]
                        assert abs(scale - np.abs(block).max() / 127) <= u * scale
                        got = (pages[table[b, j], h, i].reshape(block.shape) - 128) * scale
                        # half a step of the code, and the element's own rounding
                        assert (np.abs(got - block) <= scale * 0.501 + 2 * u * np.abs(block)).all()
            left, at = n % 64, slice(n - n % 64, n)
            for h in range(self.kvh):
                key = self.k[b][at, h]
                err = np.abs(tail[b, h, 0].reshape(64, d)[:left] - key)
                size = np.abs(key).max(-1, keepdims=True) if left else 0
                assert (err <= U[self.dt] * np.abs(key) + 2.0 ** -18 * size + TINY[self.dt]).all()
                assert np.array_equal(tail[b, h, 1].reshape(d, 64)[:, :left], self.v[b][at, h].T)


@pytest.mark.parametrize("d,rot,interleaved,dt", [(64, 64, False, F16), (128, 128, True, BF16),
                                                  (128, 48, False, F16), (64, 32, True, BF16),
                                                  (64, 16, False, BF16), (128, 0, False, F16)])
def test_norm_append_in_calls_of_every_size(dev, d, rot, interleaved, dt):
    m = NormedModel(dev, 4, 3, d, dt)
    table = table_for(dev, rot)
    calls = [(1, 63, 64, 65), (0, 1, 1, 62), (62, 1, 0, 1), (2, 200, 130, 0), (1, 1, 1, 1),
             (127, 3, 61, 64), (1, 0, 0, 0)]
    for i, new in enumerate(calls):
        m.append(new, 6, table, interleaved, seed=i, pad=8 * (i % 2), overlap=i % 3 == 2)
        m.check()


@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1e-3, 0.0), (300.0, 1e-6), (1.0, 10.0)])
def test_norm_append_scales(dev, scale, eps):
    m = NormedModel(dev, 2, 2, 64, F16, eps=eps)
    m.append((70, 5), 4, table_for(dev, 64), scale=scale)
    m.check()


def test_norm_append_zero_and_special_heads(dev):
    """A head of zeros stays zeros; one with a NaN or an infinity reaches itself only."""
    m = NormedModel(dev, 1, 2, 64, F16)
    qkv = normal(1, 3, 8 * 64).to(F16).to(dev)
    ref = q.rope_append(qkv, None, m.cache, m.starts((3,)), 4, q_norm=m.q_norm, k_norm=m.k_norm)
    qkv[0, :64], qkv[1, 64], qkv[2, 130] = 0, math.nan, math.inf
    out = q.rope_append(qkv, None, m.cache, m.starts((3,)), 4, q_norm=m.q_norm, k_norm=m.k_norm)
    assert (out[0, 0] == 0).all() and out[1, 1].isnan().all()
    assert out[2, 2, 2].isnan() and (out[2, 2, 3:] == 0).all()
    out[0, 0], out[1, 1], out[2, 2] = ref[0, 0], ref[1, 1], ref[2, 2]
    assert torch.equal(out, ref)


def test_norm_append_binding_refusals(dev):
    m = NormedModel(dev, 1, 2, 64, F16)
    qkv = torch.zeros(3, 8 * 64, dtype=F16, device=dev)
    for bad in (dict(k_norm=None), dict(q_norm=None), dict(q_norm=m.q_norm[:32]),
                dict(k_norm=m.k_norm.float()), dict(k_norm=m.k_norm.cpu())):
        with pytest.raises(ValueError):
            q.rope_append(qkv, None, m.cache, m.starts((3,)), 4,
                          **{"q_norm": m.q_norm, "k_norm": m.k_norm, **bad})
    with pytest.raises(q.QlinError):
        q.rope_append(qkv, None, m.cache, m.starts((3,)), 4, q_norm=m.q_norm, k_norm=m.k_norm,
                      eps=-1.0)


# ------------------------------------------------------------ log probabilities
def check_logprobs(x, tokens, top, overlap=False):
    lp, h, tt, tl = q.token_logprobs(x, tokens, top, overlap_previous=overlap)
    assert tt.shape == tl.shape == (len(x), top) and tt.dtype == torch.int32
    xs, v = f64(x), x.shape[1]
    for m in range(len(x)):
        r_lp, r_h, r_t, r_l = O.logprobs(xs[m], int(tokens[m]), top)
        # float32 ends at 2^128 - 2^104: what is beyond it by more than half a step, 2^103, is
        # infinite there (-3e38 under a largest logit of 3e38: -6e38 = -1.76 * 2^128)
        end = 2.0 ** 128 - 2.0 ** 103
        r_lp = -np.inf if r_lp <= -end else r_lp
        r_l = np.where(r_l <= -end, -np.inf, r_l)
        # exp's argument is rounded to 2^-24 of it (at most 128, for terms that count) and exp
        # is 2 ulp off; float32 sums of positive terms, at most 2^-15 for 2^18 of them one by
        # one, here in 512 or more parts: 2^-20 of log z and of the mean; the logarithm and a
        # difference: 2^-23 of the values
        size = 1 + abs(math.log(v))
        assert np.isclose(f64(lp)[m], r_lp, rtol=2.0 ** -21, atol=2.0 ** -20 * size), m
        assert np.isclose(f64(h)[m], r_h, rtol=2.0 ** -20, atol=2.0 ** -19 * size), m
        assert np.array_equal(tt[m].cpu().numpy(), r_t), m
        got = f64(tl)[m]
        fin = np.isfinite(r_l)
        assert np.array_equal(got[~fin], r_l[~fin])
        assert (np.abs(got[fin] - r_l[fin])
                <= 2.0 ** -21 * np.abs(r_l[fin]) + 2.0 ** -20 * size).all(), m


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 5), (3, 31), (1, 1000), (5, 4097), (2, 32000),
                                        (1, 128256), (3, 262144), (40, 151), (200, 2049),
                                        (400, 517)])
def test_logprobs_sizes(dev, dt, rows, vocab):
    x = (2.5 * normal(vocab, rows, vocab)).to(dt).to(dev)
    tokens = torch.from_numpy(np.random.default_rng(1).integers(0, vocab, rows).astype(np.int32))
    for top, pad in ((0, 0), (1, 8), (20, 3), (32, 0)):
        check_logprobs(strided(x, pad) if pad else x, tokens.to(dev), top)


@pytest.mark.parametrize("vocab", [40, 700, 20000])
def test_logprobs_special_rows(dev, vocab):
    inf, nan = math.inf, math.nan
    x = normal(1, 12, vocab).float()
    x[0] = -inf
    x[1] = nan
    x[2] = -inf
    x[2, 7] = -3.0                    # one token
    x[3, [5, 9]] = inf                # infinite ones share
    x[4] = 1.25                       # all equal
    x[5, ::2] = nan
    x[6] = torch.arange(vocab) * 1e30
    x[7] = torch.arange(vocab) % 5    # many equal
    x[8, 3:] = -inf                   # fewer than top
    x[9] = -3e38
    x[9, -1] = 3e38
    x[10, 0] = 200.0                  # all but certain
    x[11] = -x[11].abs() - 1e4
    tokens = torch.tensor([0, 0, 7, 5, 11, 2, 3, vocab - 1, 2, vocab - 1, 0, 4],
                          dtype=torch.int32)
    for dt in (F32, BF16):
        for top in (0, 20, 32):
            check_logprobs(x.to(dt).to(dev), tokens.to(dev), top)
    # tokens that are none
    tokens[:] = -1
    tokens[3], tokens[4] = vocab, 1 << 30
    lp, h, _, _ = q.token_logprobs(x.to(dev), tokens.to(dev))
    assert (lp == -inf).all() and not h.isnan().any()


@pytest.mark.parametrize("rows", [1, 500])
def test_logprobs_where_a_few_threads_have_all_large_logits(dev, rows):
    """31 of every 256 neighbourhoods of 16 bytes hold thousands of logits above the 32nd
    neighbourhood's best: more than are ranked by counting."""
    v = 65536
    x = normal(1, rows, v).to(F16)
    at = torch.arange(v) // 8 % 256
    x[:, at < 31] = (100 + normal(2, rows, int((at < 31).sum()))).to(F16)
    x[:, 31 * 8 + 5] = 50.0
    tokens = torch.full((rows,), 3, dtype=torch.int32)
    if rows == 1:
        check_logprobs(x.to(dev), tokens.to(dev), 32)
        return
    _, _, tt, tl = q.token_logprobs(x.to(dev), tokens.to(dev), 32)
    for m in range(0, rows, 83):
        ref = O.logprobs(f64(x)[m], 3, 32)
        assert np.array_equal(tt[m].cpu().numpy(), ref[2])
        assert np.allclose(f64(tl)[m], ref[3], atol=2.0 ** -16)


def test_logprobs_of_what_sample_drew(dev):
    """The likeliest token's log probability is the greedy draw's, and a draw's share of
    all logits its probability."""
    x = (2 * normal(3, 50, 5000)).to(F16).to(dev)
    m = len(x)
    one, zero = torch.ones(m, device=dev), torch.zeros(m, device=dev)
    none = torch.zeros(m, dtype=torch.int32, device=dev)
    token, prob = q.sample(x, torch.rand(m, device=dev), one, none, one, zero)
    lp, _, _, _ = q.token_logprobs(x, token)
    assert torch.allclose(lp.exp(), prob, rtol=2e-6, atol=0)
    token, _ = q.sample(x, zero, zero, none, one, zero)
    lp, _, tt, tl = q.token_logprobs(x, token, 1)
    assert torch.equal(tt[:, 0], token) and torch.equal(tl[:, 0], lp)


def test_logprobs_binding_refusals(dev):
    x = torch.zeros(3, 10, device=dev)
    t = torch.zeros(3, dtype=torch.int32, device=dev)
    for args in ((x, t[:2]), (x, t.long()), (x, t.cpu()), (x.double(), t), (x[0], t), (x, t, 33),
                 (x, t, -1), (x.t(), t)):
        with pytest.raises(ValueError):
            q.token_logprobs(*args)
    out = q.token_logprobs(x[:0], t[:0], 4)
    assert [o.shape for o in out] == [(0,), (0,), (0, 4), (0, 4)]


# ------------------------------------------------------- a K of any length
@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16)])
@pytest.mark.parametrize("k", [4544, 4608, 8384, 8512, 12800])
def test_expert_linear_long_rows(dev, bits, dt, k):
    """Around the lengths whose tokens still fit beside the weights on their way."""
    layer = Layer(dev, 3, 48, k, bits, dt, seed=k)
    for tokens in (1, 11):
        layer.check(normal(1, tokens, k).to(dt).to(dev),
                    routing_of(random_experts(3, tokens, 2, 3), 3, dev))


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e30])
def test_expert_linear_bfloat16_of_any_size(dev, scale):
    """Tokens and weights far from 1, and a token whose elements are far apart: the powers
    of two that bring them to f16 have to be undone."""
    for tokens in (4, 200):
        layer = Layer(dev, 3, 72, 192, 8, BF16)
        layer.scales.mul_(2.0 ** -20)
        layer.biases.mul_(2.0 ** -20)
        layer.w *= 2.0 ** -20
        layer.step = layer.step * 2.0 ** -20
        x = (normal(1, tokens, 192) * scale).to(BF16)
        x[1, :64] *= 2.0 ** -12
        layer.check(x.to(dev), routing_of(random_experts(3, tokens, 1, 3), 3, dev), out_dtype=F32)


# ------------------------------------------------- more elements than 32 bits count
def test_expert_linear_past_32_bits(dev):
    """Outputs of 2.3e9 elements: the last pairs' rows are where they belong."""
    n, pairs = 70000, 33000
    layer = Layer(dev, 1, n, 64, 4, F16)
    x = normal(1, pairs, 64).to(F16).to(dev)
    y = q.expert_linear(x, routing_of(np.zeros((pairs, 1)), 1, dev), layer.wq, layer.scales,
                        layer.biases, 4)
    for p in (0, 30679, pairs - 1):  # (30679 * n passes 2^31)
        ref, size = layer.w[0] @ f64(x)[p], np.abs(layer.w[0]) @ np.abs(f64(x)[p])
        close(y[p], ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * size + TINY[F16])


def test_logprobs_and_sums_past_32_bits(dev):
    rows, v = 18000, 120000
    x = torch.zeros(rows, v, dtype=F16, device=dev)
    x[-1] = normal(1, v).to(F16).to(dev)
    x[-2, 7] = 20.0
    tokens = torch.full((rows,), 7, dtype=torch.int32, device=dev)
    lp, h, tt, _ = q.token_logprobs(x, tokens, 3)
    for m in (0, rows - 2, rows - 1):
        ref = O.logprobs(f64(x[m]), 7, 3)
        assert abs(float(lp[m]) - ref[0]) < 1e-4 and abs(float(h[m]) - ref[1]) < 1e-3
        assert tt[m].tolist() == ref[2].tolist()
    # the same memory as rows of 15 experts' outputs
    tokens_, k = 1200, 15
    routing = routing_of(np.tile(np.arange(k), (tokens_, 1)), k, dev)
    out = q.combine_experts(x, routing)
    ref = (f64(routing.weights)[-1][:, None] * f64(x[-k:])).sum(0)
    size = (f64(routing.weights)[-1][:, None] * np.abs(f64(x[-k:]))).sum(0)
    close(out[-1], ref, U[F16] * np.abs(ref) + 16 * 2.0 ** -24 * size + TINY[F16])
