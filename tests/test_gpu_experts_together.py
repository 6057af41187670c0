"""Routing, the experts' products and their sum as a layer runs them, and decoders with
experts, normed heads and log probabilities."""

import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300.decoder import Decoder
from oracle import experts_oracle as O
from tests.test_gpu_decode_loop import SHAPE, distance, dev, prompts  # noqa: F401
from tests.test_gpu_decoder import U, f64, normal
from tests.test_gpu_experts import BF16, F16, F32, Layer

pytestmark = pytest.mark.gpu


class Block:
    """A layer's mixture: router, gate and up, down, with the float64 weights."""

    def __init__(self, dev, experts, hidden, ffn, top_k, bits, dt):
        self.top_k, self.ffn, self.bits, self.dt = top_k, ffn, bits, dt
        self.router = normal(5, experts, hidden).to(dt).to(dev) / hidden ** 0.5
        self.up = Layer(dev, experts, 2 * ffn, hidden, bits, dt, seed=1)
        self.down = Layer(dev, experts, hidden, ffn, bits, dt, seed=2)

    def run(self, x, logits=None, shared=None, overlap=False):
        logits = (x @ self.router.T).float() if logits is None else logits
        r = q.route_experts(logits, self.top_k, overlap_previous=overlap)
        g = q.expert_linear(x, r, self.up.wq, self.up.scales, self.up.biases, self.bits,
                            overlap_previous=overlap)
        a = F.silu(g[:, : self.ffn]) * g[:, self.ffn:]
        y = q.expert_linear(a, r, self.down.wq, self.down.scales, self.down.biases, self.bits,
                            overlap_previous=overlap)
        return q.combine_experts(y, r, add=shared, overlap_previous=overlap), r


@pytest.mark.parametrize("tokens", [1, 5, 33, 300])
@pytest.mark.parametrize("bits,dt", [(4, F16), (8, BF16)])
def test_layer_against_plain_model(dev, tokens, bits, dt):  # noqa: F811
    b = Block(dev, 8, 256, 128, 3, bits, dt)
    x = normal(tokens, tokens, 256).to(dt).to(dev)
    shared = normal(7, tokens, 256).to(dt).to(dev)
    out, r = b.run(x, shared=shared)
    experts, weights, xs = r.experts.cpu().numpy(), f64(r.weights), f64(x)
    ref = f64(shared).copy()
    for t in range(tokens):
        for e, w in zip(experts[t], weights[t]):
            g = b.up.w[e] @ xs[t]
            gate, up = g[:128], g[128:]
            ref[t] += w * (b.down.w[e] @ (gate / (1 + np.exp(-gate)) * up))
    # Roundings to dt: gate and up, the activation and its product, the second products, the
    # result: each moves a token's output by about u of its size (the weights' own, 2^-11,
    # beside them).  Six of them one-sided are 6 u; counted twice.
    u = U[dt] + 2.0 ** -11
    err = np.linalg.norm(f64(out) - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert err.max() <= 12 * u, err.max()
    assert q.device_status() == 0


def test_layer_on_another_stream_and_overlapped(dev):  # noqa: F811
    """The same bits on a side stream, and with every call started while its predecessor
    ends; workspaces and plans of calls in flight at once are their own."""
    for tokens in (3, 40, 700):
        b = Block(dev, 16, 128, 64, 4, 8, F16)
        xs = [normal(s, tokens, 128).to(F16).to(dev) for s in range(4)]
        logits = [(x @ b.router.T).float() for x in xs]
        ref = [b.run(x, z)[0] for x, z in zip(xs, logits)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in xs]
        got = []
        for s, x, z in zip(streams, xs, logits):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append([b.run(x, z, overlap=True)[0] for _ in range(5)])
        torch.cuda.synchronize()
        for g, r in zip(got, ref):
            assert all(torch.equal(o, r) for o in g)
    assert q.device_status() == 0


@pytest.mark.parametrize("tokens", [2, 500])
def test_two_captured_layers(dev, tokens):  # noqa: F811
    """Two graphs of one layer, replayed in turn on new inputs and at once on two streams."""
    b = Block(dev, 16, 128, 64, 4, 4, BF16)
    x = [torch.zeros(tokens, 128, dtype=BF16, device=dev) for _ in range(2)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.run(x[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.run(x[i], overlap=True)[0])
        graphs.append(g)
    for seed in range(3):
        new = [normal(10 * seed + i, tokens, 128).to(BF16).to(dev) for i in range(2)]
        ref = [b.run(n)[0] for n in new]
        for i in range(2):
            x[i].copy_(new[i])
        if seed < 2:
            for i in (seed, 1 - seed):
                graphs[i].replay()
        else:
            s = [torch.cuda.Stream() for _ in graphs]
            torch.cuda.synchronize()
            for _ in range(3):
                for i in range(2):
                    with torch.cuda.stream(s[i]):
                        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    assert q.device_status() == 0


def test_padded_batch(dev):  # noqa: F811
    """Rows of a batch that are padding get no expert by logits of -infinity: what stands in
    them reaches nobody, and their sum is what is added."""
    b = Block(dev, 8, 128, 64, 2, 8, F16)
    x = normal(1, 50, 128).to(F16).to(dev)
    logits = (x @ b.router.T).float()
    ref, _ = b.run(x[:30], logits[:30])
    x[30:] = math.nan
    logits[30:] = -math.inf
    shared = torch.zeros_like(x)
    shared[30:] = 5.0
    out, r = b.run(x, logits, shared=shared)
    assert torch.equal(out[:30], ref) and (out[30:] == 5).all()
    assert (r.experts[30:] == -1).all() and int(r.offsets[-1]) == 60
    assert q.device_status() == 0


# -------------------------------------------------------------------- decoders
MIXED = dict(SHAPE, experts=4, top_experts=4, ffn=128, qk_norm=True, logprobs=5)


def plain_logits(d, tokens):
    """Logits after the last of `tokens`, everything in float64 and nothing cached.  (All
    experts take part, so that no choice is near a border.)"""
    def weight(w):
        return q.dequant(*w, d.bits, out_dtype=torch.float32).double().cpu()

    def norm(h, eps=1e-5):
        return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)

    def turn(x):
        half = x.shape[-1] // 2
        angle = (torch.arange(len(tokens), dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half))
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    heads, kv, dim, t = d.q_heads, MIXED["kv_heads"], MIXED["head_dim"], len(tokens)
    r = d.embed.double().cpu()[torch.tensor(tokens)]
    for layer in d.layers:
        qkv = (norm(r) @ weight(layer["qkv"]).T).view(t, heads + 2 * kv, dim)
        query, k = (turn(norm(x, 1e-6)) for x in (qkv[:, :heads], qkv[:, heads:heads + kv]))
        k, v = (x.repeat_interleave(heads // kv, 1) for x in (k, qkv[:, heads + kv:]))
        score = torch.einsum("thd,shd->hts", query, k) / math.sqrt(dim)
        score += torch.full((t, t), -math.inf, dtype=torch.float64).triu(1)
        r = r + torch.einsum("hts,shd->thd", score.softmax(-1), v).reshape(t, -1) @ weight(
            layer["o"]).T
        h = norm(r)
        share = (h @ weight(layer["router"]).T).softmax(-1)
        for e in range(MIXED["experts"]):
            gate, up = (h @ weight([w[e] for w in layer["gate_up"]]).T).chunk(2, -1)
            down = weight([w[e] for w in layer["down"]])
            r = r + share[:, e:e + 1] * ((gate * torch.sigmoid(gate) * up) @ down.T)
    return norm(r[-1]) @ weight(d.lm_head).T


@pytest.mark.parametrize("bits,dt", [(8, F16), (4, BF16)])
def test_decoder_with_experts_against_plain_model(dev, bits, dt):  # noqa: F811
    """The bound is the one that a decoder without experts has: the cache's 8 bits set it (in
    bfloat16 its roundings, 2^-8 each and about ten a layer, add another 2 * 10 * 2^-9)."""
    d = Decoder(dev, **MIXED, bits=bits, dtype=dt)
    ids = prompts((1, 63, 130))
    d.prefill(ids)
    bound = 0.05 if dt is F16 else 0.09
    for s in range(3):
        assert distance(d.logits[s], plain_logits(d, ids[s])) < bound, s
    for _ in range(2):
        ids = [p + [t] for p, t in zip(ids, d.tokens.tolist())]
        d.decode()
    for s in range(3):
        assert distance(d.logits[s], plain_logits(d, ids[s])) < bound, (s, "decode")
    assert q.device_status() == 0


def test_decoder_with_experts_captured_equals_eager(dev):  # noqa: F811
    """Bit for bit, log probabilities among it, with few of many experts."""
    seen = []
    for captured in (False, True):
        d = Decoder(dev, **{**MIXED, "experts": 16, "top_experts": 2})
        d.temperature.fill_(0.8)
        torch.manual_seed(11)
        d.prefill(prompts((63, 5, 120)))
        first = d.logprobs.clone()
        if captured:
            d.capture()
            assert torch.equal(d.logprobs, first)
        torch.manual_seed(12)
        rows = []
        for _ in range(8):
            tokens = d.decode()
            rows.append([t.clone() for t in (tokens, d.logits, d.logprobs, d.entropy,
                                             d.top_tokens, d.top_logprobs)])
            ref = [O.logprobs(f64(d.logits)[s], int(tokens[s]), 5) for s in range(3)]
            assert np.allclose(f64(d.logprobs), [r[0] for r in ref], atol=2.0 ** -16)
            assert np.allclose(f64(d.entropy), [r[1] for r in ref], atol=2.0 ** -15)
            assert np.array_equal(d.top_tokens.cpu().numpy(), [r[2] for r in ref])
        seen.append(rows)
    for a, b in zip(*seen):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert q.device_status() == 0
