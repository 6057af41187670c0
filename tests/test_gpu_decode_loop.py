"""A whole decoder over the library's calls: against a plain float64 model of the
same (reconstructed) weights, and the captured decode step against the eager one."""

import math

import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300.decoder import Decoder

pytestmark = pytest.mark.gpu

SHAPE = dict(slots=3, max_tokens=512, layers=2, hidden=256, q_heads=4, kv_heads=2, head_dim=64,
             ffn=512, vocab=1000)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_qmv_qmm_gb300 import build_lib
    build_lib.build()
    q.lib()
    return torch.device("cuda:0")


def prompts(lengths, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, SHAPE["vocab"], (n,), generator=g).tolist() for n in lengths]


def plain_logits(d, tokens):
    """Logits after the last of `tokens`, everything in float64 and nothing cached."""
    def weight(w):
        return q.dequant(*w, d.bits, out_dtype=torch.float32).double().cpu()

    def norm(h):
        return h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5)

    def turn(x):  # [T, heads, D], the pairs i and i + D/2
        half = x.shape[-1] // 2
        angle = (torch.arange(len(tokens), dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half))
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    heads, kv, dim = d.q_heads, SHAPE["kv_heads"], SHAPE["head_dim"]
    t = len(tokens)
    r = d.embed.double().cpu()[torch.tensor(tokens)]
    for layer in d.layers:
        qkv = (norm(r) @ weight(layer["qkv"]).T).view(t, heads + 2 * kv, dim)
        query, k, v = turn(qkv[:, :heads]), turn(qkv[:, heads:heads + kv]), qkv[:, heads + kv:]
        k, v = (x.repeat_interleave(heads // kv, 1) for x in (k, v))
        score = torch.einsum("thd,shd->hts", query, k) / math.sqrt(dim)
        score += torch.full((t, t), -math.inf, dtype=torch.float64).triu(1)
        a = torch.einsum("hts,shd->thd", score.softmax(-1), v)
        r = r + a.reshape(t, -1) @ weight(layer["o"]).T
        gate, up = (norm(r) @ weight(layer["gate_up"]).T).chunk(2, -1)
        r = r + (gate * torch.sigmoid(gate) * up) @ weight(layer["down"]).T
    return norm(r[-1]) @ weight(d.lm_head).T


def distance(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


# A code is off by at most half a step of amax/127; over 64 x 64 normal elements amax
# is near 4 sigma, so keys and values carry an error of about 4/127/sqrt(12) = 0.9% of
# their size, and what a layer adds to the residual stream little more.  Roundings to
# f16 (2^-11 each) stay well below that.  Two layers add up to less than 3%: 5% is the
# bound, where a wrong position, head or slot gives a distance of order one.
BOUND = 0.05


@pytest.mark.parametrize("lengths", [(1, 63, 64), (200, 3, 130), (65, 129, 1)])
def test_logits_against_plain_model(dev, lengths):
    d = Decoder(dev, **SHAPE)
    ids = prompts(lengths)
    d.prefill(ids)
    for s in range(3):
        assert distance(d.logits[s], plain_logits(d, ids[s])) < BOUND, (s, "prefill")
    for _ in range(3):  # decode steps, from the cache
        ids = [p + [t] for p, t in zip(ids, d.tokens.tolist())]
        d.decode()
    for s in range(3):
        assert distance(d.logits[s], plain_logits(d, ids[s])) < BOUND, (s, "decode")
    assert d.lens.tolist() == [n + 3 for n in lengths] == d.held
    assert q.device_status() == 0


def test_prompt_in_pieces(dev):
    """A prompt that comes in three calls, beside slots that get nothing."""
    d = Decoder(dev, **SHAPE)
    ids = prompts((180, 40, 0))
    d.prefill([ids[0][:70], [], []])
    d.prefill([ids[0][70:71], ids[1], []])
    kept = d.tokens[1].item()
    d.prefill([ids[0][71:], [], []])
    assert d.tokens[1].item() == kept and d.lens.tolist() == [180, 40, 0]
    assert distance(d.logits[0], plain_logits(d, ids[0])) < BOUND
    assert q.device_status() == 0


@pytest.mark.parametrize("greedy", [True, False])
def test_captured_step_equals_eager(dev, greedy):
    """Over the ends of blocks, bit for bit."""
    seen = []
    for captured in (False, True):
        d = Decoder(dev, **SHAPE)
        if not greedy:
            d.temperature.fill_(0.9)
            d.top_k.fill_(50)
            d.top_p.fill_(0.9)
            d.min_p.fill_(0.01)
        torch.manual_seed(11)
        d.prefill(prompts((63, 5, 120)))
        if captured:
            d.capture()
        torch.manual_seed(12)
        seen.append([(d.decode().clone(), d.logits.clone()) for _ in range(12)])
    for (t0, l0), (t1, l1) in zip(*seen):
        assert torch.equal(t0, t1) and torch.equal(l0, l1)
    assert q.device_status() == 0


def test_no_room(dev):
    d = Decoder(dev, **{**SHAPE, "max_tokens": 70})
    with pytest.raises(ValueError, match="max_tokens"):
        d.prefill(prompts((71, 1, 1)))
    d.prefill(prompts((70, 1, 1)))
    with pytest.raises(ValueError, match="slot 0"):
        d.decode()
    with pytest.raises(ValueError, match="each slot"):
        d.prefill([[1]])
    with pytest.raises(ValueError, match="vocabulary"):
        d.prefill([[], [SHAPE["vocab"]], []])
    assert d.held == [70, 1, 1]
