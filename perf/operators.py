"""The operators of a decoder's serving path beside its packed linears, as cases that can be timed.

Four operators: rotary positions with the append to an 8-bit key/value cache, attention over
that cache, the residual addition with the root-mean-square norm, and sampling.  ``run`` computes
them in a plain form (elementary torch operations) or, where ``own`` is true, by the calls that a
user of the framework makes.

The cache holds, per sequence, complete blocks of 64 tokens in 8 bits and the incomplete last
block (the tail) in the activation type:
  pages   uint8 [pages, kv_heads, 2, 64 * head_dim]: a key block as [64 tokens][head_dim], a value
          block transposed, as [head_dim][64 tokens]; code c stands for (c - 128) * scale
  scales  float32 [pages, kv_heads, 2], one for each block of tokens, head and key/value
  tail    activation type [slots, kv_heads, 2, 64 * head_dim], same two layouts
  table   int32 [slots, max_blocks], the page of each complete block
  lens    int32 [slots], tokens held before the call
The tokens of a call are the rows starts[b] .. starts[b + 1] of sequence b, at positions lens[b] on.
"""

import math
import random

import torch

own = False

BLOCK = 64
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # a chat's first tokens: one short sequence, one new token, where latency is all
        dict(name="attend 1x200", op="attend", batch=1, prompts=0, tokens=1, context=200,
             q_heads=32, kv_heads=8, head_dim=64, type="f16"),
        # a serving batch in the middle of its answers, every sequence of another length
        dict(name="attend 32x8192", op="attend", batch=32, prompts=0, tokens=1, context=8192,
             q_heads=32, kv_heads=8, head_dim=64, type="f16"),
        # one very long document (the last block is one token short), wide heads, eight to a group
        dict(name="attend 1x131071", op="attend", batch=1, prompts=0, tokens=1, context=131070,
             q_heads=64, kv_heads=8, head_dim=128, type="bf16"),
        # three drafted tokens of each sequence checked at once, five heads to a group
        dict(name="attend 12x3 drafts", op="attend", batch=12, prompts=12, tokens=3, context=3001,
             q_heads=40, kv_heads=8, head_dim=128, type="bf16"),
        # two prompts' next chunks on top of what the cache holds
        dict(name="attend 2x2048 chunk", op="attend", batch=2, prompts=2, tokens=2048,
             context=6001, q_heads=32, kv_heads=8, head_dim=128, type="bf16"),
        # a mixed batch: new prompts beside sequences that decode, three heads to a group
        dict(name="attend mixed 16", op="attend", batch=16, prompts=3, tokens=1100, context=4000,
             q_heads=24, kv_heads=8, head_dim=64, type="f16"),
        # one new token of each sequence of a serving batch; the first one's completes its block
        dict(name="append 32", op="append", batch=32, prompts=0, tokens=1, context=3007,
             q_heads=32, kv_heads=8, head_dim=64, type="f16", rot=64, interleaved=False),
        # prompts of ragged lengths on top of what their caches hold, half of each head rotated
        dict(name="append 4x2048", op="append", batch=4, prompts=4, tokens=2048, context=700,
             q_heads=32, kv_heads=8, head_dim=128, type="bf16", rot=64, interleaved=True),
        # one token's norm in a decode step, the residual stream kept in 32 bits
        dict(name="norm 1x2048", op="norm", rows=1, width=2048, type="f16", wide=True),
        # a prompt's norm
        dict(name="norm 8192x4096", op="norm", rows=8192, width=4096, type="bf16", wide=False),
        # one sequence's next token from 32-bit logits
        dict(name="sample 1x128256", op="sample", rows=1, vocab=128256, type="f32"),
        # a serving batch's next tokens, each row with settings of its own
        dict(name="sample 96x128256", op="sample", rows=96, vocab=128256, type="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("decode", "decode", "chunk", "mixed", "append", "norm", "sample"))
    type_ = rng.choice(("f16", "bf16"))
    if kind == "norm":
        wide = rng.random() < 0.5
        rows = _log(rng, 1, 8192)
        width = _log(rng, 64, min(16384, 8192 * 4096 * (2 if wide else 3) // 3 // rows))
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        if width == 3072:
            width += 64
        return dict(op="norm", rows=rows, width=width, type=type_, wide=wide)
    if kind == "sample":
        vocab = _log(rng, 1000, 200000)
        rows = min(_log(rng, 1, 96), 96 * 128256 // vocab)
        return dict(op="sample", rows=rows, vocab=vocab, type=rng.choice(("f32", "f16", "bf16")))
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    q_heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8))
    case = dict(op="attend", batch=1, prompts=0, tokens=1, context=1, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, type=type_)
    if kind == "decode":
        case["batch"] = _log(rng, 1, 64)
        case["prompts"] = rng.choice((0, 0, case["batch"]))
        case["tokens"] = 1 if not case["prompts"] else rng.randint(2, 6)
        case["context"] = _log(rng, 1, 131070)
    elif kind == "chunk":
        case["batch"] = case["prompts"] = _log(rng, 1, 8)
        case["tokens"] = _log(rng, 16, 2048)
        case["context"] = rng.choice((0, _log(rng, 1, 16000)))
    elif kind == "mixed":
        case["batch"] = _log(rng, 3, 32)
        case["prompts"] = rng.randint(1, case["batch"] - 1)
        case["tokens"] = _log(rng, 2, 1100)
        case["context"] = _log(rng, 1, 8000)
    else:
        case["op"] = "append"
        case["batch"] = _log(rng, 1, 64)
        case["prompts"] = rng.choice((0, case["batch"]))
        case["tokens"] = _log(rng, 1, max(1, 8192 // case["batch"])) if case["prompts"] else 1
        case["context"] = _log(rng, 1, 8000)
        case["rot"] = rng.choice((head_dim, head_dim // 2, 48))
        case["interleaved"] = rng.random() < 0.5
    most = work(listed()[2])["bytes"], work(listed()[4])["flops"]
    while work(case)["bytes"] > most[0] or work(case)["flops"] > most[1]:
        if case["op"] == "attend" and case["context"] > case["tokens"]:
            case["context"] = case["context"] * 2 // 3
        else:
            case["tokens"] = case["tokens"] * 2 // 3
    return case


def _lengths(case):
    """(tokens held, new tokens) of every sequence: from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    held, new = [], []
    for b in range(case["batch"]):
        first = b == 0  # the first sequence has the full lengths
        prompt = b < case["prompts"]
        n = case["tokens"] if prompt else 1
        n = n if first or not prompt or n < 16 else rng.randint(n // 2, n)
        c = case["context"]
        c = c if first else rng.randint(c // 4, c)
        if prompt and 0 < case["prompts"] < case["batch"]:
            c = 0  # in a mixed batch the prompts are new
        held.append(c)
        new.append(n)
    return held, new


def work(case):
    """The bytes and operations that one pass cannot do without."""
    op = case["op"]
    if op == "norm":
        n, es = case["rows"] * case["width"], 4 if case["wide"] else 2
        return {"bytes": n * (2 + 2 + 2 * es) + 2 * case["width"], "flops": 6 * n}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["type"] == "f32" else 2) + 28 * case["rows"],
                "flops": 5 * n}
    held, new = _lengths(case)
    kvh, qh, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    bytes_, flops = 0, 0
    for h, n in zip(held, new):
        total = h + n
        if op == "attend":
            blocks = total // BLOCK
            bytes_ += blocks * kvh * (2 * BLOCK * d + 8) + (total % BLOCK) * kvh * 2 * d * 2
            bytes_ += 2 * n * qh * d * 2 + 4 * blocks
            flops += 4 * d * qh * (n * h + n * (n + 1) // 2)
        else:
            done = total // BLOCK - h // BLOCK
            bytes_ += n * (qh + 2 * kvh) * d * 2 + n * qh * d * 2 + n * case["rot"] * 4
            # blocks that this call completes: the old tail is read, codes are written, and read
            # again with the values returned; the rest goes to the tail
            old = h % BLOCK if done else 0
            rest = total % BLOCK if done else n
            bytes_ += kvh * 2 * d * (2 * old + done * BLOCK * (1 + 1 + 2) + 2 * rest)
            flops += n * (qh + kvh) * case["rot"] * 3 + done * BLOCK * kvh * 2 * d * 3
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------- preparation

def _quantised(x):
    """Whole blocks [.., n] in 8 bits: (codes, scale of each block)."""
    scale = x.abs().amax(-1) / 127
    codes = torch.where(scale[..., None] > 0, (x / scale[..., None]).round(), 0)
    return (codes + 128).to(torch.uint8), scale


def _table(n, rot, base, dev):
    """(cos, sin) of every position and pair, from angles in 64 bits."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case)
    if case["op"] == "norm":
        dt = TYPES[case["type"]]
        s["x"] = normal(case["rows"], case["width"]).to(dt)
        wide = torch.float32 if case["wide"] else dt
        res = 3 * normal(case["rows"], case["width"])
        res[:, : max(1, case["width"] // 256)] *= 20  # the residual stream's few large features
        s["residual"] = res.to(wide)
        s["weight"] = (1 + 0.2 * normal(case["width"])).to(dt)
        return s
    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = 2.5 * normal(rows, vocab)
        x[:, :: 997] += 6 * torch.rand(rows, 1, generator=gen, device=dev)  # likely tokens
        x[:, 5 :: 1009] = -math.inf  # tokens that are not allowed
        s["logits"] = x.to({"f32": torch.float32, **TYPES}[case["type"]])
        s["u"] = torch.rand(rows, generator=gen, device=dev)
        kind = (torch.arange(rows, device=dev) + 1) % 6
        pick = torch.tensor  # by kind: top-k and top-p, top-p, all three, min-p, nothing, greedy
        s["temperature"] = pick([1.0, 0.8, 0.7, 1.2, 1.0, 0.0], device=dev)[kind]
        s["top_k"] = pick([0, 50, 0, 200, 0, 0], device=dev, dtype=torch.int32)[kind]
        s["top_p"] = pick([0.95, 0.9, 0.8, 0.99, 1.0, 1.0], device=dev)[kind]
        s["min_p"] = pick([0.0, 0.0, 0.0, 0.02, 0.05, 0.0], device=dev)[kind]
        return s

    dt, d, kvh, qh = TYPES[case["type"]], case["head_dim"], case["kv_heads"], case["q_heads"]
    held, new = _lengths(case)
    batch, attend = case["batch"], case["op"] == "attend"
    total = [h + n for h, n in zip(held, new)]
    # what is in the cache: for attention all tokens, for the append those held before it
    blocks = [t // BLOCK for t in total]
    s["lens"] = torch.tensor(held, dtype=torch.int32, device=dev)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["most"] = max(new)
    wide = max(max(blocks), 1)
    # pages in no order; for the append only the blocks that the call completes have their own
    first = [0 if attend else h // BLOCK for h in held]
    pages = sum(b - f for b, f in zip(blocks, first)) + 1
    place = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((batch, wide), place[-1], dtype=torch.int32)
    at = 0
    for b in range(batch):
        n = blocks[b] - first[b]
        table[b, first[b] : blocks[b]] = torch.tensor(place[at : at + n], dtype=torch.int32)
        at += n
    s["table"] = table.to(dev)
    s["pages"] = torch.full((pages, kvh, 2, BLOCK * d), 128, dtype=torch.uint8, device=dev)
    s["scales"] = torch.zeros(pages, kvh, 2, device=dev)
    if attend:
        spread = torch.ones(d, device=dev)
        spread[:: 16] = 3  # channels of keys that stand out
        for p in range(0, pages, 4096):
            n = min(4096, pages - p)
            kv = normal(n, kvh, 2, BLOCK * d)
            kv[:, :, 0] *= spread.repeat(BLOCK)
            s["pages"][p : p + n], s["scales"][p : p + n] = _quantised(kv)
    s["tail"] = normal(batch, kvh, 2, BLOCK * d).to(dt)
    rows = starts[-1]
    if attend:
        s["q"] = normal(rows, qh, d).mul_(1.2).to(dt)
        # where each row goes among sequences padded to the longest
        s["longest"] = max(total)
    else:
        s["qkv"] = normal(rows, (qh + 2 * kvh) * d).to(dt)
        s["rope"] = _table(max(total) + 1, case["rot"], 500000.0, dev)
        # the blocks that the call touches, the complete ones first
        touched = [(b, j) for b in range(batch)
                   for j in range(held[b] // BLOCK, (total[b] - 1) // BLOCK + 1)]
        touched.sort(key=lambda t: (t[1] + 1) * BLOCK > total[t[0]])
        s["done"] = sum((j + 1) * BLOCK <= total[b] for b, j in touched)
        number = {t: i for i, t in enumerate(touched)}
        s["touched_seq"] = torch.tensor([b for b, _ in touched], device=dev)
        s["touched_end"] = torch.tensor([total[b] - j * BLOCK for b, j in touched], device=dev)
        s["row_block"] = torch.tensor([number[b, (held[b] + i) // BLOCK] for b in range(batch)
                                       for i in range(new[b])], device=dev)
        s["filled"] = torch.tensor([table[b, j].item() for b, j in touched[: s["done"]]],
                                   dtype=torch.int32, device=dev)
    s["row_seq"] = torch.repeat_interleave(torch.arange(batch), torch.tensor(new)).to(dev)
    if own:
        import int8_qmv_qmm_gb300 as q

        # the handle of the cache that a serving program keeps
        s["cache"] = q.KVCache(s["pages"], s["scales"], s["tail"], s["table"], s["lens"])
        s["workspace"] = q.attention_workspace(d, dev)
    return s


# ---------------------------------------------------------------------- the plain forms

def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h / (h.square().mean(-1, keepdim=True) + 1e-5).sqrt() * s["weight"].float()
    return {"out": y.to(s["x"].dtype), "residual": h.to(s["residual"].dtype)}


def _plain_sample(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    x = torch.where(x.isnan(), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    tau = s["temperature"][:, None]
    index = torch.arange(vocab, device=x.device)
    best = torch.where(x == top, index, vocab).amin(-1, keepdim=True)
    e = torch.where(x == top, 1.0, ((x - top) / tau).exp())
    e = torch.where(tau > 0, e, (index == best).float())
    # weights are whole numbers of 2^-36, so that their sums are exact in any order
    w = (e * 2.0 ** 36).round().long()
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    ws, es = w.gather(-1, order), e.gather(-1, order)
    k = s["top_k"][:, None]
    keep = (index < k) | (k <= 0)
    mass = (ws * keep).sum(-1, keepdim=True)
    before = ws.cumsum(-1) - ws
    p = s["top_p"][:, None].double()
    keep &= (before.double() < p * mass.double()) | (p >= 1)
    keep &= es >= s["min_p"][:, None]
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(-1, order, ws * keep)
    cum = kept.cumsum(-1)
    all_ = cum[:, -1:]
    t = (s["u"][:, None].double() * all_.double()).floor().long()
    t = torch.minimum(t, all_ - 1)
    token = torch.searchsorted(cum, t, right=True).clamp(max=vocab - 1)
    prob = kept.gather(-1, token).double() / all_.double()
    none = top == -math.inf  # no token is allowed
    token = torch.where(none, -1, token).int()
    prob = torch.where(none, 0.0, prob).float()
    return {"token": token[:, 0], "prob": prob[:, 0]}


def _plain_rotate(x, cs, interleaved):
    """x [T, heads, D] with its first pairs turned by cs [T, pairs, 2]."""
    half = cs.shape[1]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    turned, rest = x[..., : 2 * half], x[..., 2 * half :]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        new = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        new = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((new, rest), -1)


def _plain_append(s):
    c = s["case"]
    qh, kvh, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    dt = s["qkv"].dtype
    rows = s["qkv"].shape[0]
    seq = s["row_seq"]
    pos = s["lens"][seq] + torch.arange(rows, device=seq.device) - s["starts"][seq]
    x = s["qkv"].float().view(rows, qh + 2 * kvh, d)
    turned = _plain_rotate(x[:, : qh + kvh], s["rope"][pos], c["interleaved"]).to(dt)
    k, v = turned[:, qh:], x[:, qh + kvh :].to(dt)
    # every touched block as it will be: the tail's tokens, then the new ones
    n = s["touched_seq"].shape[0]
    tail = s["tail"]
    kb = tail[s["touched_seq"], :, 0].view(n, kvh, BLOCK, d)
    vb = tail[s["touched_seq"], :, 1].view(n, kvh, d, BLOCK)
    at, row = pos % BLOCK, s["row_block"]
    kb[row, :, at] = k
    vb[row, :, :, at] = v
    kv = torch.stack((kb.flatten(-2), vb.flatten(-2)), 2)
    done = s["done"]
    codes, scale = _quantised(kv[:done].float())
    s["pages"][s["filled"]], s["scales"][s["filled"]] = codes, scale
    # the incomplete blocks become the tails, up to their last token
    held = torch.arange(BLOCK, device=seq.device) < s["touched_end"][done:, None]
    held = torch.stack((held[:, :, None].expand(-1, -1, d).flatten(1),
                        held[:, None, :].expand(-1, d, -1).flatten(1)), 1)[:, None]
    left = s["touched_seq"][done:]
    tail[left] = torch.where(held, kv[done:], tail[left])
    values = (s["pages"][s["filled"]].float() - 128) * s["scales"][s["filled"]][..., None]
    return {"q": turned[:, :qh], "values": values.to(dt), "scales": s["scales"], "tail": tail}


def _plain_attend(s):
    c = s["case"]
    qh, kvh, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    batch, group = c["batch"], qh // kvh
    lens, starts, table = s["lens"].long(), s["starts"].long(), s["table"].long()
    total = lens + starts[1:] - starts[:-1]
    blocks = s["longest"] // BLOCK + 1
    table = table[:, : blocks - 1]
    kv = (s["pages"][table].float() - 128) * s["scales"][table][..., None]
    kv = torch.cat((kv, kv.new_zeros(batch, blocks - kv.shape[1], kvh, 2, BLOCK * d)), 1)
    every = torch.arange(batch, device=kv.device)
    kv[every, total // BLOCK] = s["tail"].float()
    k = kv[:, :, :, 0].view(batch, blocks, kvh, BLOCK, d).transpose(1, 2)
    v = kv[:, :, :, 1].view(batch, blocks, kvh, d, BLOCK).permute(0, 2, 1, 4, 3)
    k, v = (t.reshape(batch, kvh, blocks * BLOCK, d) for t in (k, v))
    place = torch.arange(blocks * BLOCK, device=kv.device)
    v = torch.where((place < total[:, None])[:, None, :, None], v, 0)
    # the rows of every sequence, padded to the longest
    step = torch.arange(s["most"], device=kv.device)
    row = (starts[:-1, None] + step).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(batch, -1, kvh, group, d).transpose(1, 2)
    score = torch.matmul(q.reshape(batch, kvh, -1, d), k.transpose(-1, -2)) / math.sqrt(d)
    seen = (place <= (lens[:, None] + step)[..., None])[:, None, :, None]
    score = score.view(batch, kvh, s["most"], group, -1).masked_fill_(~seen, -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp()
    p = (p / p.sum(-1, keepdim=True)).view(batch, kvh, -1, blocks * BLOCK)
    out = torch.matmul(p, v).view(batch, kvh, s["most"], group, d).transpose(1, 2)
    seq = s["row_seq"]
    at = torch.arange(seq.shape[0], device=seq.device) - starts[seq]
    return out[seq, at].reshape(-1, qh, d).to(s["q"].dtype)


# ------------------------------------------------------------------- the framework's calls

def _own(s):
    import int8_qmv_qmm_gb300 as q

    c = s["case"]
    if c["op"] == "norm":
        out, residual = q.add_rms_norm(s["x"], s["weight"], s["residual"], eps=1e-5)
        return {"out": out, "residual": residual}
    if c["op"] == "sample":
        token, prob = q.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"],
                               s["min_p"])
        return {"token": token, "prob": prob}
    if c["op"] == "append":
        out = q.rope_append(s["qkv"], s["rope"], s["cache"], s["starts"], c["q_heads"],
                            interleaved=c["interleaved"])
        return {"q": out, "values": q.cache_dequant(s["cache"], s["filled"]),
                "scales": s["scales"], "tail": s["tail"]}
    return q.cache_attention(s["q"], s["cache"], s["starts"], s["most"],
                             workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "sample": _plain_sample, "append": _plain_append,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "sample": _exact_sample, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](s)


def _exact_norm(s):
    h = s["x"].double() + s["residual"].double()
    rms = torch.sqrt(torch.einsum("rk,rk->r", h, h) / h.shape[1] + 1e-5)
    return {"out": torch.einsum("rk,k,r->rk", h, s["weight"].double(), 1 / rms), "residual": h}


def _exact_sample(s):
    """The probability of each row's token, row by row; the token itself is a whole number."""
    probs = []
    for r in range(s["logits"].shape[0]):
        x = s["logits"][r].double()
        tau, k = s["temperature"][r].item(), s["top_k"][r].item()
        if tau <= 0:
            probs.append(1.0)
            continue
        p = torch.softmax(x / tau, 0)
        order = torch.argsort(x, descending=True, stable=True)
        kept = order[: k] if k > 0 else order
        if s["top_p"][r].item() < 1:
            share = p[kept] / p[kept].sum()
            kept = kept[share.cumsum(0) - share < s["top_p"][r].double()]
        kept = kept[p[kept] >= s["min_p"][r].double() * p.max()]
        kept = kept.sort()[0]
        share = p[kept] / p[kept].sum()
        at = (share.cumsum(0) <= s["u"][r].double()).sum().clamp(max=kept.numel() - 1)
        probs.append(share[at].item())
    return {"token": None, "prob": torch.tensor(probs, dtype=torch.float64)}


def _exact_append(s):
    c = s["case"]
    qh, kvh, d, half = c["q_heads"], c["kv_heads"], c["head_dim"], c["rot"] // 2
    dt, lens, starts = s["qkv"].dtype, s["lens"].tolist(), s["starts"].tolist()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else (
        slice(0, half), slice(half, 2 * half))
    q, scales, tail = [], s["scales"].double(), s["tail"].double()
    values = torch.zeros(s["done"], kvh, 2, BLOCK * d, dtype=torch.float64, device=tail.device)
    page_at = {p: i for i, p in enumerate(s["filled"].tolist())}
    for b in range(c["batch"]):
        x = s["qkv"][starts[b] : starts[b + 1]].double().view(-1, qh + 2 * kvh, d)
        z = torch.complex(*s["rope"][lens[b] : lens[b] + x.shape[0]].double().unbind(-1))
        z = torch.complex(x[..., first], x[..., second])[:, : qh + kvh] * z[:, None]
        x[:, : qh + kvh, first], x[:, : qh + kvh, second] = z.real, z.imag
        q.append(x[:, :qh])
        kv = x[:, qh:].to(dt).double()  # the cache is fed from values of the activation type
        kv = kv.view(-1, 2, kvh, d).transpose(1, 2)  # [T, kv_heads, 2, D]
        at = lens[b] % BLOCK
        old = torch.stack((tail[b, :, 0].view(kvh, BLOCK, d).transpose(0, 1)[:at],
                           tail[b, :, 1].view(kvh, d, BLOCK).permute(2, 0, 1)[:at]), 2)
        kv = torch.cat((old, kv))
        for j, block in enumerate(kv.split(BLOCK)):
            keys, vals = block[:, :, 0].transpose(0, 1), block[:, :, 1].permute(1, 2, 0)
            if block.shape[0] < BLOCK:
                tail[b, :, 0].view(kvh, BLOCK, d)[:, : block.shape[0]] = keys
                tail[b, :, 1].view(kvh, d, BLOCK)[:, :, : block.shape[0]] = vals
                continue
            page = s["table"][b, lens[b] // BLOCK + j].item()
            for h, flat in enumerate((keys.flatten(1), vals.flatten(1))):
                top = flat.abs().amax(1)
                scales[page, :, h] = top / 127
                codes = (flat * (127 / top)[:, None]).round()
                values[page_at[page], :, h] = codes * (top / 127)[:, None]
    return {"q": torch.cat(q), "values": values, "scales": scales, "tail": tail}


def _exact_attend(s):
    c = s["case"]
    qh, kvh, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.zeros(starts[-1], qh, d, dtype=torch.float64, device=s["q"].device)
    for b in range(c["batch"]):
        n = starts[b + 1] - starts[b]
        total = lens[b] + n
        page = s["table"][b, : total // BLOCK].long()
        left = total % BLOCK
        mask = torch.ones(n, total, dtype=torch.bool, device=out.device).tril(lens[b])
        for h in range(kvh):
            codes = s["pages"][page, h].double() - 128
            kv = codes * s["scales"][page, h].double()[..., None]
            keys = kv[:, 0].reshape(-1, d)
            vals = kv[:, 1].view(-1, d, BLOCK).transpose(1, 2).reshape(-1, d)
            tail = s["tail"][b, h].double()
            keys = torch.cat((keys, tail[0].view(BLOCK, d)[:left]))
            vals = torch.cat((vals, tail[1].view(d, BLOCK).t()[:left]))
            for g in range(h * (qh // kvh), (h + 1) * (qh // kvh)):
                score = s["q"][starts[b] : starts[b + 1], g].double() @ keys.t() / d ** 0.5
                p = torch.softmax(score.masked_fill(~mask, -math.inf), -1)
                out[starts[b] : starts[b + 1], g] = p @ vals
    return out
