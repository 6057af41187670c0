"""The operators of a mixture-of-experts decoder with packed weights, as cases that can be timed.

Five operators: routing tokens to experts (with the plan that groups their rows), the experts'
products from packed 4- or 8-bit weights, the weighted sum of each token's experts, rotary positions
with norms of queries and keys for each head and the append to an 8-bit key/value cache, and log
probabilities of given tokens with entropy and top alternatives.  ``run`` computes them in a plain
form (elementary torch operations) or, where ``own`` is true, by the calls that a user of the
framework makes.

Routing: token t's j-th expert is pair p = t * top_k + j.  experts int32 and weights float32
[tokens, top_k]; order int32 [pairs], the pairs sorted by expert (those of one expert in their own
order, pairs without an expert, -1, at the end); offsets int32 [experts + 1], where each expert's
pairs start in it.

Packed weights of all experts: uint32 [experts, N, K * bits / 32], codes low bits first, one scale
and bias for each group of 64 along K; a weight is code * scale + bias.

The cache: complete blocks of 64 tokens in 8 bits (pages, float32 scales), the incomplete last block
of each sequence (tail) in the activation type; values are held transposed.
"""

import math
import random

import torch

own = False

BLOCK = 64
GROUP = 64
EPS = 1e-6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's experts, where latency is all
        dict(name="route 1x64", op="route", rows=1, experts=64, top_k=8, type="f32",
             scoring="softmax", bias=False, groups=1, top_groups=1, group_score="max",
             renormalise=True, scale=1.0),
        # a long prompt's routing among many experts: groups first, a bias that balances the load
        dict(name="route 8192x256", op="route", rows=8192, experts=256, top_k=8, type="f32",
             scoring="sigmoid", bias=True, groups=8, top_groups=4, group_score="top2",
             renormalise=True, scale=2.5),
        # one decoded token's first products (gate and up as one matrix)
        dict(name="experts 1 up", op="experts", rows=1, experts=64, top_k=8, width=2048,
             features=2048, bits=4, type="f16", per_pair=False),
        # a serving batch's second products, about four rows an expert
        dict(name="experts 32 down", op="experts", rows=32, experts=64, top_k=8, width=1024,
             features=2048, bits=8, type="bf16", per_pair=True),
        # a short chunk with ragged numbers of rows and odd sizes
        dict(name="experts 500 odd", op="experts", rows=500, experts=60, top_k=6, width=1408,
             features=2501, bits=8, type="f16", per_pair=False),
        # a prompt's first products
        dict(name="experts 4096 up", op="experts", rows=4096, experts=64, top_k=8, width=2048,
             features=2048, bits=4, type="f16", per_pair=False),
        # a serving batch's sums
        dict(name="combine 32x8", op="combine", rows=32, top_k=8, width=2048, type="f16",
             add=False),
        # a prompt's sums, on top of what an expert that every token uses has given
        dict(name="combine 4096x8", op="combine", rows=4096, top_k=8, width=2048, type="bf16",
             add=True),
        # one new token of each sequence of a serving batch; the first one's completes its block
        dict(name="append 32", op="append", batch=32, prompts=0, tokens=1, context=3007,
             q_heads=32, kv_heads=4, head_dim=128, type="bf16", rot=128, interleaved=False),
        # prompts of ragged lengths on top of what their caches hold, half of each head rotated
        dict(name="append 4x2048", op="append", batch=4, prompts=4, tokens=2048, context=700,
             q_heads=24, kv_heads=8, head_dim=64, type="f16", rot=32, interleaved=True),
        # one sequence's next token, answered with its alternatives
        dict(name="score 1x128256", op="score", rows=1, vocab=128256, top=20, type="f32"),
        # a prompt's tokens scored
        dict(name="score 2048x128256", op="score", rows=2048, vocab=128256, top=5, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("route", "experts", "experts", "experts", "combine", "append", "score"))
    type_ = rng.choice(("f16", "bf16"))
    if kind == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.randint(max(1, 4 // groups), 320 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op="route", rows=_log(rng, 1, 8192), experts=experts,
                    top_k=rng.randint(1, min(8, experts // groups * top_groups)),
                    type=rng.choice(("f32", "f16", "bf16")),
                    scoring=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5,
                    groups=groups, top_groups=top_groups,
                    group_score=rng.choice(("max", "top2")), renormalise=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5)))
    if kind == "experts":
        experts = rng.choice((8, 16, 32, 60, 64, 128))
        case = dict(op="experts", rows=_log(rng, 1, 4096), experts=experts,
                    top_k=rng.randint(1, 8), width=64 * _log(rng, 2, 64),
                    features=_log(rng, 64, 4096), bits=rng.choice((4, 8)), type=type_,
                    per_pair=rng.random() < 0.5)
        if rng.random() < 0.5:
            case["features"] = max(64, case["features"] // 64 * 64)
        most = listed()[5]
        size = most["experts"] * most["width"] * most["features"]
        while experts * case["width"] * case["features"] > size:
            case["features"] = case["features"] * 2 // 3
        size *= most["rows"] * most["top_k"] // most["experts"]
        while case["rows"] * case["top_k"] * case["width"] * case["features"] > size:
            case["rows"] = case["rows"] * 2 // 3
        return case
    if kind == "combine":
        width = _log(rng, 64, 8192)
        top_k = rng.randint(1, 8)
        return dict(op="combine", rows=min(_log(rng, 1, 8192), 4096 * 8 * 2048 // (width * top_k)),
                    top_k=top_k, width=width if rng.random() < 0.3 else (width + 7) // 8 * 8,
                    type=type_, add=rng.random() < 0.5)
    if kind == "score":
        vocab = _log(rng, 1000, 200000)
        rows = min(_log(rng, 1, 2048), 2048 * 128256 // vocab)
        type_ = rng.choice(("f32", "f16", "bf16"))
        return dict(op="score", rows=rows if type_ != "f32" else (rows + 1) // 2, vocab=vocab,
                    top=rng.choice((0, 1, 5, 20)), type=type_)
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    batch = _log(rng, 1, 64)
    prompts = rng.choice((0, batch))
    case = dict(op="append", batch=batch, prompts=prompts,
                tokens=_log(rng, 1, max(1, 8192 // batch)) if prompts else 1,
                context=_log(rng, 1, 8000), q_heads=kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8)),
                kv_heads=kv_heads, head_dim=head_dim, type=type_,
                rot=rng.choice((head_dim, head_dim // 2, 48)), interleaved=rng.random() < 0.5)
    most = work(listed()[9])["bytes"]
    while work(case)["bytes"] > most:
        case["tokens"] = case["tokens"] * 2 // 3
    return case


def _from(case):
    """A generator that goes by the case alone."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(tokens held, new tokens) of every sequence: from the case alone."""
    rng = _from(case)
    held, new = [], []
    for b in range(case["batch"]):
        first = b == 0  # the first sequence has the full lengths
        n = case["tokens"] if case["prompts"] else 1
        n = n if first or not case["prompts"] or n < 16 else rng.randint(n // 2, n)
        held.append(case["context"] if first else rng.randint(case["context"] // 4,
                                                              case["context"]))
        new.append(n)
    return held, new


def _chosen(case):
    """Experts [rows, top_k] of every token, some more popular than others: from the case alone
    (a state numbers the experts anew and shuffles the tokens)."""
    gen = torch.Generator().manual_seed(_from(case).getrandbits(40))
    like = torch.randn(case["rows"], case["experts"], generator=gen)
    like += 0.5 * torch.randn(case["experts"], generator=gen)
    return like.topk(min(case["top_k"], case["experts"]), dim=1)[1]


def work(case):
    """The bytes and operations that one pass cannot do without."""
    op = case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["type"]]
    if op == "route":
        t, e, k = case["rows"], case["experts"], case["top_k"]
        return {"bytes": t * e * size + 12 * t * k + 4 * (e + 1) + (4 * e if case["bias"] else 0),
                "flops": 6 * t * e}
    if op == "experts":
        chosen = _chosen(case)
        used, pairs = chosen.unique().numel(), chosen.numel()
        n, k = case["features"], case["width"]
        rows = pairs if case["per_pair"] else case["rows"]
        packed = n * k * case["bits"] // 8 + 2 * n * (k // GROUP) * size
        return {"bytes": used * packed + (rows * k + pairs * n) * size + 4 * pairs,
                "flops": 2 * pairs * n * k}
    if op == "combine":
        n = case["rows"] * case["width"]
        return {"bytes": n * (case["top_k"] + 1 + case["add"]) * size
                + 4 * case["rows"] * case["top_k"], "flops": 2 * n * case["top_k"]}
    if op == "score":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * (12 + 8 * case["top"]), "flops": 6 * n}
    held, new = _lengths(case)
    kvh, qh, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    bytes_, flops = 0, 0
    for h, n in zip(held, new):
        total = h + n
        done = total // BLOCK - h // BLOCK
        bytes_ += n * (qh + 2 * kvh) * d * 2 + n * qh * d * 2 + n * case["rot"] * 4
        # blocks that this call completes: the old tail is read, codes are written, and read again
        # with the values returned; the rest goes to the tail
        old = h % BLOCK if done else 0
        rest = total % BLOCK if done else n
        bytes_ += kvh * 2 * d * (2 * old + done * BLOCK * (1 + 1 + 2) + 2 * rest)
        flops += n * (qh + kvh) * (case["rot"] * 3 + d * 4) + done * BLOCK * kvh * 2 * d * 3
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------- preparation

def _plan(experts, n):
    """order and offsets of a routing."""
    flat = torch.where(experts < 0, n, experts).flatten().long()
    order = torch.sort(flat, stable=True)[1]
    offsets = (flat[:, None] < torch.arange(n + 1, device=flat.device)).sum(0)
    return order.int(), offsets.int()


def _packed(w, bits, dt):
    """Groups of w [N, K] in 4 or 8 bits: (words, scales, biases)."""
    n, k = w.shape
    g = w.view(n, k // GROUP, GROUP)
    low, high = g.amin(-1), g.amax(-1)
    scale, bias = ((high - low) / (2 ** bits - 1)).to(dt), low.to(dt)
    code = ((g - bias.float()[..., None]) / scale.float()[..., None]).round()
    code = code.clamp(0, 2 ** bits - 1).view(n, -1, 32 // bits).int()
    shift = torch.arange(0, 32, bits, device=w.device, dtype=torch.int32)
    return (code << shift).sum(-1, dtype=torch.int32), scale, bias


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
    dt = TYPES[case["type"]]
    if case["op"] == "route":
        popular = 0.5 * normal(case["experts"])
        s["logits"] = (1.5 * normal(case["rows"], case["experts"]) + popular).to(dt)
        s["bias"] = -0.2 * popular + 0.02 * normal(case["experts"]) if case["bias"] else None
        return s
    if case["op"] == "experts":
        n, k, e = case["features"], case["width"], case["experts"]
        x = _chosen(case).to(dev)
        x = torch.randperm(e, generator=gen, device=dev)[x]
        s["chosen"] = x[torch.randperm(case["rows"], generator=gen, device=dev)].int()
        s["order"], s["offsets"] = _plan(s["chosen"], e)
        s["weights"] = torch.softmax(normal(*x.shape), -1)
        s["most"] = int(s["offsets"].diff().max())
        parts = [_packed(normal(n, k) / math.sqrt(k), case["bits"], dt) for _ in range(e)]
        s["wq"], s["scales"], s["biases"] = (torch.stack(p) for p in zip(*parts))
        s["x"] = normal(x.numel() if case["per_pair"] else case["rows"], k).to(dt)
        if own:
            import int8_qmv_qmm_gb300 as q

            # the handle of a routing that the program has made before
            s["routing"] = q.Routing(s["chosen"], s["weights"], s["order"], s["offsets"])
        return s
    if case["op"] == "combine":
        t, k = case["rows"], case["top_k"]
        s["chosen"] = torch.rand(t, 64, generator=gen, device=dev).topk(k, dim=1)[1].int()
        s["weights"] = torch.softmax(normal(t, k), -1)
        s["order"], s["offsets"] = _plan(s["chosen"], 64)
        s["y"] = normal(t * k, case["width"]).to(dt)
        s["add"] = normal(t, case["width"]).to(dt) if case["add"] else None
        if own:
            import int8_qmv_qmm_gb300 as q

            s["routing"] = q.Routing(s["chosen"], s["weights"], s["order"], s["offsets"])
        return s
    if case["op"] == "score":
        rows, vocab = case["rows"], case["vocab"]
        x = 2.5 * normal(rows, vocab)
        x[:, ::997] += 6 * torch.rand(rows, 1, generator=gen, device=dev)  # likely tokens
        x[:, 5::1009] = -math.inf  # tokens that are not allowed
        s["logits"] = x.to(dt)
        # the text's tokens: half of them among the likely ones
        any_ = torch.randint(vocab // 1009, (rows,), generator=gen, device=dev)
        likely = torch.rand(rows, generator=gen, device=dev) < 0.5
        s["tokens"] = torch.where(likely, any_ * 997 % vocab, any_ * 1009 + 4).int()
        return s

    d, kvh, qh = case["head_dim"], case["kv_heads"], case["q_heads"]
    held, new = _lengths(case)
    batch = case["batch"]
    total = [h + n for h, n in zip(held, new)]
    blocks = [t // BLOCK for t in total]
    s["lens"] = torch.tensor(held, dtype=torch.int32, device=dev)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    # pages in no order; only the blocks that the call completes have their own
    first = [h // BLOCK for h in held]
    pages = sum(b - f for b, f in zip(blocks, first)) + 1
    place = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((batch, max(max(blocks), 1)), place[-1], dtype=torch.int32)
    at = 0
    for b in range(batch):
        n = blocks[b] - first[b]
        table[b, first[b] : blocks[b]] = torch.tensor(place[at : at + n], dtype=torch.int32)
        at += n
    s["table"] = table.to(dev)
    s["pages"] = torch.full((pages, kvh, 2, BLOCK * d), 128, dtype=torch.uint8, device=dev)
    s["scales"] = torch.zeros(pages, kvh, 2, device=dev)
    s["tail"] = normal(batch, kvh, 2, BLOCK * d).to(dt)
    spread = torch.ones(d, device=dev)
    spread[::16] = 4  # channels that stand out, as a linear's outputs have them
    x = normal(starts[-1], qh + 2 * kvh, d) * (0.5 + normal(starts[-1], 1, 1).abs())
    s["qkv"] = (x * spread).flatten(1).to(dt)
    s["q_norm"] = (1 + 0.2 * normal(d)).to(dt)
    s["k_norm"] = (1 + 0.2 * normal(d)).to(dt)
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
    return s


# ---------------------------------------------------------------------- the plain forms

def _plain_route(s):
    """Scores, choices and their sums are float32, operation by operation, so that near ties are
    the same wherever they are computed; without a bias the order is the logits' own."""
    c = s["case"]
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    e = torch.where(x == top, 1.0, (x - top).exp())
    if c["scoring"] == "softmax":
        score = e / e.double().sum(-1, keepdim=True).float()
    else:
        score = e = 1 / (1 + (-x).exp())
    key = x if s["bias"] is None else score + s["bias"]
    rows, n = x.shape
    if c["groups"] > 1:
        g = (e if s["bias"] is None and c["group_score"] == "top2" else key)
        g = torch.where(x == -math.inf, -math.inf, g).view(rows, c["groups"], -1)
        g = g.sort(dim=-1, descending=True)[0]
        value = g[..., 0]
        if c["group_score"] == "top2" and g.shape[-1] > 1:
            value = torch.where(g[..., 1] == -math.inf, g[..., 0], g[..., 0] + g[..., 1])
        best = value.sort(dim=-1, descending=True, stable=True)[1][:, : c["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(-1, best, True)
        kept = kept.repeat_interleave(n // c["groups"], -1)
    else:
        kept = torch.ones_like(x, dtype=torch.bool)
    key = torch.where(kept & (x > -math.inf), key, -math.inf)
    key, chosen = key.sort(dim=-1, descending=True, stable=True)
    key, chosen = key[:, : c["top_k"]], chosen[:, : c["top_k"]]
    w = torch.where(key > -math.inf, score.gather(-1, chosen), 0)
    if c["renormalise"]:
        w = w / w.double().sum(-1, keepdim=True).float()
    w = w * c["scale"]
    chosen = torch.where(key > -math.inf, chosen, -1).int()
    order, offsets = _plan(chosen, n)
    return {"experts": chosen, "weights": w, "order": order, "offsets": offsets}


def _weights_of(s, wq, scales, biases):
    """float32 weights of packed ones [.., N, K * bits / 32]."""
    bits = s["case"]["bits"]
    shift = torch.arange(0, 32, bits, device=wq.device, dtype=torch.int32)
    code = (wq[..., None] >> shift).bitwise_and_(2 ** bits - 1).flatten(-2).float()
    code = code.unflatten(-1, (-1, GROUP))
    return (code * scales.float()[..., None] + biases.float()[..., None]).flatten(-2)


def _plain_experts(s):
    x, chosen = s["x"].float(), s["chosen"].long()
    pairs = torch.arange(chosen.numel(), device=x.device)
    source = pairs if s["case"]["per_pair"] else pairs // chosen.shape[1]
    if chosen.numel() < s["wq"].shape[0]:  # few rows: a matrix for each
        e = chosen.flatten()
        w = _weights_of(s, s["wq"][e], s["scales"][e], s["biases"][e])
        return torch.matmul(w, x[source][..., None])[..., 0].to(s["x"].dtype)
    w = _weights_of(s, s["wq"], s["scales"], s["biases"])
    # the rows of every expert, padded to the most that one has
    order, offsets = s["order"].long(), s["offsets"].long()
    at = (offsets[:-1, None] + torch.arange(s["most"], device=x.device)).clamp(max=len(order) - 1)
    y = torch.matmul(x[source[order[at]]], w.transpose(-1, -2))
    e = chosen.flatten()[order]
    out = torch.empty(len(order), y.shape[-1], dtype=s["x"].dtype, device=x.device)
    out[order] = y[e, pairs - offsets[e]].to(out.dtype)
    return out


def _plain_combine(s):
    c = s["case"]
    y = s["y"].float().view(c["rows"], c["top_k"], -1)
    out = torch.matmul(s["weights"][:, None], y)[:, 0]
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(s["y"].dtype)


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
    qk = x[:, : qh + kvh]
    qk = qk / (qk.square().mean(-1, keepdim=True) + EPS).sqrt()
    weight = torch.cat((s["q_norm"].float().expand(qh, d), s["k_norm"].float().expand(kvh, d)))
    turned = _plain_rotate(qk * weight, s["rope"][pos], c["interleaved"]).to(dt)
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


def _plain_score(s):
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    d = x - x.amax(-1, keepdim=True)
    e = d.exp()
    z = e.sum(-1, keepdim=True, dtype=torch.float64)
    log_z = z.log()
    given = d.gather(-1, s["tokens"].long()[:, None]).double() - log_z
    # p * d is 0 where p is
    mean = torch.where(e > 0, e * d, 0).sum(-1, dtype=torch.float64) / z[:, 0]
    out = {"logprob": given[:, 0].float(), "entropy": (log_z[:, 0] - mean).float()}
    if s["case"]["top"]:
        best, index = s["logits"].sort(dim=-1, descending=True, stable=True)
        index = index[:, : s["case"]["top"]]
        out["top"] = index.int()
        out["top_logprob"] = (d.gather(-1, index).double() - log_z).float()
    return out


# ------------------------------------------------------------------- the framework's calls

def _own(s):
    import int8_qmv_qmm_gb300 as q

    c = s["case"]
    if c["op"] == "route":
        r = q.route_experts(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"],
                            groups=c["groups"], top_groups=c["top_groups"],
                            group_score=c["group_score"], renormalise=c["renormalise"],
                            scale=c["scale"])
        return {"experts": r.experts, "weights": r.weights, "order": r.order,
                "offsets": r.offsets}
    if c["op"] == "experts":
        return q.expert_linear(s["x"], s["routing"], s["wq"], s["scales"], s["biases"], c["bits"])
    if c["op"] == "combine":
        return q.combine_experts(s["y"], s["routing"], add=s["add"])
    if c["op"] == "score":
        logprob, entropy, top, top_logprob = q.token_logprobs(s["logits"], s["tokens"], c["top"])
        out = {"logprob": logprob, "entropy": entropy}
        if c["top"]:
            out["top"], out["top_logprob"] = top, top_logprob
        return out
    out = q.rope_append(s["qkv"], s["rope"], s["cache"], s["starts"], c["q_heads"],
                        interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                        eps=EPS)
    return {"q": out, "values": q.cache_dequant(s["cache"], s["filled"]), "scales": s["scales"],
            "tail": s["tail"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "experts": _plain_experts, "combine": _plain_combine,
            "append": _plain_append, "score": _plain_score}[state["case"]["op"]](state)


# ------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "combine": _exact_combine,
            "append": _exact_append, "score": _exact_score}[case["op"]](s)


def _exact_route(s):
    """The weights, of the experts that float32 scores choose."""
    c = s["case"]
    chosen = _plain_route(s)["experts"].long()
    x = s["logits"].double()
    score = torch.softmax(x, -1) if c["scoring"] == "softmax" else torch.sigmoid(x)
    w = torch.take_along_dim(score, chosen, 1)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"experts": None, "weights": w * c["scale"], "order": None, "offsets": None}


def _exact_experts(s):
    c = s["case"]
    n, k, bits = c["features"], c["width"], c["bits"]
    chosen = s["chosen"].flatten()
    out = torch.zeros(len(chosen), n, dtype=torch.float64, device=chosen.device)
    for e in chosen.unique().tolist():
        words = s["wq"][e].long() & 0xffffffff
        code = torch.stack([words >> (bits * i) & (2 ** bits - 1) for i in range(32 // bits)], 2)
        w = code.reshape(n, k // GROUP, GROUP).double()
        w = w * s["scales"][e].double().unsqueeze(2) + s["biases"][e].double().unsqueeze(2)
        pairs = (chosen == e).nonzero()[:, 0]
        x = s["x"][pairs if c["per_pair"] else pairs // c["top_k"]].double()
        out[pairs] = x @ w.reshape(n, k).t()
    return out


def _exact_combine(s):
    c = s["case"]
    y = s["y"].double().view(c["rows"], c["top_k"], c["width"])
    out = torch.einsum("tk,tkn->tn", s["weights"].double(), y)
    return out if s["add"] is None else out + s["add"].double()


def _exact_score(s):
    tokens = s["tokens"].long()
    out = {"logprob": [], "entropy": []}
    if s["case"]["top"]:
        out |= {"top": None, "top_logprob": []}
    for x, token in zip(s["logits"].double().split(256), tokens.split(256)):
        lp = torch.log_softmax(x, -1)
        out["logprob"].append(lp[torch.arange(len(x)), token])
        out["entropy"].append(torch.special.entr(lp.exp()).sum(-1))
        if s["case"]["top"]:
            out["top_logprob"].append(lp.topk(s["case"]["top"])[0])
    return {k: v if v is None else torch.cat(v) for k, v in out.items()}


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
        for heads, weight in ((slice(0, qh), s["q_norm"]), (slice(qh, qh + kvh), s["k_norm"])):
            rms = torch.sqrt(torch.einsum("thd,thd->th", x[:, heads], x[:, heads]) / d + EPS)
            x[:, heads] = torch.einsum("thd,d,th->thd", x[:, heads], weight.double(), 1 / rms)
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
