"""The decoder's calls as they are used together: overlapping one another, over many
slots, shared pages and used workspaces, and sampling of many unlike rows."""

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from oracle import decoder_oracle as O
from tests.test_gpu_decoder import (BF16, F16, F32, TINY, U, Model, dev, f64, normal,  # noqa: F401
                                    table_for)

pytestmark = pytest.mark.gpu


def test_overlapped_calls_give_the_same(dev):  # noqa: F811
    """norm, linear, append, attention, norm and sampling in a chain, each started
    while the one before runs: the same bits as one after the other."""
    hidden, heads, kvh, d, vocab, slots = 512, 8, 2, 64, 5000, 3
    width = (heads + 2 * kvh) * d
    packed = [q.quantize_affine((normal(i, n, hidden) * 0.05).float().to(dev), 8)
              for i, n in ((1, width), (2, hidden), (3, vocab))]
    weight = torch.ones(hidden, dtype=F16, device=dev)
    table, ws = table_for(dev, d), q.attention_workspace(d, dev)
    starts = torch.arange(slots + 1, dtype=torch.int32, device=dev)
    rows = dict(u=torch.tensor([0.1, 0.5, 0.9]), temperature=torch.tensor([0.9, 1.0, 0.0]),
                top_k=torch.tensor([40, 0, 0], dtype=torch.int32),
                top_p=torch.tensor([1.0, 0.9, 1.0]), min_p=torch.tensor([0.0, 0.0, 0.1]))
    rows = {k: v.to(dev) for k, v in rows.items()}
    seen = []
    for overlap in (False, True):
        m = Model(dev, slots, kvh, d, F16)
        m.append([200, 63, 1], heads, table, seed=9)
        got = []
        x = normal(10, slots, hidden).to(F16).to(dev)
        r = x.float()
        for _ in range(8):
            h, r = q.add_rms_norm(x, weight, r, residual_out=r, overlap_previous=overlap)
            qkv = q.qmv(h, *packed[0], 8, overlap_previous=overlap)
            query = q.rope_append(qkv, table, m.cache, starts, heads, overlap_previous=overlap)
            a = q.cache_attention(query, m.cache, starts, 1, ws, overlap_previous=overlap)
            x = q.qmv(a.view(slots, -1), *packed[1], 8, overlap_previous=overlap)
            h, r = q.add_rms_norm(x, weight, r, overlap_previous=overlap)
            logits = q.qmv(h, *packed[2], 8, overlap_previous=overlap)
            tokens, probs = q.sample(logits, **rows, overlap_previous=overlap)
            m.cache.lens += 1
            got += [x, r.clone(), tokens, probs]
        seen.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    assert q.device_status() == 0


@pytest.mark.parametrize("d,dt", [(64, F16), (128, BF16)])
def test_many_slots(dev, d, dt):  # noqa: F811
    """As many slots as a cache takes, a token each and some with none, one prompt."""
    slots = 1024
    m = Model(dev, slots, 1, d, dt, blocks=4)
    held = [(37 * b) % 131 for b in range(slots)]
    m.append(held, 2, table_for(dev, d, 256), seed=1)
    new = [0 if b % 7 == 3 else 1 for b in range(slots)]
    m.append(new, 2, table_for(dev, d, 256), seed=2, advance=False)
    total = sum(new)
    m.attend(new, 2, seed=3, only={0, 1, 100, 511, 512, 600, total - 1})
    m.cache.lens += torch.tensor(new, dtype=torch.int32, device=dev)
    new = [90 if b == 700 else int(b % 2) for b in range(slots)]
    m.append(new, 2, table_for(dev, d, 256), seed=4, advance=False)
    first = sum(new[:700])
    m.attend(new, 2, seed=5, only={0, 5, first - 1, first, first + 45, first + 89, first + 90,
                                   sum(new) - 1})
    m.check()
    assert q.device_status() == 0


def test_too_many_slots(dev):  # noqa: F811
    c = q.KVCache.empty(1025, 64, 1, 64, F16, dev)
    starts = torch.zeros(1026, dtype=torch.int32, device=dev)
    with pytest.raises(q.QlinError):
        q.rope_append(torch.zeros(1, 192, dtype=F16, device=dev), None, c, starts, 1)
    with pytest.raises(q.QlinError):
        q.cache_attention(torch.zeros(1, 1, 64, dtype=F16, device=dev), c, starts, 1,
                          q.attention_workspace(64, dev))


def test_shared_pages_and_a_used_workspace(dev):  # noqa: F811
    """Two slots whose first blocks are the same pages, and scratch with anything in
    it: as for slots with pages of their own and zeroed scratch."""
    out = []
    for shared in (False, True):
        m = Model(dev, 2, 2, 64, F16, blocks=6, seed=4)
        x = normal(5, 300, 8 * 64)
        m.append([128, 128], 4, None, values=torch.cat((x[:128], x[:128])))
        if shared:
            m.cache.table[1, :2] = m.cache.table[0, :2]
        m.append([40, 9], 4, None, values=x[128:177])
        m.append([1, 30], 4, None, values=x[177:208], advance=False)
        ws = q.attention_workspace(64, dev)
        if shared:
            ws.fill_(255)
        out.append(m.attend([1, 30], 4, seed=6, workspace=ws)[0])
    assert torch.equal(*out)
    assert q.device_status() == 0


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("m,v", [(1100, 300), (130, 20000)])
def test_sample_many_unlike_rows(dev, m, v, dt):  # noqa: F811
    """Rows with settings of every kind in one call: each as in a call of its own."""
    logits = (normal(1, m, v) * 2.5).to(dt).to(dev)
    kind = torch.arange(m) * 7 % 6
    pick = {"temperature": [1.0, 0.8, 0.7, 0.0, 1.3, 1.0], "top_p": [0.9, 1.0, 0.95, 1.0, 1.0, 0.5],
            "min_p": [0.0, 0.1, 0.0, 0.0, 0.0, 0.0]}
    rows = {k: torch.tensor(x, dtype=F32)[kind].to(dev) for k, x in pick.items()}
    rows["top_k"] = torch.tensor([0, 20, 5, 0, 0, 290], dtype=torch.int32)[kind].to(dev)
    rows["u"] = ((torch.arange(m) + 0.5) / m).to(dev)
    tokens, probs = q.sample(logits, **rows)
    for r in list(range(0, m, 13)) + [m - 1]:
        t, p = q.sample(logits[r:r + 1], **{k: x[r:r + 1].contiguous() for k, x in rows.items()})
        assert t.item() == tokens[r].item() and p.item() == probs[r].item(), (r, int(kind[r]))


@pytest.mark.parametrize("d,dt", [(64, F16), (128, BF16)])
def test_mixed_batches_back_to_back(dev, d, dt):  # noqa: F811
    """Prompts beside decoding sequences, call after call without a pause: the same
    bits as with the device idle before each call."""
    heads, kvh, new = 8, 2, [150, 1, 1, 40, 1, 200, 1]
    total, weight = sum(new), torch.ones(heads * d, dtype=dt, device=dev)
    table, ws = table_for(dev, d, 2048), q.attention_workspace(d, dev)
    x = [normal(i, total, (heads + 2 * kvh) * d).to(dt).to(dev) for i in range(6)]
    seen = []
    for pause in (True, False):
        m = Model(dev, len(new), kvh, d, dt, blocks=24)
        m.append([300, 700, 63, 0, 64, 10, 1], heads, table, seed=9)
        starts, got = m.starts(new), []
        counts = starts.diff()
        for qkv in x:
            query = q.rope_append(qkv, table, m.cache, starts, heads, overlap_previous=not pause)
            if pause:
                torch.cuda.synchronize()
            a = q.cache_attention(query, m.cache, starts, 200, ws, overlap_previous=not pause)
            if pause:
                torch.cuda.synchronize()
            h, _ = q.add_rms_norm(a.view(total, -1), weight, overlap_previous=not pause)
            if pause:
                torch.cuda.synchronize()
            got += [a, h]
            m.cache.lens += counts
        seen.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    assert q.device_status() == 0


def test_calls_without_rows(dev):  # noqa: F811
    """No token in any slot, no page, no row of logits: nothing happens."""
    m = Model(dev, 3, 2, 64, F16)
    m.append([70, 0, 5], 4, None, seed=1)
    before = [t.clone() for t in (m.cache.pages, m.cache.tail)]
    starts = m.starts([0, 0, 0])
    out = q.rope_append(torch.empty(0, 8 * 64, dtype=F16, device=dev), table_for(dev, 64),
                        m.cache, starts, 4)
    assert out.shape == (0, 4, 64)
    a = q.cache_attention(out, m.cache, starts, 0, q.attention_workspace(64, dev))
    assert a.shape == (0, 4, 64)
    assert q.cache_dequant(m.cache, starts[:0]).shape == (0, 2, 2, 64 * 64)
    none = torch.empty(0, device=dev)
    tokens, probs = q.sample(torch.empty(0, 100, device=dev), none, none,
                             torch.empty(0, dtype=torch.int32, device=dev), none, none)
    assert tokens.numel() == probs.numel() == 0
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for x, y in zip(before, (m.cache.pages, m.cache.tail)))
    m.check()
    assert q.device_status() == 0


@pytest.mark.parametrize("new", [1, 5, 100])
def test_a_block_without_a_page_is_left_out(dev, new):  # noqa: F811
    """As if its tokens were not there, in both kernels."""
    heads, kvh, d, held = 4, 2, 64, 250
    group = heads // kvh
    m = Model(dev, 1, kvh, d, F16, blocks=8)
    m.append([held], heads, None, seed=1)
    m.append([new], heads, None, seed=2, advance=False)
    m.cache.table[0, 1] = m.cache.pages.shape[0]
    x = (normal(3, new, heads, d) * 1.5).to(F16).to(dev)
    out = f64(q.cache_attention(x, m.cache, m.starts([new]), new, q.attention_workspace(d, dev)))
    assert q.device_status() == 2 << 24
    there = np.r_[0:64, 128:held + new]
    for h in range(kvh):
        k, v = (t[there] for t in m.values(0, h))
        for i in sorted({0, new // 2, new - 1}):
            for g in range(h * group, (h + 1) * group):
                ref, size, total, most = O.attention(f64(x)[i, g], k, v, held + i - 64, d ** -0.5)
                # the bound of Model.attend
                seen = held + i - 63
                e = (d + 8) * 2.0 ** -23 * (most + 1)
                bound = size * (2.0 ** -11 + 2 * e + (seen / 16 + 8) * 2.0 ** -22)
                bound += seen * 2.0 ** -25 * np.abs(v).max() / total
                bound += U[F16] * np.abs(ref) + TINY[F16]
                assert (np.abs(out[i, g] - ref) <= bound).all(), (h, i, g)
