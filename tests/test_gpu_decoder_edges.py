"""GPU parity of the calls between a decoder's linears where their work splits unevenly
or their values are far apart, infinite or NaN, against the float64 oracle."""

import math

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from oracle import decoder_oracle as O
from tests.test_gpu_decoder import (BF16, BLOCK, F16, F32, TINY, U, Model,  # noqa: F401
                                    check_sample, close, dev, f64, normal, settings)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ sampling
@pytest.mark.parametrize("v", [8200, 16392, 33000])
def test_sample_small_parts_of_a_row(dev, v):  # noqa: F811
    """Clusters of 2, 4 and 8 CTAs whose first exchange comes soon after their start:
    the same token every time, and the oracle's."""
    row = (2.5 * normal(v, v)).to(F32)
    check_sample(dev, row, m=8, p=0.9)
    x, u = row.to(dev).view(1, v), torch.tensor([0.37], device=dev)
    got = [q.sample(x, u, *settings(dev, 1, p=0.9)) for _ in range(300)]
    assert len({(t.item(), p.item()) for t, p in got}) == 1


@pytest.mark.parametrize("dt", [F32, F16])
@pytest.mark.parametrize("v", [131009, 131071, 131073, 131463, 131464])
def test_sample_where_the_last_part_is_short(dev, v, dt):  # noqa: F811
    """Eight CTAs share a row, the last with fewer than 16384 logits, the others with
    16384 or more: a bound by weight, alone and after top-k."""
    row = (3.0 * normal(v, v)).to(dt)
    for kw in (dict(p=0.9), dict(p=0.3, tau=2.0), dict(k=v // 2, p=0.95), dict(p=0.7, mp=0.01),
               dict(k=50, p=0.9), dict(p=0.999, tau=0.5)):
        check_sample(dev, row, m=16, **kw)


# ------------------------------------------------------------------ attention
def test_parts_of_both_kernels_joined_in_one_call(dev):  # noqa: F811
    """Sequences that decode over caches long enough to be cut, beside prompts whose
    tiles are cut too: both kernels leave parts, and one launch joins them."""
    m = Model(dev, 5, 2, 64, F16, blocks=70)
    m.append([4000, 3000, 200, 2500, 0], 8, None, seed=1)
    new = [1, 2, 150, 1, 90]
    m.append(new, 8, None, seed=2, advance=False)
    m.attend(new, 8, seed=3, q_scale=1.5, only={0, 1, 2, 3, 80, 152, 153, 154, 200, 243})
    assert q.device_status() == 0


def attend_copies(m, n, copies, x, max_new=None, scale=None, check=True):
    """cache_attention over `copies` sequences that are all slot 0 of m (shared pages),
    so that warps and CTAs walk over several blocks, with the n last tokens of each as
    the rows of x.  For rows of the first and the last sequence, what the float64 oracle
    and the definition's roundings need: (out, [(row, head, ref, size, total, most, seen,
    largest)]), largest being the largest p_j * max|v of j's block|."""
    c, heads = m.cache, x.shape[1]
    many = q.KVCache(c.pages, c.scales, *(t[:1].repeat(copies, *[1] * (t.dim() - 1))
                                          for t in (c.tail, c.table, c.lens)))
    out = q.cache_attention(x, many, m.starts([n] * copies), max_new or n,
                            q.attention_workspace(m.d, m.dev), scale=scale)
    s = m.d ** -0.5 if scale is None else scale
    rows, held, group = [], len(m.k[0]) - n, heads // m.kvh
    for h in range(m.kvh if check else 0):
        k, v = m.values(0, h)
        tops = np.repeat([np.abs(v[j:j + BLOCK]).max() for j in range(0, len(v), BLOCK)],
                         BLOCK)[:len(v)]
        for first in sorted({0, (copies - 1) * n}):
            for i in sorted({0, n // 2, n - 1}):
                seen = held + i + 1
                for g in range(h * group, (h + 1) * group):
                    xn = f64(x[first + i, g])
                    ref, size, total, most = O.attention(xn, k, v, held + i, s)
                    p = k[:seen] @ xn * s
                    p = np.exp(p - p.max()) / total
                    rows.append((first + i, g, ref, size, total, most, seen,
                                 (p * tops[:seen]).max()))
    return out, rows


@pytest.mark.parametrize("d,dt,small,large", [(64, F16, 2.0 ** -13, 2.0 ** 13),
                                              (128, F16, 2.0 ** -13, 2.0 ** 13),
                                              (64, BF16, 2.0 ** -20, 2.0 ** 20),
                                              (128, BF16, 1.0, 2.0 ** 40)])
@pytest.mark.parametrize("n,copies", [(1, 200), (3, 100), (100, 40)])
@pytest.mark.parametrize("at", [0, 3])
def test_attention_beside_a_block_of_large_values(dev, d, dt, small, large, n, copies,  # noqa: F811
                                                  at):
    """One block's values are far larger than all others', and its keys leave it no
    probability: the small values' sums keep their precision.

    Bound: probabilities enter the second product in f16 in units of the largest
    p * (value scale) so far, so that a token is off by 2^-11 of itself or 2^-25 of that
    unit (2^-24 here, since a bf16 tail's unit is a power of two), times its block's
    largest code; the rest as in Model.attend."""
    heads, kvh, held = 16, 4, 700
    m = Model(dev, 1, kvh, d, dt, blocks=13)
    x = normal(1, held + n, (heads + 2 * kvh) * d)
    parts = x.view(held + n, heads + 2 * kvh, d)
    big = slice(at * BLOCK, (at + 1) * BLOCK)
    parts[:, heads:heads + kvh, 0] = 0.0
    parts[big, heads:heads + kvh, 0] = -60.0  # against sqrt(d) in every query: exp(-60)
    parts[:, heads + kvh:] *= small
    parts[big, heads + kvh:] *= large / small
    m.append([held], heads, None, values=x[:held])
    m.append([n], heads, None, values=x[held:], advance=False)
    qx = normal(2, n * copies, heads, d)
    qx[..., 0] = math.sqrt(d)
    out, rows = attend_copies(m, n, copies, qx.to(dt).to(dev))
    for row, g, ref, size, total, most, seen, largest in rows:
        e = (d + 8) * 2.0 ** -23 * (most + 1)
        bound = size * (2.0 ** -11 + 2 * e + (seen / 16 + 8) * 2.0 ** -22)
        bound += seen * 2.0 ** -24 * largest + U[dt] * np.abs(ref) + TINY[dt]
        close(out[row, g], ref, bound, f"row {row} head {g}")
    assert q.device_status() == 0


@pytest.mark.parametrize("d,dt", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("n,copies", [(1, 1), (1, 200), (3, 1), (3, 100), (100, 1), (100, 40)])
@pytest.mark.parametrize("where", ["query", "key"])
def test_attention_of_nan(dev, d, dt, n, copies, where):  # noqa: F811
    """A row whose query, or whose own key, is NaN is NaN, whether one warp or CTA
    finishes it or its parts are joined; all other rows keep their bits."""
    heads, kvh, held = 16, 4, 700
    m = Model(dev, 1, kvh, d, dt, blocks=13)
    m.append([held], heads, None, seed=1)
    x = normal(2, n, (heads + 2 * kvh) * d)
    m.append([n], heads, None, values=x, advance=False)
    qx = normal(3, n * copies, heads, d).to(dt).to(dev)
    clean, _ = attend_copies(m, n, copies, qx, check=False)
    bad = torch.zeros(n * copies, heads, dtype=torch.bool, device=dev)
    if where == "query":
        for row, g in ((0, 1), (n * copies - 1, 14)):
            qx[row, g, d // 3] = math.nan
            bad[row, g] = True
    else:  # of the last token, which only the last row of each sequence sees
        x.view(n, -1, d)[n - 1, heads + 2, 5] = math.nan
        m = Model(dev, 1, kvh, d, dt, blocks=13)
        m.append([held], heads, None, seed=1)
        q.rope_append(x.to(dt).to(dev), None, m.cache, m.starts([n]), heads)
        bad[n - 1::n, 8:12] = True
    out, _ = attend_copies(m, n, copies, qx, check=False)
    assert out[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad])
    assert q.device_status() == 0


@pytest.mark.parametrize("d,dt", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["key", "value"])
def test_a_completed_block_that_is_not_finite(dev, d, dt, value, which):  # noqa: F811
    """Its scale is infinite, it stands for NaN, and so do the rows that see it, in both
    kernels; the blocks, heads and rows beside it keep their bits."""
    heads, kvh, held = 16, 4, 100
    out = []
    for bad in (False, True):
        m = Model(dev, 1, kvh, d, dt, blocks=13)
        x = normal(4, held + 150, (heads + 2 * kvh) * d).to(dt)
        if bad:  # token 130, of head 2, in block 2: rows 30 - .. see it
            at = heads + 2 if which == "key" else heads + kvh + 2
            x.view(held + 150, -1, d)[130, at, 7] = value
        q.rope_append(x[:held].to(dev), None, m.cache, m.starts([held]), heads)
        m.cache.lens += held
        q.rope_append(x[held:].to(dev), None, m.cache, m.starts([150]), heads)
        ids = m.cache.table[0, :3].contiguous()
        back = q.cache_dequant(m.cache, ids)
        qx = normal(5, 150, heads, d).to(dt).to(dev)
        ws = q.attention_workspace(d, dev)
        tile = q.cache_attention(qx, m.cache, m.starts([150]), 150, ws)
        m.cache.lens += 146  # the same with the last four tokens alone
        few = q.cache_attention(qx[146:], m.cache, m.starts([4]), 4, ws)
        out.append((back, m.cache.scales[ids.long()].clone(), tile, few))
    (back0, scales0, tile0, few0), (back, scales, tile, few) = out
    here = torch.zeros(3, kvh, 2, dtype=torch.bool, device=dev)
    here[2, 2, 0 if which == "key" else 1] = True
    assert torch.equal(scales[~here], scales0[~here]) and (scales[here] == math.inf).all()
    assert torch.equal(back[~here], back0[~here]) and back[here].isnan().all()
    rows = torch.zeros(150, heads, dtype=torch.bool, device=dev)
    # the whole block is NaN, so a row that sees its first token, 128, does
    rows[128 - held:, 8:12] = True
    assert tile[rows].isnan().all() and torch.equal(tile[~rows], tile0[~rows])
    assert few[rows[146:]].isnan().all() and torch.equal(few[~rows[146:]], few0[~rows[146:]])
    assert q.device_status() == 0


@pytest.mark.parametrize("d,dt", [(64, F16), (128, F16), (64, BF16), (128, BF16)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["key", "value"])
@pytest.mark.parametrize("n", [3, 13, 50])
def test_a_tail_that_is_not_finite(dev, d, dt, value, which, n):  # noqa: F811
    """A token of the incomplete block, one that the first rows of the call do not see:
    those keep their bits, the others are not finite."""
    heads, kvh, held, at = 16, 4, 201, 2 if n < 50 else 30
    out = []
    for bad in (False, True):
        m = Model(dev, 1, kvh, d, dt, blocks=13)
        x = normal(6, held + n, (heads + 2 * kvh) * d).to(dt)
        if bad:
            head = heads + 1 if which == "key" else heads + kvh + 1
            x.view(held + n, -1, d)[held + at, head, 3] = value
        q.rope_append(x[:held].to(dev), None, m.cache, m.starts([held]), heads)
        m.cache.lens += held
        q.rope_append(x[held:].to(dev), None, m.cache, m.starts([n]), heads)
        qx = normal(7, n, heads, d).to(dt)
        qx[..., 3] = 0.5  # (no product of zero and infinity)
        ws = q.attention_workspace(d, dev)
        out.append(q.cache_attention(qx.to(dev), m.cache, m.starts([n]), n, ws))
    rows = torch.zeros(n, heads, dtype=torch.bool, device=dev)
    rows[at:, 4:8] = True
    if which == "key" and value == -math.inf:  # no probability for that token, and no harm
        assert out[1][rows].isfinite().all()
    else:
        assert (~out[1][rows].isfinite()).any(-1).all()
    assert torch.equal(out[1][~rows], out[0][~rows])
    assert q.device_status() == 0


@pytest.mark.parametrize("n,copies", [(1, 60), (3, 40), (100, 2), (100, 40)])
@pytest.mark.parametrize("dt,scale", [(F16, 0.0), (F16, -0.2), (BF16, -0.05), (F16, 2.0)])
def test_attention_scales_of_both_kernels(dev, n, copies, dt, scale):  # noqa: F811
    """Negative and zero scales among them; from few rows to whole rounds of tiles."""
    heads, kvh, d, held = 16, 4, 64, 500
    m = Model(dev, 1, kvh, d, dt, blocks=13)
    m.append([held], heads, None, seed=1)
    m.append([n], heads, None, seed=2, advance=False)
    x = normal(3, n * copies, heads, d).to(dt).to(dev)
    out, rows = attend_copies(m, n, copies, x, scale=scale)
    for row, g, ref, size, total, most, seen, largest in rows:  # (as beside large values)
        e = (d + 8) * 2.0 ** -23 * (abs(most) + 1)
        bound = size * (2.0 ** -11 + 2 * e + (seen / 16 + 8) * 2.0 ** -22)
        bound += seen * 2.0 ** -24 * largest + U[dt] * np.abs(ref) + TINY[dt]
        close(out[row, g], ref, bound, f"row {row} head {g}")
    assert q.device_status() == 0


def test_prompts_with_offsets_beyond_32_bits(dev):  # noqa: F811
    """Pages whose byte offsets pass 2^32, read for more rows than single tokens."""
    kvh, d, n_pages = 8, 128, 33000  # 128 KB a page
    c = q.KVCache(torch.empty((n_pages, kvh, 2, 64 * d), dtype=torch.uint8, device=dev),
                  torch.zeros((n_pages, kvh, 2), device=dev),
                  torch.zeros((1, kvh, 2, 64 * d), dtype=BF16, device=dev),
                  torch.tensor([[32999, 3, 16500, 32000, 32768]], dtype=torch.int32, device=dev),
                  torch.zeros(1, dtype=torch.int32, device=dev))
    m = Model(dev, 1, kvh, d, BF16, blocks=5)
    m.cache = c
    m.append([200], 8, None, seed=51)
    m.append([100], 8, None, seed=52, advance=False)
    m.attend([100], 8, seed=53, only={0, 50, 99})
    assert q.device_status() == 0


@pytest.mark.parametrize("n,copies", [(1, 1), (3, 60), (100, 40)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_attention_of_an_infinite_query(dev, dt, n, copies):  # noqa: F811
    """The row is not finite; the others keep their bits."""
    heads, kvh, d = 16, 4, 64
    m = Model(dev, 1, kvh, d, dt, blocks=13)
    m.append([300], heads, None, seed=1)
    m.append([n], heads, None, seed=2, advance=False)
    x = normal(3, n * copies, heads, d).to(dt).to(dev)
    clean, _ = attend_copies(m, n, copies, x, check=False)
    x[0, 3, 5] = math.inf
    out, _ = attend_copies(m, n, copies, x, check=False)
    assert not out[0, 3].isfinite().any()
    out[0, 3] = clean[0, 3]
    assert torch.equal(out, clean)
    assert q.device_status() == 0


def test_prompts_between_products_of_the_tensor_cores(dev):  # noqa: F811
    """Both kinds of kernel take tensor memory, and each starts while the one before it
    runs: small products after prompts, call after call, the same bits as with pauses."""
    heads, kvh, d, slots, n = 8, 2, 64, 12, 60
    rows, width = slots * n, (heads + 2 * kvh) * d
    packed = q.quantize_affine((normal(1, width, heads * d) * 0.05).float().to(dev), 8)
    starts = torch.arange(slots + 1, dtype=torch.int32, device=dev) * n
    ws, table = q.attention_workspace(d, dev), q.rope_table(512, d, device=dev)
    seen = []
    for pause in (True, False):
        m = Model(dev, slots, kvh, d, F16)
        x, got = normal(2, rows, heads * d).to(F16).to(dev), []
        for _ in range(6):
            qkv = q.qmm(x, *packed, 8, overlap_previous=not pause)
            if pause:
                torch.cuda.synchronize()
            query = q.rope_append(qkv, table, m.cache, starts, heads, overlap_previous=not pause)
            a = q.cache_attention(query, m.cache, starts, n, ws, overlap_previous=not pause)
            if pause:
                torch.cuda.synchronize()
            x = q.qmm(a.view(rows, -1), *packed, 8,
                      overlap_previous=not pause)[:, :heads * d].contiguous()
            m.cache.lens += n
            got.append(x)
        seen.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    assert q.device_status() == 0
