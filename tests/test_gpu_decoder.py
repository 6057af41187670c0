"""GPU parity of what stands between a decoder's linears against the float64
oracle: RMS norm with the residual's addition, rotary positions and the 8-bit
cache, attention over it, sampling.

Tolerances come from the roundings that the definitions name (u = 2^-11 for
f16, 2^-8 for bf16: one rounding to nearest of a result) plus the float32
operations behind them (2^-24 each); each test says how it counts them."""

import math

import numpy as np
import pytest
import torch

import int8_qmv_qmm_gb300 as q
from oracle import decoder_oracle as O

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
BLOCK = q.KV_BLOCK


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_qmv_qmm_gb300 import build_lib
    build_lib.build()
    q.lib()
    return torch.device("cuda:0")


def normal(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape))


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, bound, what=""):
    err = np.abs(f64(got) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside; worst "
                           f"{float((err - bound).max())} over the bound")


# ------------------------------------------------------------------ RMS norm
def check_norm(dev, m, k, dt, rdt, seed=0, scale=1.0, x_pad=0, r_pad=0, shift=0, in_place=False,
               eps=1e-5):
    def place(v, dtype, pad):
        buf = torch.empty(m * (k + pad) + shift, dtype=dtype, device=dev)
        t = buf[shift:].view(m, k + pad)[:, :k]
        t.copy_(v.to(dtype))
        return t

    x = place(normal(seed, m, k) * scale, dt, x_pad)
    w = (1 + 0.3 * normal(seed + 1, k)).to(dt).to(dev)
    res = place(3 * scale * normal(seed + 2, m, k), rdt, r_pad) if rdt else None
    y_ref, h_ref = O.add_rms_norm(f64(x), f64(w), f64(res) if rdt else None, eps)
    out, new = q.add_rms_norm(x, w, res, eps=eps, residual_out=res if in_place else None,
                              out=x if in_place else None)
    # y: one rounding to dt; the float32 sum of squares (pairwise over at least
    # 32 lanes, runs of at most 1024) and the four operations on each element
    # stay within 2^-18.
    close(out, y_ref, (U[dt] + 2.0 ** -18) * np.abs(y_ref) + TINY[dt], "y")
    if rdt:
        close(new, h_ref, (U[rdt] + 2.0 ** -23) * np.abs(h_ref) + TINY[rdt], "residual")
    else:
        assert new is None
    return out, new


@pytest.mark.parametrize("dt,rdt", [(F16, F32), (F16, F16), (BF16, BF16), (BF16, F32),
                                    (F16, None)])
@pytest.mark.parametrize("m,k", [(1, 2048), (3, 1), (5, 64), (7, 2047), (2, 8192), (3, 8200),
                                 (2, 32768), (1, 32767), (300, 96), (9, 4104), (2, 12290)])
def test_norm(dev, m, k, dt, rdt):
    check_norm(dev, m, k, dt, rdt)


@pytest.mark.parametrize("kw", [dict(x_pad=8, r_pad=16), dict(x_pad=3), dict(r_pad=5),
                                dict(shift=1), dict(shift=4), dict(in_place=True),
                                dict(scale=1e-6), dict(scale=3000.0), dict(eps=0.5)])
def test_norm_strides_alignment_and_scales(dev, kw):
    check_norm(dev, 6, 512, F16, F32, **kw)
    check_norm(dev, 6, 511, BF16, BF16, **kw)


def test_norm_zero_rows_and_no_rows(dev):
    w = torch.ones(128, dtype=F16, device=dev)
    x = torch.zeros(3, 128, dtype=F16, device=dev)
    out, new = q.add_rms_norm(x, w, torch.zeros_like(x))
    assert (out == 0).all() and (new == 0).all()
    out, new = q.add_rms_norm(x[:0], w, x[:0])
    assert out.shape == (0, 128)


def test_norm_binding_refusals(dev):
    x = torch.zeros(4, 64, dtype=F16, device=dev)
    w = torch.ones(64, dtype=F16, device=dev)
    for bad in (dict(weight=w[:32]), dict(weight=w.float()), dict(residual=x.double()),
                dict(residual=x[:2]), dict(residual_out=x), dict(out=x[:2])):
        with pytest.raises(ValueError):
            q.add_rms_norm(x, **{"weight": w, **bad})
    with pytest.raises(q.QlinError):  # rows that overlap
        q.add_rms_norm(x[:1].expand(4, 64), w)


# ------------------------------------------------------------------ the table
@pytest.mark.parametrize("rot,base,scaling", [(64, 10000.0, {}), (16, 500000.0, {}),
                                              (128, 10000.0, dict(factor=4.0)),
                                              (64, 500000.0, dict(factor=32.0,
                                                                  short_wavelength=2048.0,
                                                                  long_wavelength=8192.0))])
def test_rope_table(dev, rot, base, scaling):
    n = 131072
    got = f64(q.rope_table(n, rot, base, device=dev, **scaling))
    f = O.rope_frequencies(rot, base, scaling.get("factor", 1.0),
                           scaling.get("short_wavelength", 0.0),
                           scaling.get("long_wavelength", 0.0))
    at = np.unique(np.concatenate([np.arange(300), np.arange(0, n, 997), [n - 1]]))
    angle = at[:, None] * f
    # float32 rounding, and the angle's float64 error: a few 2^-52 of 131071
    ref = np.stack((np.cos(angle), np.sin(angle)), -1)
    assert np.abs(got[at] - ref).max() <= 2.0 ** -25 + 2.0 ** -33


# ------------------------------------------------- rotation and the cache
class Model:
    """A cache on the GPU beside the tokens it should hold."""

    def __init__(self, dev, slots, kv_heads, d, dt, blocks=8, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        n_pages = slots * blocks + spare
        table = torch.from_numpy(rng.permutation(n_pages)[: slots * blocks].astype(np.int32))
        self.cache = q.KVCache.empty(slots, blocks * BLOCK, kv_heads, d, dt, dev, n_pages,
                                     table.view(slots, blocks).to(dev))
        # what was never written is as bad as it can be
        self.cache.pages.fill_(255)
        self.cache.scales.fill_(math.nan)
        self.cache.tail.fill_(math.nan)
        self.slots, self.kvh, self.d, self.dt, self.dev = slots, kv_heads, d, dt, dev
        self.k = [np.zeros((0, kv_heads, d), np.float32) for _ in range(slots)]
        self.v = [np.zeros((0, kv_heads, d), np.float32) for _ in range(slots)]

    def starts(self, new):
        return torch.tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32),
                            device=self.dev)

    def append(self, new, heads, table, interleaved=False, seed=0, pad=0, values=None,
               advance=True, scale=1.0):
        """One call with new[b] tokens of each slot; checks the queries."""
        rows, width = sum(new), (heads + 2 * self.kvh) * self.d
        x = normal(seed, rows, width) * scale if values is None else values
        buf = torch.zeros(rows, width + pad, dtype=self.dt, device=self.dev)
        qkv = buf[:, :width]
        qkv.copy_(x.to(self.dt))
        out = q.rope_append(qkv, table, self.cache, self.starts(new), heads, interleaved)
        x = qkv.float().cpu().numpy().reshape(rows, -1, self.d)
        pos = np.concatenate([len(self.k[b]) + np.arange(n) for b, n in enumerate(new)])
        turned = x[:, : heads + self.kvh]
        if table is not None:
            turned = O.rotate(turned, table.cpu().numpy()[pos.astype(int)], interleaved)
        turned = torch.from_numpy(turned).to(self.dt)
        assert torch.equal(out.cpu(), turned[:, :heads]), "queries"
        keys, vals = turned[:, heads:].float().numpy(), x[:, heads + self.kvh:]
        at = 0
        for b, n in enumerate(new):
            self.k[b] = np.concatenate([self.k[b], keys[at:at + n]])
            self.v[b] = np.concatenate([self.v[b], vals[at:at + n]])
            at += n
        if advance:
            self.cache.lens += torch.tensor(new, dtype=torch.int32, device=self.dev)
        return out

    def check(self):
        """The cache holds the tokens, bit for bit."""
        c, d = self.cache, self.d
        pages, scales = c.pages.cpu().numpy(), c.scales.cpu().numpy()
        tail, table = c.tail.float().cpu().numpy(), c.table.cpu().numpy()
        for b in range(self.slots):
            n = len(self.k[b])
            for j in range(n // BLOCK):
                at = slice(j * BLOCK, (j + 1) * BLOCK)
                for h in range(self.kvh):
                    for i, block in enumerate((self.k[b][at, h], self.v[b][at, h].T)):
                        codes, scale = O.quantise_block(block)
                        page = table[b, j]
                        assert scales[page, h, i] == scale, (b, j, h, i)
                        assert np.array_equal(pages[page, h, i].reshape(codes.shape), codes)
            left = n % BLOCK
            at = slice(n - left, n)
            for h in range(self.kvh):
                assert np.array_equal(tail[b, h, 0].reshape(BLOCK, d)[:left], self.k[b][at, h])
                assert np.array_equal(tail[b, h, 1].reshape(d, BLOCK)[:, :left],
                                      self.v[b][at, h].T)

    def values(self, b, h):
        """Keys and values of a slot's head as the cache stands for them, float64."""
        k, v = self.k[b][:, h].astype(np.float64), self.v[b][:, h].astype(np.float64)
        for j in range(len(k) // BLOCK):
            at = slice(j * BLOCK, (j + 1) * BLOCK)
            for x in (k, v):
                codes, scale = O.quantise_block(x[at].astype(np.float32))
                x[at] = (codes.astype(np.float64) - 128) * np.float64(scale)
        return k, v

    def attend(self, new, heads, seed=0, pad=0, q_scale=1.0, max_new=None, scale=None,
               workspace=None, only=None):
        """Attention of the last new[b] tokens of each slot (appended without
        advancing); checks every row, or the rows in `only`."""
        rows, d, group = sum(new), self.d, heads // self.kvh
        buf = torch.zeros(rows, heads * d + pad, dtype=self.dt, device=self.dev)
        qt = buf[:, : heads * d].view(rows, heads, d) if not pad else \
            buf.as_strided((rows, heads, d), (heads * d + pad, d, 1))
        qt.copy_((normal(seed + 77, rows, heads, d) * q_scale).to(self.dt))
        workspace = q.attention_workspace(d, self.dev) if workspace is None else workspace
        out = q.cache_attention(qt, self.cache, self.starts(new), max_new or max(new), workspace,
                                scale=scale)
        s = d ** -0.5 if scale is None else scale
        got, qn = f64(out), f64(qt)
        row = 0
        for b, n in enumerate(new):
            held = len(self.k[b]) - n
            if n and (only is None or any(row <= r < row + n for r in only)):
                for h in range(self.kvh):
                    k, v = self.values(b, h)
                    big = np.abs(v).max()
                    for i in range(n):
                        if only is not None and row + i not in only:
                            continue
                        for g in range(h * group, (h + 1) * group):
                            ref, size, total, most = O.attention(qn[row + i, g], k, v, held + i, s)
                            seen = held + i + 1
                            # a score's float32 sum of d products and the steps
                            # to exp2; its error e moves p and the total by e
                            # each; p rounds to f16 (2^-11, or 2^-25 of the
                            # largest below f16's normal range); the output's
                            # sum in float32, sixteen terms at a time
                            e = (d + 8) * 2.0 ** -23 * (most + 1)
                            bound = size * (2.0 ** -11 + 2 * e + (seen / 16 + 8) * 2.0 ** -22)
                            bound += seen * 2.0 ** -25 * big / total
                            bound += U[self.dt] * np.abs(ref) + TINY[self.dt]
                            err = np.abs(got[row + i, g] - ref)
                            assert (err <= bound).all(), (b, i, g, float((err / bound).max()))
            row += n
        return out, qt


def table_for(dev, rot, n=1024):
    return q.rope_table(n, rot, 10000.0, device=dev) if rot else None


@pytest.mark.parametrize("d,rot,interleaved,dt", [(64, 64, False, F16), (128, 128, True, BF16),
                                                  (128, 48, False, F16), (64, 32, True, BF16),
                                                  (64, 16, False, BF16), (128, 0, False, F16)])
def test_append_in_calls_of_every_size(dev, d, rot, interleaved, dt):
    m = Model(dev, 4, 3, d, dt)
    table = table_for(dev, rot)
    calls = [(1, 63, 64, 65), (0, 1, 1, 62), (62, 1, 0, 1), (2, 200, 130, 0), (1, 1, 1, 1),
             (127, 3, 61, 64), (1, 0, 0, 0)]
    for i, new in enumerate(calls):
        m.append(new, 6, table, interleaved, seed=i, pad=8 * (i % 2))
        m.check()
    assert q.device_status() == 0


def test_append_does_not_depend_on_the_calls(dev):
    """130 tokens at once, and one by one: the same cache, bit for bit."""
    table, heads, d, kvh = table_for(dev, 64), 4, 64, 2
    x = normal(5, 130, (heads + 2 * kvh) * d).to(F16).double()
    one, many = Model(dev, 1, kvh, d, F16), Model(dev, 1, kvh, d, F16)
    one.append((130,), heads, table, values=x)
    for i in range(130):
        many.append((1,), heads, table, values=x[i:i + 1])
    one.check()
    many.check()
    assert torch.equal(one.cache.pages, many.cache.pages)


def test_append_of_constant_and_extreme_blocks(dev):
    """A block of zeros has scale 0 and codes 128; the largest f16 values and
    subnormal ones keep their codes in range."""
    kvh, d, heads = 2, 64, 2
    for fill in (0.0, 65504.0, 6e-8, -1.0):
        m = Model(dev, 1, kvh, d, F16)
        x = torch.full((70, (heads + 2 * kvh) * d), fill, dtype=torch.float64)
        m.append((70,), heads, None, values=x)
        m.check()
        ids = m.cache.table[0, :1].contiguous()
        got = f64(q.cache_dequant(m.cache, ids))
        held = float(torch.tensor(fill).to(F16))  # what the cache was given
        assert np.abs(got - held).max() <= abs(held) * 2.0 ** -10


@pytest.mark.parametrize("d,dt", [(64, BF16), (128, F16)])
def test_cache_dequant(dev, d, dt):
    m = Model(dev, 2, 3, d, dt)
    m.append((200, 64), 3, table_for(dev, 32))
    ids = torch.cat((m.cache.table[0, :3], m.cache.table[1, :1])).contiguous()
    got = q.cache_dequant(m.cache, ids)
    codes = m.cache.pages[ids.long()].cpu().float() - 128
    ref = (codes * m.cache.scales[ids.long()].cpu()[..., None]).to(dt)
    assert torch.equal(got.cpu(), ref)
    assert q.cache_dequant(m.cache, ids[:0]).shape[0] == 0
    bad = torch.tensor([-1, 10 ** 6], dtype=torch.int32, device=dev)
    assert (q.cache_dequant(m.cache, bad) == 0).all()
    assert q.device_status() == 2 << 24


def test_append_refuses_on_the_device(dev):
    """What only the device can see is left out and reported: nothing of the
    slot is written, the others are."""
    table, heads = table_for(dev, 64, 100), 2
    for kind, bit in (("position", 4), ("blocks", 2), ("page", 2), ("rows", 1), ("lens", 1)):
        m = Model(dev, 2, 1, 64, F16, blocks=2 if kind == "blocks" else 8)
        c = m.cache
        new = [10, 70]
        if kind == "position":
            c.lens[1] = 64
        if kind == "blocks":
            c.lens[1] = 128 - 6
        if kind == "page":
            c.table[1] = 10 ** 8
        if kind == "lens":
            c.lens[1] = -3
        starts = m.starts(new)
        if kind == "rows":
            starts[2] = 200
        before = [t.clone() for t in (c.pages, c.scales, c.tail[1])]
        qkv = normal(3, 80, 4 * 64).to(F16).to(dev)
        big = q.rope_table(4096, 64, device=dev) if kind == "blocks" else table
        q.rope_append(qkv, big, c, starts, heads)
        assert q.device_status() == bit << 24, kind
        same = [torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                for a, b in zip(before, (c.pages, c.scales, c.tail[1]))]
        assert all(same[:2]), kind
        assert same[2] or kind == "page"  # (the tail beyond the lost block is kept)
        assert not c.tail[0, :, 0].view(64, 64)[:10].isnan().any()
    assert q.device_status() == 0


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("d,kvh,group", [(64, 2, 4), (128, 1, 8), (64, 3, 1), (128, 2, 5),
                                         (64, 1, 16), (128, 1, 3)])
def test_attention_single_tokens(dev, d, kvh, group, dt):
    """One new token of slots of every kind of length, idle slots between."""
    held = [0, 1, 62, 63, 64, 65, 127, 200, 511, 5]
    m = Model(dev, len(held) + 1, kvh, d, dt, blocks=9)
    table = table_for(dev, d)
    m.append(held + [0], kvh * group, table, seed=1)
    new = [1] * len(held) + [0]
    m.append(new, kvh * group, table, seed=2, advance=False)
    m.attend(new, kvh * group, seed=3, q_scale=2.0)
    assert q.device_status() == 0


@pytest.mark.parametrize("d,kvh,group,dt", [(64, 2, 4, F16), (128, 2, 5, BF16), (128, 1, 1, F16),
                                            (64, 1, 7, BF16)])
@pytest.mark.parametrize("new", [(2, 3, 4, 0, 1), (16, 33, 1, 7, 64), (130, 65, 128, 2, 129)])
def test_attention_several_tokens(dev, d, kvh, group, dt, new):
    """Drafts, chunks and prompts on top of what is held, causal inside."""
    held = [0, 40, 64, 100, 191]
    m = Model(dev, 5, kvh, d, dt, blocks=6)
    table = table_for(dev, 32)
    m.append(held, kvh * group, table, seed=11)
    m.append(new, kvh * group, table, seed=12, advance=False)
    m.attend(list(new), kvh * group, seed=13, q_scale=1.5, pad=8)
    assert q.device_status() == 0


@pytest.mark.parametrize("d,dt", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("new", [1, 3, 300])
def test_attention_over_a_long_cache(dev, d, dt, new):
    """A long sequence beside short ones: the split over the long axis."""
    held = [9000, 10, 700]
    m = Model(dev, 3, 2, d, dt, blocks=150)
    m.append(held, 8, None, seed=21)
    m.append([new, 1, 2], 8, None, seed=22, advance=False)
    ws = q.attention_workspace(d, dev)
    rows = {0, new - 1, new // 2, new, new + 1, new + 2}
    out, qt = m.attend([new, 1, 2], 8, seed=23, q_scale=2.0, workspace=ws, only=rows)
    again = q.cache_attention(qt, m.cache, m.starts([new, 1, 2]), max(new, 2), ws)
    assert torch.equal(out, again), "the same inputs, the same bits"
    wide = q.cache_attention(qt, m.cache, m.starts([new, 1, 2]), new + 900, ws)
    m_out = f64(wide) - f64(out)
    assert np.abs(m_out).max() <= 4 * U[dt] * np.abs(f64(out)).max()
    assert q.device_status() == 0


@pytest.mark.parametrize("scale", [0.0, 1e-4, 3.0])
def test_attention_scales_and_peaks(dev, scale):
    """From the plain mean of the values to one token that takes all."""
    m = Model(dev, 2, 1, 64, F16, blocks=6)
    m.append([300, 64], 2, None, seed=31, scale=2.0)
    m.append([1, 1], 2, None, seed=32, advance=False)
    m.attend([1, 1], 2, seed=33, scale=scale)


@pytest.mark.parametrize("dt,v_scale", [(F16, 1e-4), (F16, 200.0), (BF16, 1e-20), (BF16, 1e18)])
def test_attention_of_small_and_large_values(dev, dt, v_scale):
    """Values far from 1, and blocks whose scales differ by orders of magnitude."""
    heads, kvh, d = 4, 1, 64
    m = Model(dev, 1, kvh, d, dt, blocks=6)
    x = normal(41, 200, (heads + 2 * kvh) * d)
    x[:, (heads + kvh) * d:] *= v_scale
    x[64:128, (heads + kvh) * d:] *= 1e-3
    m.append([200], heads, None, values=x)
    y = normal(42, 40, (heads + 2 * kvh) * d)
    y[:, (heads + kvh) * d:] *= v_scale
    m.append([40], heads, None, values=y, advance=False)
    m.attend([40], heads, seed=43)


def test_attention_with_offsets_beyond_32_bits(dev):
    """Pages whose byte offsets pass 2^32."""
    kvh, d, n_pages = 8, 128, 33000  # 128 KB a page
    c = q.KVCache(torch.empty((n_pages, kvh, 2, 64 * d), dtype=torch.uint8, device=dev),
                  torch.zeros((n_pages, kvh, 2), device=dev),
                  torch.zeros((1, kvh, 2, 64 * d), dtype=F16, device=dev),
                  torch.tensor([[32999, 3, 16500, 32000]], dtype=torch.int32, device=dev),
                  torch.zeros(1, dtype=torch.int32, device=dev))
    m = Model(dev, 1, kvh, d, F16, blocks=4)
    m.cache = c
    m.append([200], 8, None, seed=51)
    m.append([20], 8, None, seed=52, advance=False)
    ids = c.table[0, :3].long()
    host = c.pages[ids].cpu().numpy()
    for j in range(3):
        codes, scale = O.quantise_block(m.k[0][j * 64:(j + 1) * 64, 7])
        assert np.array_equal(host[j, 7, 0].reshape(64, d), codes)
    m.attend([20], 8, seed=53, only={0, 19})
    m.attend([20], 8, seed=54, only={7}, max_new=4000)


def test_attention_refuses_on_the_device(dev):
    m = Model(dev, 2, 1, 64, F16)
    m.append([100, 100], 2, None, seed=61)
    m.append([1, 3], 2, None, seed=62, advance=False)
    ws = q.attention_workspace(64, dev)
    x = normal(63, 4, 2, 64).to(F16).to(dev)
    out = q.cache_attention(x, m.cache, m.starts([1, 3]), 2, ws)  # slot 1 has 3 rows
    assert (out[1:] == 0).all() and (out[0] != 0).any()
    assert q.device_status() == 8 << 24
    m.cache.table[0, 0] = -5  # a page that does not exist: the rest is attended
    out = q.cache_attention(x, m.cache, m.starts([1, 3]), 3, ws)
    assert torch.isfinite(out).all()
    assert q.device_status() == 2 << 24
    starts = m.starts([1, 3])
    starts[2] = 99
    out = torch.full_like(x, 7.0)
    q.cache_attention(x, m.cache, starts, 3, ws, out=out)
    assert (out[1:] == 7.0).all()
    assert q.device_status() & (1 << 24)
    with pytest.raises(ValueError):
        q.cache_attention(x.float(), m.cache, starts, 3, ws)
    with pytest.raises(ValueError):
        q.cache_attention(x, m.cache, starts[:2], 3, ws)
    with pytest.raises(q.QlinError):
        q.cache_attention(x, m.cache, starts, 3, ws[:16])


def test_attention_on_another_stream(dev):
    m = Model(dev, 2, 2, 64, F16)
    table = table_for(dev, 64)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.append([90, 5], 4, table, seed=71)
        m.append([1, 1], 4, table, seed=72, advance=False)
        m.attend([1, 1], 4, seed=73)
    side.synchronize()


# ------------------------------------------------------------------ sampling
def settings(dev, m, tau=1.0, k=0, p=1.0, mp=0.0):
    return (torch.full((m,), tau, device=dev), torch.full((m,), k, dtype=torch.int32, device=dev),
            torch.full((m,), p, device=dev), torch.full((m,), mp, device=dev))


def check_sample(dev, row, m=512, pad=0, **kw):
    """One row of logits drawn from m times with evenly spaced u: every token is
    the one whose share of the float64 distribution holds u, up to the edges'
    error, and its probability is that share.  The weights' float32 exponential
    is good to 2^-22 relative (its argument's rounding: 2^-24 of at most 25, the
    rest weighs under 2^-36, plus 2 ulp), the whole-number weights to 2^-37 of
    the largest each; a cut that moves by one element of weight w moves the
    edges by w, so cuts next to a near-tie with the bound are not tested here."""
    v = row.numel()
    buf = torch.zeros(m, v + pad, dtype=row.dtype, device=dev)
    x = buf[:, :v]
    x.copy_(row.to(dev).expand(m, v))
    u = (torch.arange(m, device=dev) + 0.5) / m
    tokens, probs = q.sample(x, u, *settings(dev, m, **kw))
    # (the settings as the float32 values that the kernel is given)
    p = O.sample_distribution(f64(row), float(np.float32(kw.get("tau", 1.0))), kw.get("k", 0),
                              float(np.float32(kw.get("p", 1.0))),
                              float(np.float32(kw.get("mp", 0.0))))
    tokens, probs, u = tokens.cpu().numpy(), f64(probs), f64(u)
    if p is None:
        assert (tokens == -1).all() and (probs == 0).all()
        return tokens
    cum = np.cumsum(p)
    eps = 2.0 ** -19 + v * 2.0 ** -36
    assert (tokens >= 0).all() and (tokens < v).all()
    assert (p[tokens] > 0).all(), "a token that is not kept"
    assert (cum[tokens] >= u - eps).all() and (cum[tokens] - p[tokens] <= u + eps).all()
    assert (np.abs(probs - p[tokens]) <= eps * p[tokens] + v * 2.0 ** -36).all()
    return tokens


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("v", [1, 2, 31, 1000, 4097, 50257, 128256])
def test_sample(dev, dt, v):
    row = (3.0 * normal(v, v)).to(dt)
    for kw in (dict(), dict(tau=0.7), dict(k=5), dict(k=1), dict(p=0.9), dict(mp=0.1),
               dict(k=40, p=0.8, mp=0.02, tau=1.3), dict(p=1e-9), dict(tau=0.0),
               dict(k=v), dict(k=max(1, v // 2), p=0.95), dict(p=0.5, tau=5.0)):
        check_sample(dev, row, m=96, pad=3, **kw)


def test_sample_ties_go_to_the_lowest_index(dev):
    flat = torch.zeros(3000, dtype=F32)
    assert set(check_sample(dev, flat, k=7)) == set(range(7))
    assert set(check_sample(dev, flat, p=0.01)) == set(range(30))
    assert set(check_sample(dev, flat, tau=0.0)) == {0}
    assert len(set(check_sample(dev, flat, m=3000))) == 3000
    mixed = torch.full((40000,), -1.0, dtype=BF16)
    mixed[17::13] = 2.0
    mixed[5] = 4.0
    assert set(check_sample(dev, mixed, k=4)) == {5, 17, 30, 43}
    signed = torch.tensor([-0.0, 0.0, -0.0, 0.0], dtype=F32)  # one value
    assert set(check_sample(dev, signed, k=2)) == {0, 1}


def test_sample_masked_and_special_logits(dev):
    row = 2.0 * normal(9, 700).float()
    row[::2] = -math.inf
    row[1::4] = torch.finfo(F32).min
    row[3] = math.nan
    check_sample(dev, row)
    check_sample(dev, row, k=300, p=0.99)
    check_sample(dev, torch.full((50,), -math.inf))
    check_sample(dev, torch.full((50,), math.nan))
    row[7] = row[9] = math.inf
    assert set(check_sample(dev, row)) == {7, 9}
    assert set(check_sample(dev, torch.full((50,), torch.finfo(F16).min, dtype=F16))) == set(
        range(50))


def test_sample_limits_of_u(dev):
    row = torch.tensor([0.0, 1.0, 2.0, -math.inf], device=dev)
    u = torch.tensor([0.0, 1.0, -1.0, 2.0, math.nan], device=dev)
    tokens, _ = q.sample(row.expand(5, 4).contiguous(), u, *settings(dev, 5))
    assert tokens.tolist() == [0, 2, 0, 2, 0]


def test_sample_rows_do_not_depend_on_each_other(dev):
    """Every row with settings of its own, alone and in a batch: the same bits."""
    m, v = 37, 20011
    x = (2.5 * normal(4, m, v)).to(F16).to(dev)
    gen = np.random.default_rng(8)
    u = torch.from_numpy(gen.random(m)).float().to(dev)
    tau = torch.from_numpy(gen.choice([0.0, 0.6, 1.0, 1.5], m)).float().to(dev)
    k = torch.from_numpy(gen.choice([0, 1, 20, 5000], m)).int().to(dev)
    p = torch.from_numpy(gen.choice([0.3, 0.9, 1.0], m)).float().to(dev)
    mp = torch.from_numpy(gen.choice([0.0, 0.05], m)).float().to(dev)
    tokens, probs = q.sample(x, u, tau, k, p, mp)
    for i in range(m):
        at = slice(i, i + 1)
        t, r = q.sample(x[at], u[at], tau[at], k[at], p[at], mp[at])
        assert t.item() == tokens[i].item() and r.item() == probs[i].item()
        dist = O.sample_distribution(f64(x[i]), tau[i].item(), k[i].item(), p[i].item(),
                                     mp[i].item())
        assert dist[t.item()] > 0


def test_sample_largest_vocabulary(dev):
    row = (2.0 * normal(6, 262144)).float()
    check_sample(dev, row, m=16)
    check_sample(dev, row, m=16, p=0.9)
    check_sample(dev, row, m=16, k=100)
    empty = q.sample(row.to(dev).view(1, -1)[:0], *(t[:0] for t in (
        torch.zeros(1, device=dev), *settings(dev, 1))))
    assert empty[0].shape == (0,)
