"""Host-side tests of the entry points between a decoder's linears: every bad
argument is refused before anything is launched (no GPU: no call here reaches a
launch)."""

import ctypes

import pytest
import torch

import int8_qmv_qmm_gb300 as q
from int8_qmv_qmm_gb300 import build_lib

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
FAKE = 0x10000  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return q.lib()


def cache(**over):
    v = dict(pages=FAKE, scales=FAKE, tail=FAKE, table=FAKE, lens=FAKE, n_pages=4, slots=2,
             max_blocks=2, kv_heads=2, head_dim=64, dtype=q.QLIN_F16)
    v.update(over)
    return q._KVCacheStruct(*(v[f] for f, _ in q._KVCacheStruct._fields_))


CACHE_FAULTS = [(dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
                (dict(dtype=q.QLIN_F32), UNSUPPORTED), (dict(slots=0), INVALID),
                (dict(kv_heads=0), INVALID), (dict(n_pages=0), INVALID),
                (dict(max_blocks=-1), INVALID), (dict(pages=0), INVALID),
                (dict(table=0), INVALID), (dict(lens=0), INVALID),
                (dict(tail=FAKE + 8), MISALIGNED), (dict(pages=FAKE + 4), MISALIGNED),
                (dict(scales=FAKE + 4), MISALIGNED), (dict(lens=FAKE + 2), MISALIGNED)]


def norm(L, x=FAKE, xs=64, w=FAKE, r=FAKE, rs=64, ro=FAKE, y=FAKE, M=3, K=64, eps=1e-5,
         dt=q.QLIN_F16, rdt=q.QLIN_F32, flags=0):
    return L.qlin_add_rms_norm(x, xs, w, r, rs, ro, y, M, K, eps, dt, rdt, flags, None)


def test_norm_refusals(L):
    assert norm(L, dt=q.QLIN_F32) == UNSUPPORTED
    assert norm(L, rdt=q.QLIN_BF16) == UNSUPPORTED
    assert norm(L, K=32769, xs=40000, rs=40000) == UNSUPPORTED
    assert norm(L, K=0) == INVALID
    assert norm(L, M=-1) == INVALID
    assert norm(L, eps=-1.0) == INVALID
    assert norm(L, eps=float("nan")) == INVALID
    assert norm(L, flags=2) == INVALID
    assert norm(L, x=None) == INVALID
    assert norm(L, r=None) == INVALID          # residual_out without a residual
    assert norm(L, xs=63) == INVALID
    assert norm(L, rs=63) == INVALID
    assert norm(L, x=FAKE + 1) == MISALIGNED
    assert norm(L, r=FAKE + 2) == MISALIGNED   # float32 residual
    assert norm(L, M=0, x=None, y=None) == OK


def test_rope_table_refusals(L):
    def table(p=FAKE, n=8, rot=64, base=1e4, f=1.0, s=0.0, l=0.0):
        return L.qlin_rope_table(p, n, rot, base, f, s, l, None)

    assert table(rot=63) == INVALID
    assert table(rot=0) == INVALID
    assert table(n=-1) == INVALID
    assert table(base=1.0) == INVALID
    assert table(base=float("inf")) == INVALID
    assert table(f=0.5) == INVALID
    assert table(s=2.0, l=1.0) == INVALID
    assert table(s=-1.0) == INVALID
    assert table(p=None) == INVALID
    assert table(p=FAKE + 4) == MISALIGNED
    assert table(n=0, p=None) == OK


def append(L, c=None, qkv=FAKE, qs=8 * 64, out=FAKE, table=FAKE, n=100, rot=64, inter=0,
           starts=FAKE, T=3, heads=4, flags=0):
    c = c or cache()
    return L.qlin_rope_append(qkv, qs, out, table, n, rot, inter, ctypes.byref(c), starts, T,
                              heads, flags, None)


def test_rope_append_refusals(L):
    for over, status in CACHE_FAULTS:
        assert append(L, cache(**over)) == status, over
    assert L.qlin_rope_append(FAKE, 512, FAKE, FAKE, 1, 64, 0, None, FAKE, 1, 4, 0, None) == INVALID
    assert append(L, rot=24) == UNSUPPORTED
    assert append(L, rot=80) == UNSUPPORTED
    assert append(L, rot=-16) == UNSUPPORTED
    assert append(L, inter=2) == INVALID
    assert append(L, heads=3) == INVALID
    assert append(L, heads=0) == INVALID
    assert append(L, heads=34, qs=40 * 64) == UNSUPPORTED
    assert append(L, T=-1) == INVALID
    assert append(L, qs=8 * 64 - 8) == INVALID
    assert append(L, qkv=None) == INVALID
    assert append(L, starts=None) == INVALID
    assert append(L, table=None) == INVALID
    assert append(L, flags=4) == INVALID
    assert append(L, qs=8 * 64 + 4) == MISALIGNED
    assert append(L, out=FAKE + 8) == MISALIGNED
    assert append(L, T=0, qkv=None) == OK


def attend(L, c=None, qp=FAKE, qs=256, out=FAKE, starts=FAKE, T=3, heads=4, scale=0.1, new=2,
           ws=FAKE, size=1 << 30, flags=0):
    c = c or cache()
    return L.qlin_cache_attention(qp, qs, out, ctypes.byref(c), starts, T, heads, scale, new, ws,
                                  size, flags, None)


def test_attention_refusals(L):
    for over, status in CACHE_FAULTS:
        assert attend(L, cache(**over)) == status, over
    assert attend(L, heads=5, qs=512) == INVALID
    assert attend(L, heads=34, qs=40 * 64) == UNSUPPORTED
    assert attend(L, scale=float("nan")) == INVALID
    assert attend(L, scale=float("inf")) == INVALID
    assert attend(L, new=-1) == INVALID
    assert attend(L, qs=248) == INVALID
    assert attend(L, T=-2) == INVALID
    assert attend(L, T=1 << 40) == UNSUPPORTED
    assert attend(L, ws=None) == INVALID
    assert attend(L, size=16) == INVALID
    assert b"workspace" in L.qlin_last_error()
    assert attend(L, out=None) == INVALID
    assert attend(L, flags=8) == INVALID
    assert attend(L, qs=260) == MISALIGNED
    assert attend(L, qp=FAKE + 8) == MISALIGNED
    assert attend(L, ws=FAKE + 8) == MISALIGNED
    assert attend(L, T=0, qp=None) == OK
    assert L.qlin_cache_attention_workspace_size(96) == 0


def test_cache_dequant_refusals(L):
    def call(c=None, ids=FAKE, n=2, out=FAKE):
        c = c or cache()
        return L.qlin_cache_dequant(ctypes.byref(c), ids, n, out, None)

    for over, status in CACHE_FAULTS:
        assert call(cache(**over)) == status, over
    assert call(n=-1) == INVALID
    assert call(ids=None) == INVALID
    assert call(out=FAKE + 8) == MISALIGNED
    assert call(n=0, out=None) == OK


def test_sample_refusals(L):
    def call(x=FAKE, xs=100, u=FAKE, tau=FAKE, k=FAKE, p=FAKE, mp=FAKE, tok=FAKE, prob=FAKE, M=2,
             V=100, dt=q.QLIN_F16, flags=0):
        return L.qlin_sample(x, xs, u, tau, k, p, mp, tok, prob, M, V, dt, flags, None)

    assert call(dt=7) == UNSUPPORTED
    assert call(V=262145, xs=300000) == UNSUPPORTED
    assert call(V=0) == INVALID
    assert call(M=-1) == INVALID
    assert call(xs=99) == INVALID
    assert call(u=None) == INVALID
    assert call(tok=None) == INVALID
    assert call(flags=2) == INVALID
    assert call(x=FAKE + 1) == MISALIGNED
    assert call(dt=q.QLIN_F32, x=FAKE + 2) == MISALIGNED
    assert call(prob=FAKE + 2) == MISALIGNED
    assert call(M=0, x=None, tok=None) == OK


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.add_rms_norm(x, torch.ones(64, dtype=torch.float16))
    with pytest.raises(ValueError):
        q.sample(torch.zeros(1, 8), *([torch.zeros(1)] * 5))
    with pytest.raises(ValueError):
        q.rope_table(8, 64, device="cpu")
    with pytest.raises(ValueError):
        q.KVCache.empty(1, 64, 1, 64, device="cpu")
