"""Fused affine-dequantise-into-matmul for MLX-style packed 4/8-bit weights on
GB300 (sm_103a).

This package is a thin ctypes binding over the C ABI of ``libqlin.so``
(declared in ``include/qlin.h``): it checks tensor placement and shape,
allocates outputs with PyTorch and passes raw device pointers and the current
CUDA stream.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback -- if the library is missing the
calls raise.

Layouts (row-major): packed weights ``wq`` uint32 [N, K*bits/32] (codes low
bits first), ``scales``/``biases`` [N, K/64] in the activation dtype,
activations ``x`` [M, K], output ``y`` [M, N].

Beside the linears stand what a decoder runs between them: ``add_rms_norm``,
``rope_table`` / ``rope_append``, ``KVCache`` with ``cache_attention`` and
``cache_dequant``, and ``sample``.
"""

from __future__ import annotations

import ctypes
import os

import torch

from .build_lib import LIB_PATH

__all__ = [
    "QlinError", "lib", "quantize_affine", "dequant", "qmv", "qmm", "linear",
    "crossover_m", "device_status", "QLIN_F32", "QLIN_F16", "QLIN_BF16", "Link", "make_links",
    "chain_workspace", "qmv_chain", "KVCache", "add_rms_norm", "rope_table", "rope_append",
    "cache_dequant", "attention_workspace", "cache_attention", "sample", "KV_BLOCK",
]

QLIN_F32, QLIN_F16, QLIN_BF16 = 0, 1, 2
QLIN_OVERLAP_PREVIOUS = 1
_DTYPE_CODE = {torch.float32: QLIN_F32, torch.float16: QLIN_F16, torch.bfloat16: QLIN_BF16}
GROUP_SIZE = 64
KV_BLOCK = 64

_c_i64, _c_int, _c_vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p

# name -> (restype, argtypes); names match include/qlin.h
_SIGNATURES = {
    "qlin_status_str": (ctypes.c_char_p, [_c_int]),
    "qlin_last_error": (ctypes.c_char_p, []),
    "qlin_version": (_c_int, []),
    "qlin_quantize_affine": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_vp, _c_vp,
                                      _c_vp, _c_vp]),
    "qlin_dequant": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int,
                              _c_vp, _c_vp]),
    "qlin_qmv": (_c_int, [_c_vp] * 5 + [_c_i64] * 3 + [_c_int] * 3 + [_c_vp]),
    "qlin_qmv_ex": (_c_int, [_c_vp] * 5 + [_c_i64] * 3 + [_c_int] * 3 + [ctypes.c_uint, _c_vp]),
    "qlin_qmm": (_c_int, [_c_vp] * 5 + [_c_i64] * 3 + [_c_int] * 3 + [_c_vp]),
    "qlin_qmm_ex": (_c_int, [_c_vp] * 5 + [_c_i64] * 3 + [_c_int] * 3 + [ctypes.c_uint, _c_vp]),
    "qlin_linear": (_c_int, [_c_vp] * 5 + [_c_i64] * 3 + [_c_int] * 3 + [_c_vp]),
    "qlin_linear_ex": (_c_int, [_c_vp] * 6 + [_c_i64] * 3 + [_c_int] * 4 + [_c_vp]),
    "qlin_crossover_m": (_c_i64, [_c_i64, _c_i64, _c_int]),
    "qlin_crossover_m_dtype": (_c_i64, [_c_i64, _c_i64, _c_int, _c_int]),
    "qlin_qmv_chain_workspace_size": (ctypes.c_size_t, [_c_int]),
    "qlin_qmv_chain": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int, _c_vp,
                                ctypes.c_size_t, _c_vp]),
    "qlin_qmv_chain_static": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int, _c_vp]),
    "qlin_device_status": (_c_int, [ctypes.POINTER(_c_int)]),
    "qlin_add_rms_norm": (_c_int, [_c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64,
                                   _c_i64, ctypes.c_float, _c_int, _c_int, ctypes.c_uint, _c_vp]),
    "qlin_rope_table": (_c_int, [_c_vp, _c_i64, _c_int] + [ctypes.c_double] * 4 + [_c_vp]),
    "qlin_rope_append": (_c_int, [_c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_int, _c_int, _c_vp,
                                  _c_vp, _c_i64, _c_int, ctypes.c_uint, _c_vp]),
    "qlin_cache_dequant": (_c_int, [_c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "qlin_cache_attention_workspace_size": (ctypes.c_size_t, [_c_int]),
    "qlin_cache_attention": (_c_int, [_c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_int,
                                      ctypes.c_float, _c_int, _c_vp, ctypes.c_size_t,
                                      ctypes.c_uint, _c_vp]),
    "qlin_sample": (_c_int, [_c_vp, _c_i64] + [_c_vp] * 7 + [_c_i64, _c_i64, _c_int,
                                                             ctypes.c_uint, _c_vp]),
    # include/qlin_testing.h: failure paths and host-side choices, for the
    # library's own tests
    "qlin_testing_qmv_chain_stalled": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int,
                                                _c_vp, ctypes.c_size_t, _c_int, ctypes.c_uint,
                                                _c_vp]),
    "qlin_testing_qmv_split": (_c_int, [_c_i64, _c_i64, _c_int, _c_int]),
    "qlin_testing_sample_plan": (_c_int, [_c_i64, _c_i64, _c_int]
                                 + [ctypes.POINTER(_c_int)] * 3),
    "qlin_testing_sample_quotient": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64]),
}

_LIB = None


class Link(ctypes.Structure):
    """qlin_link: one M = 1 product of a chain (include/qlin.h)."""
    _fields_ = [("wq", _c_vp), ("scales", _c_vp), ("biases", _c_vp), ("y", _c_vp),
                ("N", _c_i64), ("K", _c_i64), ("input", ctypes.c_int32),
                ("input_offset", ctypes.c_int32)]


class QlinError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(detail)


def lib(path: str | None = None):
    """The loaded libqlin (ctypes).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        p = path or os.environ.get("QLIN_LIBRARY", LIB_PATH)
        if not os.path.exists(p):
            raise RuntimeError(
                f"libqlin.so not found at {p}; build it with "
                "`python -m int8_qmv_qmm_gb300.build_lib` (needs nvcc)")
        handle = ctypes.CDLL(p)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _LIB = handle
    return _LIB


def _check(status: int):
    if status != 0:
        L = lib()
        raise QlinError(status, f"{L.qlin_status_str(status).decode()}: "
                                f"{L.qlin_last_error().decode()}")


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(t.data_ptr() if t is not None and t.numel() else 0)


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def quantize_affine(w: torch.Tensor, bits: int, group_size: int = GROUP_SIZE,
                    sdtype: torch.dtype = torch.float16, out=None):
    """Quantise float32 W[N, K] on the GPU -> (wq, scales, biases).

    out: optional (wq, scales, biases) tensors to write into (e.g. views of
    one weight region)."""
    _need_cuda(w)
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    n, k = w.shape
    if out is not None:
        wq, sc, bi = out
        _need_cuda(wq, sc, bi)
        if (tuple(wq.shape) != (n, k * bits // 32) or tuple(sc.shape) != (n, k // group_size)
                or tuple(bi.shape) != tuple(sc.shape) or sc.dtype != sdtype
                or bi.dtype != sdtype or wq.element_size() != 4):
            raise ValueError("out tensors do not match W's shape, bits and scale dtype")
    else:
        wq = torch.empty((n, k * bits // 32), dtype=torch.int32, device=w.device)
        sc = torch.empty((n, k // group_size), dtype=sdtype, device=w.device)
        bi = torch.empty_like(sc)
    _check(lib().qlin_quantize_affine(_ptr(w), n, k, bits, group_size, _DTYPE_CODE[sdtype],
                                      _ptr(wq), _ptr(sc), _ptr(bi), _stream(w)))
    return wq, sc, bi


def dequant(wq: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, bits: int,
            group_size: int = GROUP_SIZE, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Materialise w_hat[N, K] = RNE(q*scale + bias) (unfused reference path)."""
    _need_cuda(wq, scales, biases)
    n = wq.shape[0]
    k = wq.shape[1] * 32 // bits
    out_dtype = out_dtype or scales.dtype
    out = torch.empty((n, k), dtype=out_dtype, device=wq.device)
    _check(lib().qlin_dequant(_ptr(wq), _ptr(scales), _ptr(biases), n, k, bits, group_size,
                              _DTYPE_CODE[scales.dtype], _DTYPE_CODE[out_dtype], _ptr(out),
                              _stream(wq)))
    return out


def _matmul(name: str, x, wq, scales, biases, bits, group_size, out, flags=None, extra=()):
    _need_cuda(x, wq, scales, biases)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    m, k = x.shape
    n = wq.shape[0]
    if wq.shape[1] * 32 // bits != k:
        raise ValueError("wq does not match K")
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    _need_cuda(out)
    fn = getattr(lib(), name)
    args = (() if flags is None else (flags,)) + tuple(extra)
    _check(fn(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(out), m, n, k, bits,
              group_size, _DTYPE_CODE[x.dtype], *args, _stream(x)))
    return out


def qmv(x, wq, scales, biases, bits, group_size=GROUP_SIZE, out=None, overlap_previous=False):
    """y = x . w_hat^T on CUDA cores (decode, small M).

    overlap_previous=True launches with QLIN_OVERLAP_PREVIOUS (programmatic
    dependent launch): only valid when the preceding work on the stream does
    not write wq/scales/biases."""
    if overlap_previous:
        return _matmul("qlin_qmv_ex", x, wq, scales, biases, bits, group_size, out,
                       flags=QLIN_OVERLAP_PREVIOUS)
    return _matmul("qlin_qmv", x, wq, scales, biases, bits, group_size, out)


def qmm(x, wq, scales, biases, bits, group_size=GROUP_SIZE, out=None, overlap_previous=False):
    """y = x . w_hat^T on the tcgen05 tensor cores (batched decode, prefill).

    overlap_previous=True launches with QLIN_OVERLAP_PREVIOUS (qlin_qmm_ex):
    only valid when the preceding work on the stream does not write
    wq/scales/biases."""
    if overlap_previous:
        return _matmul("qlin_qmm_ex", x, wq, scales, biases, bits, group_size, out,
                       flags=QLIN_OVERLAP_PREVIOUS)
    return _matmul("qlin_qmm", x, wq, scales, biases, bits, group_size, out)


def linear(x, wq, scales, biases, bits, group_size=GROUP_SIZE, out=None, bias=None,
           out_dtype=None):
    """qmv below the measured crossover M, qmm above it.

    bias: optional [N] tensor in the activation dtype (a linear layer's own
    bias, added before the final rounding); out_dtype: torch.float32 for a
    float32 result, else the activation dtype (qlin_linear_ex)."""
    if bias is None and (out_dtype is None or out_dtype == x.dtype):
        return _matmul("qlin_linear", x, wq, scales, biases, bits, group_size, out)
    _need_cuda(x, wq, scales, biases)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    m, k = x.shape
    n = wq.shape[0]
    if wq.shape[1] * 32 // bits != k:
        raise ValueError("wq does not match K")
    if bias is not None:
        _need_cuda(bias)
        if bias.shape != (n,) or bias.dtype != x.dtype:
            raise ValueError("bias must be [N] in the activation dtype")
    out_dtype = out_dtype or x.dtype
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
    _need_cuda(out)
    _check(lib().qlin_linear_ex(_ptr(x), _ptr(wq), _ptr(scales), _ptr(biases), _ptr(bias),
                                _ptr(out), m, n, k, bits, group_size, _DTYPE_CODE[x.dtype],
                                _DTYPE_CODE[out_dtype], _stream(x)))
    return out


def chain_workspace(n_links: int, device) -> torch.Tensor:
    """Device scratch for qmv_chain (one counter per link)."""
    nbytes = int(lib().qlin_qmv_chain_workspace_size(n_links))
    return torch.zeros(nbytes // 4, dtype=torch.int32, device=device)


def make_links(links):
    """ctypes array of Link from dicts with wq, scales, biases, y, input,
    input_offset (tensors must stay alive while the array is used)."""
    arr = (Link * len(links))()
    for i, d in enumerate(links):
        n, k = d["wq"].shape[0], None
        arr[i] = Link(d["wq"].data_ptr(), d["scales"].data_ptr(), d["biases"].data_ptr(),
                      d["y"].data_ptr(), n, d["K"], d.get("input", -1), d.get("input_offset", 0))
    return arr


def qmv_chain(x0, link_array, n_links, bits, dtype, workspace, group_size=GROUP_SIZE):
    """Run a chain of dependent M = 1 products in one launch (qlin_qmv_chain).

    x0: device tensor (or None); link_array: from make_links; workspace: from
    chain_workspace.  Outputs are written into each link's y."""
    dev = workspace.device
    _check(lib().qlin_qmv_chain(_ptr(x0) if x0 is not None else None, link_array, n_links,
                                bits, group_size, _DTYPE_CODE[dtype], _ptr(workspace),
                                workspace.numel() * 4,
                                ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)))


class _KVCacheStruct(ctypes.Structure):
    """qlin_kv_cache (include/qlin.h)."""
    _fields_ = [("pages", _c_vp), ("scales", _c_vp), ("tail", _c_vp), ("table", _c_vp),
                ("lens", _c_vp), ("n_pages", _c_i64), ("slots", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


class KVCache:
    """The 8-bit key/value cache of one layer (qlin_kv_cache in include/qlin.h):
    a handle on its tensors, which must not be moved or resized.

    pages  uint8 [n_pages, kv_heads, 2, 64*head_dim], scales float32
    [n_pages, kv_heads, 2]: complete blocks of 64 tokens; tail (the activation
    dtype) [slots, kv_heads, 2, 64*head_dim]: each slot's incomplete last block;
    table int32 [slots, max_blocks]: the page of each block; lens int32 [slots]:
    the tokens held before the call.  table and lens may be shared by the layers
    of a model; the caller fills the table and advances lens once per step, in place
    (the calls use the memory that the handle was made with, so its tensors cannot
    be replaced)."""

    _TENSORS = ("pages", "scales", "tail", "table", "lens")

    def __init__(self, pages, scales, tail, table, lens):
        _need_cuda(pages, scales, tail, table, lens)
        _need(pages.dtype == torch.uint8 and pages.dim() == 4 and pages.shape[2] == 2
              and pages.shape[3] % KV_BLOCK == 0,
              "pages must be uint8 [n_pages, kv_heads, 2, 64*head_dim]")
        n_pages, kv_heads, _, width = pages.shape
        slots = lens.numel()
        _need(scales.dtype == torch.float32 and tuple(scales.shape) == (n_pages, kv_heads, 2),
              "scales must be float32 [n_pages, kv_heads, 2]")
        _need(tail.dtype in (torch.float16, torch.bfloat16)
              and tuple(tail.shape) == (slots, kv_heads, 2, width),
              "tail must be float16 or bfloat16 [slots, kv_heads, 2, 64*head_dim]")
        _need(table.dtype == torch.int32 and table.dim() == 2 and table.shape[0] == slots,
              "table must be int32 [slots, max_blocks]")
        _need(lens.dtype == torch.int32 and lens.dim() == 1, "lens must be int32 [slots]")
        _need(len({t.device for t in (pages, scales, tail, table, lens)}) == 1,
              "the cache's tensors must be on one device")
        self.pages, self.scales, self.tail, self.table, self.lens = (pages, scales, tail, table,
                                                                     lens)
        self.kv_heads, self.head_dim, self.dtype = kv_heads, width // KV_BLOCK, tail.dtype
        self.slots, self.device, self._index = slots, pages.device, pages.get_device()
        self._struct = _KVCacheStruct(
            pages.data_ptr(), scales.data_ptr(), tail.data_ptr(), table.data_ptr(),
            lens.data_ptr(), n_pages, slots, table.shape[1], kv_heads, self.head_dim,
            _DTYPE_CODE[tail.dtype])
        self._ref = ctypes.byref(self._struct)

    def __setattr__(self, name, value):
        # (cache.lens += n assigns the tensor that it has changed in place)
        if name in self._TENSORS and getattr(self, name, value) is not value:
            raise AttributeError(f"the cache's {name} cannot be replaced: write into it "
                                 f"(cache.{name}.copy_(...)), or make another KVCache")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, slots: int, max_tokens: int, kv_heads: int, head_dim: int,
              dtype: torch.dtype = torch.float16, device="cuda", n_pages: int | None = None,
              table=None, lens=None):
        """A cache without tokens.  Without a table each slot gets pages of its
        own for max_tokens; with one (shared by a model's layers, or filled page
        by page) n_pages says how many there are."""
        blocks = (max_tokens + KV_BLOCK - 1) // KV_BLOCK
        if n_pages is None:
            n_pages = slots * blocks
        if table is None:
            table = torch.arange(slots * blocks, dtype=torch.int32,
                                 device=device).view(slots, blocks)
        if lens is None:
            lens = torch.zeros(slots, dtype=torch.int32, device=device)
        width = KV_BLOCK * head_dim
        return cls(torch.empty((n_pages, kv_heads, 2, width), dtype=torch.uint8, device=device),
                   torch.empty((n_pages, kv_heads, 2), dtype=torch.float32, device=device),
                   torch.empty((slots, kv_heads, 2, width), dtype=dtype, device=device),
                   table, lens)


# These calls run between a decoder's linears, some microseconds each, so each
# looks its arguments over in one expression and goes into what is wrong only
# where something is.
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(*checks):
    """Raises for the first check (ok, what) that does not hold."""
    for ok, what in checks:
        if not ok:
            raise ValueError(what)
    raise ValueError("tensors do not fit together")


def _row_stride(t: torch.Tensor, width: int) -> int:
    """Elements from row to row (a single row has no stride of its own)."""
    return t.stride(0) if t.shape[0] > 1 else width


def add_rms_norm(x, weight, residual=None, eps: float = 1e-5, out=None, residual_out=None,
                 overlap_previous=False):
    """h = x + residual; out = h * weight / sqrt(mean(h*h) + eps), per row.

    x [M, K] and weight [K] in the activation dtype, residual [M, K] in that or
    float32; rows may be strided.  Returns (out, residual_out), residual_out
    being h rounded to the residual's dtype (None without a residual);
    residual_out=residual updates it in place."""
    dt, rdt, shape, index = x.dtype, x.dtype, x.shape, x.get_device()
    ok = (index >= 0 and len(shape) == 2 and x.stride(1) == 1
          and (dt is torch.float16 or dt is torch.bfloat16) and weight.get_device() == index
          and weight.dtype is dt and weight.dim() == 1 and weight.is_contiguous()
          and weight.shape[0] == shape[1])
    r_ptr = ro_ptr = None
    rs = 0
    if ok and residual is not None:
        rdt = residual.dtype
        ok = (residual.get_device() == index and residual.shape == shape
              and residual.stride(1) == 1 and (rdt is dt or rdt is torch.float32))
        if ok:
            rs, r_ptr = _row_stride(residual, shape[1]), residual.data_ptr()
            if residual_out is None:
                residual_out = (torch.empty_like(residual) if residual.is_contiguous()
                                else torch.empty(shape, dtype=rdt, device=x.device))
            else:
                ok = (residual_out.get_device() == index and residual_out.is_contiguous()
                      and residual_out.shape == shape and residual_out.dtype is rdt)
            ro_ptr = residual_out.data_ptr()
    elif residual_out is not None:
        ok = False
    if ok:
        if out is None:
            out = (torch.empty_like(x) if x.is_contiguous()
                   else torch.empty(shape, dtype=dt, device=x.device))
        else:
            ok = (out.get_device() == index and out.is_contiguous() and out.shape == shape
                  and out.dtype is dt)
    if not ok:
        _refuse((x.is_cuda and x.dim() == 2 and x.stride(1) == 1,
                 "x must be a 2-D CUDA tensor with contiguous rows"),
                (dt in (torch.float16, torch.bfloat16), "x must be float16 or bfloat16"),
                (weight.device == x.device and weight.is_contiguous() and weight.dtype == dt
                 and tuple(weight.shape) == tuple(shape[1:]),
                 "weight must be [K] in x's dtype, on its device"),
                (residual is not None or residual_out is None,
                 "residual_out without a residual"),
                (residual is None or (residual.device == x.device and residual.shape == shape
                                      and residual.stride(1) == 1
                                      and residual.dtype in (dt, torch.float32)),
                 "residual must have x's device, shape and contiguous rows, in its dtype or "
                 "float32"),
                (residual_out is None or (residual_out.device == x.device
                                          and residual_out.is_contiguous()
                                          and residual_out.shape == shape
                                          and residual_out.dtype == rdt),
                 "residual_out must be contiguous, of the residual's device, shape and dtype"),
                (False, "out must be contiguous, of x's device, shape and dtype"))
    m, k = shape
    status = lib().qlin_add_rms_norm(
        x.data_ptr(), _row_stride(x, k), weight.data_ptr(), r_ptr, rs, ro_ptr, out.data_ptr(),
        m, k, eps, _DTYPE_CODE[dt], _DTYPE_CODE[rdt], 1 if overlap_previous else 0,
        _current_raw_stream(index))
    if status:
        _check(status)
    return out, residual_out


def rope_table(n_positions: int, rot_dim: int, base: float = 10000.0, factor: float = 1.0,
               short_wavelength: float = 0.0, long_wavelength: float = 0.0, device="cuda"):
    """(cos, sin) of every position and pair, float32 [n_positions, rot_dim/2, 2]
    (load time; qlin_rope_table has the scaling for long contexts)."""
    device = torch.device(device)
    _need(device.type == "cuda", "the table is made on a CUDA device")
    _need(n_positions >= 0 and rot_dim >= 2, "n_positions and rot_dim must be positive")
    table = torch.empty((n_positions, rot_dim // 2, 2), dtype=torch.float32, device=device)
    _check(lib().qlin_rope_table(table.data_ptr(), n_positions, rot_dim, base, factor,
                                 short_wavelength, long_wavelength, _stream(table)))
    return table


def rope_append(qkv, table, cache: KVCache, starts, q_heads: int, interleaved: bool = False,
                out=None, overlap_previous=False):
    """Rotates new tokens' queries and keys and appends keys and values to the cache.

    qkv [T, (q_heads + 2*kv_heads)*head_dim] (a fused linear's output; rows may
    be strided), table from rope_table (None: no rotation), starts int32
    [slots+1].  Returns the rotated queries [T, q_heads, head_dim]."""
    dt, d, shape, index = cache.dtype, cache.head_dim, qkv.shape, cache._index
    n_pos = rot = 0
    t_ptr = None
    ok = (qkv.dtype is dt and qkv.get_device() == index and len(shape) == 2
          and qkv.stride(1) == 1 and shape[1] == (q_heads + 2 * cache.kv_heads) * d
          and starts.dtype is torch.int32 and starts.get_device() == index
          and starts.is_contiguous() and starts.numel() == cache.slots + 1)
    if ok and table is not None:
        n_pos, pairs, two = table.shape if table.dim() == 3 else (0, 0, 0)
        ok = (two == 2 and table.dtype is torch.float32 and table.is_contiguous()
              and table.get_device() == index)
        rot = 2 * pairs
        t_ptr = table.data_ptr() if rot else None
    if ok:
        if out is None:
            out = torch.empty((shape[0], q_heads, d), dtype=dt, device=cache.device)
        else:
            ok = (out.is_contiguous() and out.dtype is dt and out.get_device() == index
                  and tuple(out.shape) == (shape[0], q_heads, d))
    if not ok:
        _refuse((qkv.dtype == dt and qkv.device == cache.device,
                 "qkv must have the cache's dtype and device"),
                (len(shape) == 2 and qkv.stride(1) == 1
                 and shape[1] == (q_heads + 2 * cache.kv_heads) * d,
                 "qkv must be [T, (q_heads + 2*kv_heads)*head_dim] with contiguous rows"),
                (starts.dtype == torch.int32 and starts.device == cache.device
                 and starts.is_contiguous() and starts.numel() == cache.slots + 1,
                 "starts must be int32 [slots + 1] on the cache's device"),
                (table is None or (table.dim() == 3 and table.shape[2] == 2
                                   and table.dtype == torch.float32 and table.is_contiguous()
                                   and table.device == cache.device),
                 "table must be float32 [n_positions, rot_dim/2, 2] on the cache's device"),
                (False, "out must be contiguous [T, q_heads, head_dim] in qkv's dtype"))
    status = lib().qlin_rope_append(
        qkv.data_ptr(), _row_stride(qkv, shape[1]), out.data_ptr(), t_ptr, n_pos, rot,
        1 if interleaved else 0, cache._ref, starts.data_ptr(), shape[0], q_heads,
        1 if overlap_previous else 0, _current_raw_stream(index))
    if status:
        _check(status)
    return out


def cache_dequant(cache: KVCache, page_ids, out=None):
    """The values that pages of the cache stand for, [n, kv_heads, 2, 64*head_dim]
    in the activation dtype (value blocks transposed, as in the pages)."""
    ok = (page_ids.dtype is torch.int32 and page_ids.get_device() == cache._index
          and page_ids.is_contiguous() and page_ids.dim() == 1)
    n = page_ids.numel()
    if ok:
        shape = (n, cache.kv_heads, 2, KV_BLOCK * cache.head_dim)
        if out is None:
            out = torch.empty(shape, dtype=cache.dtype, device=cache.device)
        else:
            ok = (out.is_contiguous() and out.dtype is cache.dtype
                  and out.get_device() == cache._index and tuple(out.shape) == shape)
    if not ok:
        _refuse((page_ids.dtype == torch.int32 and page_ids.device == cache.device
                 and page_ids.is_contiguous() and page_ids.dim() == 1,
                 "page_ids must be int32 [n] on the cache's device"),
                (False, "out must be contiguous, one block for each page"))
    status = lib().qlin_cache_dequant(cache._ref, page_ids.data_ptr(), n, out.data_ptr(),
                                      _current_raw_stream(cache._index))
    if status:
        _check(status)
    return out


def attention_workspace(head_dim: int, device="cuda") -> torch.Tensor:
    """Device scratch for cache_attention (calls that can overlap need one each)."""
    with torch.cuda.device(device):
        nbytes = int(lib().qlin_cache_attention_workspace_size(head_dim))
    _need(nbytes > 0, f"head_dim {head_dim} is not supported")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def cache_attention(q, cache: KVCache, starts, max_new: int, workspace, scale=None, out=None,
                    overlap_previous=False):
    """Causal attention of new tokens over the cache that already holds them.

    q [T, q_heads, head_dim] (rows may be strided), starts int32 [slots+1] as
    for rope_append, max_new: the most new tokens of any slot; workspace from
    attention_workspace; scale: 1/sqrt(head_dim) by default.  Returns
    [T, q_heads, head_dim]; rows that no slot owns are left unwritten."""
    shape, dt, index = q.shape, cache.dtype, cache._index
    ok = (len(shape) == 3 and q.dtype is dt and q.get_device() == index
          and shape[2] == cache.head_dim and q.stride(2) == 1
          and (q.stride(1) == shape[2] or shape[1] == 1)
          and starts.dtype is torch.int32 and starts.get_device() == index
          and starts.is_contiguous() and starts.numel() == cache.slots + 1
          and workspace.get_device() == index and workspace.is_contiguous())
    if ok:
        if out is None:
            out = (torch.empty_like(q) if q.is_contiguous()
                   else torch.empty(shape, dtype=dt, device=q.device))
        else:
            ok = (out.is_contiguous() and out.dtype is dt and out.get_device() == index
                  and out.shape == shape)
    if not ok:
        _refuse((q.dim() == 3 and q.dtype == dt and q.device == cache.device
                 and shape[-1] == cache.head_dim,
                 "q must be [T, q_heads, head_dim] with the cache's dtype, device and head "
                 "dimension"),
                (q.stride(-1) == 1 and (q.stride(-2) == shape[-1] or shape[-2] == 1),
                 "q's heads must be contiguous in a row"),
                (starts.dtype == torch.int32 and starts.device == cache.device
                 and starts.is_contiguous() and starts.numel() == cache.slots + 1,
                 "starts must be int32 [slots + 1] on the cache's device"),
                (workspace.device == cache.device and workspace.is_contiguous(),
                 "workspace must be contiguous on the cache's device"),
                (False, "out must be contiguous, of q's shape and dtype"))
    t, heads, d = shape
    status = lib().qlin_cache_attention(
        q.data_ptr(), _row_stride(q, heads * d), out.data_ptr(), cache._ref, starts.data_ptr(), t,
        heads, d ** -0.5 if scale is None else scale, max_new, workspace.data_ptr(),
        workspace.nbytes, 1 if overlap_previous else 0, _current_raw_stream(index))
    if status:
        _check(status)
    return out


def sample(logits, u, temperature, top_k, top_p, min_p, tokens=None, probs=None,
           overlap_previous=False):
    """One token per row of logits [M, V] (float32, float16 or bfloat16; rows may
    be strided) from given uniform numbers u [M].

    temperature, top_p, min_p float32 [M] and top_k int32 [M]; <= 0, >= 1 and
    <= 0 switch top_k, top_p and min_p off, temperature <= 0 takes the largest
    logit.  Returns (tokens int32 [M], probs float32 [M]): the share of the
    token among what the filters kept (-1 and 0 for a row without a token)."""
    shape, index = logits.shape, logits.get_device()
    m = shape[0] if len(shape) == 2 else -1

    def row_values(t, dt):
        return (t.dtype is dt and t.get_device() == index and t.is_contiguous()
                and t.numel() == m)

    f32, i32 = torch.float32, torch.int32
    ok = (logits.is_cuda and m >= 0 and logits.stride(1) == 1 and logits.dtype in _DTYPE_CODE
          and row_values(u, f32) and row_values(temperature, f32) and row_values(top_k, i32)
          and row_values(top_p, f32) and row_values(min_p, f32))
    if ok:
        if tokens is None:
            tokens = torch.empty_like(top_k)
        else:
            ok = row_values(tokens, i32)
        if probs is None:
            probs = torch.empty_like(u)
        else:
            ok = ok and row_values(probs, f32)
    if not ok:
        _refuse((logits.is_cuda and m >= 0 and logits.stride(-1) == 1,
                 "logits must be a 2-D CUDA tensor with contiguous rows"),
                (logits.dtype in _DTYPE_CODE, "logits must be float32, float16 or bfloat16"),
                *((row_values(t, dt), f"{what} must be {dt} [M] on the logits' device")
                  for t, dt, what in ((u, f32, "u"), (temperature, f32, "temperature"),
                                      (top_k, i32, "top_k"), (top_p, f32, "top_p"),
                                      (min_p, f32, "min_p"))),
                (False, "tokens must be int32 [M] and probs float32 [M] on the logits' device"))
    status = lib().qlin_sample(
        logits.data_ptr(), _row_stride(logits, shape[1]), u.data_ptr(), temperature.data_ptr(),
        top_k.data_ptr(), top_p.data_ptr(), min_p.data_ptr(), tokens.data_ptr(),
        probs.data_ptr(), m, shape[1], _DTYPE_CODE[logits.dtype], 1 if overlap_previous else 0,
        _current_raw_stream(index))
    if status:
        _check(status)
    return tokens, probs


def crossover_m(n: int, k: int, bits: int, dtype: torch.dtype = torch.float16) -> int:
    """Smallest M for which linear() takes the tensor-core kernel."""
    return int(lib().qlin_crossover_m_dtype(n, k, bits, _DTYPE_CODE[dtype]))


def device_status() -> int:
    """Reads and clears the kernels' device status word (synchronises)."""
    v = ctypes.c_int(0)
    _check(lib().qlin_device_status(ctypes.byref(v)))
    return v.value
