"""ctypes binding of the attention-side operators (the C ABI in include/lily_attn.h):
residual addition with RMSNorm, rotation and paged append, shared-prefix attention, and the
append to and attention over an 8-bit cache.

Argument marshalling only, as in ``_lib``; the checks here are those the library cannot
make from addresses: that tensors live on the GPU, their element types, that arrays given by a
pointer alone (indices, lengths, scales, lse) hold as many elements as the call's dims say, that
the heads of the tensors that dims were made from are the cache's, and, of the 8-bit cache's
operators, that q, k, v and the outputs reach as far as the dims do.  An int in a tensor's place
is taken as an address, unchecked.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import LILY_ERR_INVALID_ARG, LilyError, _check, _raw_stream, _stream

LILY_DTYPE_F16 = 2
LILY_DTYPE_E4M3 = 3
LILY_STATUS_BAD_PAGE = 0x10
LILY_STATUS_BAD_SLOT = 0x20
LILY_STATUS_BAD_LEN = 0x40
LILY_PREFIX_NONE, LILY_PREFIX_WARP, LILY_PREFIX_TENSOR = 0, 1, 2

# Every symbol include/lily_attn.h declares.
ATTN_EXPORTS = ("lily_attn_add_rmsnorm", "lily_attn_rope_append", "lily_attn_workspace_bytes",
                "lily_attn_prefix_kernel", "lily_attn_shared_prefix", "lily_attn_set_wait_ns",
                "lily_attn_rope_append8", "lily_attn_decode8_workspace_bytes", "lily_attn_decode8")

_DTYPES = {torch.bfloat16: _lib.LILY_DTYPE_BF16, torch.float32: _lib.LILY_DTYPE_F32,
           torch.float16: LILY_DTYPE_F16, torch.float8_e4m3fn: LILY_DTYPE_E4M3}


class _Struct(ctypes.Structure):
    """A struct passed by address; the address is looked up once."""

    def __init__(self, *values):
        super().__init__(*values)
        self._at = ctypes.addressof(self)


class NormDims(_Struct):
    types = None  # torch's, of x, residual, weight and out (make_norm_dims)
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "d", "x_dtype", "res_dtype", "w_dtype",
                                               "out_dtype", "group")]
                + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("x_stride", "res_stride", "res_out_stride",
                                                 "out_stride")])


class Cache(_Struct):
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]
                + [(n, ctypes.c_int32) for n in ("dtype", "n_pages", "page_size", "n_kv_heads",
                                                 "head_dim")]
                + [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")])


class Cache8(_Struct):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")]
                + [(n, ctypes.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim")]
                + [(n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride",
                                                 "scale_page_stride", "scale_head_stride",
                                                 "scale_token_stride")])


class RopeDims(_Struct):
    hkv = D = None  # heads of k and v, and their size, where known (make_rope_dims)
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "n_q_heads", "rotary_dim", "style")]
                + [(n, ctypes.c_int64) for n in (
                    "q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride",
                    "v_token_stride", "v_head_stride", "qo_token_stride", "qo_head_stride")])


class AttnDims(_Struct):
    D = None  # size of a head, where known (make_attn_dims)
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_tokens", "n_q_heads", "n_seqs", "max_q_len",
                                               "prefix_len", "max_seq_len", "table_stride")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride",
                                                 "out_token_stride", "out_head_stride")])


_attn = None


def _L():
    global _attn
    if _attn is None:
        L = _lib.lib()
        P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        # dims and cache structs go by the address that their objects keep (_at)
        sig = {
            "lily_attn_add_rmsnorm": (I, [P, P, P, P, P, P, P, P]),
            "lily_attn_rope_append": (I, [P, P, P, P, P, P, P, P, P, P, SZ, P]),
            "lily_attn_workspace_bytes": (SZ, [P, P]),
            "lily_attn_prefix_kernel": (I, [P, P]),
            "lily_attn_shared_prefix": (I, [P, P, P, P, P, P, P, P, P, P, SZ, P]),
            "lily_attn_set_wait_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
            "lily_attn_rope_append8": (I, [P, P, ctypes.c_int32, P, P, P, P, P, P, P, P, SZ, P]),
            "lily_attn_decode8_workspace_bytes": (SZ, [P, P]),
            "lily_attn_decode8": (I, [P, P, ctypes.c_int32, P, P, P, P, P, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _attn = L
    return _attn


def _refuse(what):
    raise LilyError(LILY_ERR_INVALID_ARG, what)


def _at(what, t, dtype):
    """Address of a GPU tensor of this type; an address as it is; None stays."""
    if t is None or t.__class__ is int:
        return t
    if t.is_cuda and t.dtype is dtype:
        return t.data_ptr()
    _not_taken(what, t, dtype, 0)


def _array_at(what, t, dtype, n):
    """The same of an array given by its pointer alone: contiguous, n elements or more."""
    if t is None or t.__class__ is int:
        return t
    if t.is_cuda and t.dtype is dtype and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    _not_taken(what, t, dtype, n)


def _reach_at(what, t, dtype, n):
    """Address of a GPU tensor of this type whose memory goes on for n elements or more from its
    first one, whatever its strides; an address as it is; None stays."""
    if t is None or t.__class__ is int:
        return t
    if t.is_cuda and t.dtype is dtype and ((t.numel() >= n and t.is_contiguous()) or _reach(t) >= n):
        return t.data_ptr()
    _not_taken(what, t, dtype, n, strided=True)


def _reach(t):
    return t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()


def _not_taken(what, t, dtype, n, strided=False):
    if not t.is_cuda:
        _refuse(f"{what}: a tensor is not on the GPU")
    if t.dtype is not dtype:
        _refuse(f"{what}: a tensor of {t.dtype} where {dtype} belongs")
    if strided:
        _refuse(f"{what}: a tensor ends before the {n} elements that the dims reach over")
    _refuse(f"{what}: an array must be contiguous, of {n} elements or more")


def _alike(what, a, b):
    """Two [tokens][heads][D] tensors (or None) have the same heads."""
    if a is not None and b is not None and a.shape[1:] != b.shape[1:]:
        _refuse(f"{what}: heads of {tuple(a.shape[1:])} and {tuple(b.shape[1:])}")


def _on(stream, tensor):
    """A stream's handle; by default the current stream of the tensor's device."""
    if stream is None and _raw_stream is not None and tensor.__class__ is not int:
        return _raw_stream(tensor.get_device())
    return _stream(stream)


def _code(dtype) -> int:
    if dtype not in _DTYPES:
        _refuse(f"element type {dtype}")
    return _DTYPES[dtype]


class PagedCache:
    """Views of a K and a V tensor as a paged cache: [page][token][head][D] (layout "nhd")
    or [page][head][token][D] ("hnd"), of any page, token and head strides that both share.
    Keeps the tensors alive; .c is the ctypes struct."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, layout: str = "nhd"):
        if layout not in ("nhd", "hnd"):
            _refuse("cache layout")
        if (k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype
                or k.stride(3) != 1):
            _refuse("cache: k and v must be 4-D, alike in shape, strides and type, last stride 1")
        _at("cache", k, k.dtype)
        _at("cache", v, k.dtype)
        token, head = (1, 2) if layout == "nhd" else (2, 1)
        self.k, self.v, self.layout = k, v, layout
        self.dtype, self.page, self.heads, self.D = k.dtype, k.shape[token], k.shape[head], k.shape[3]

        def stride(dim):  # a dimension of size 1 has no step; any valid one serves
            return k.stride(dim) if k.shape[dim] > 1 else max(8, (k.shape[3] + 7) // 8 * 8)

        self.c = Cache(k.data_ptr(), v.data_ptr(), _code(k.dtype), k.shape[0], k.shape[token],
                       k.shape[head], k.shape[3], stride(0), stride(head), stride(token))


class PagedCache8:
    """Views of K and V codes (float8_e4m3fn, 4-D as PagedCache's) and their scales (fp32, the same
    without the last dimension) as an 8-bit paged cache.  Keeps the tensors alive; .c is the
    ctypes struct."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, layout: str = "nhd"):
        if layout not in ("nhd", "hnd"):
            _refuse("cache layout")
        if (k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1):
            _refuse("8-bit cache: k and v must be 4-D, alike in shape and strides, last stride 1")
        if (k_scales.shape != k.shape[:3] or v_scales.shape != k.shape[:3]
                or k_scales.stride() != v_scales.stride()):
            _refuse("8-bit cache: scales must have the pages' shape without the last dimension, "
                    "alike in strides")
        for t, dt in ((k, torch.float8_e4m3fn), (v, torch.float8_e4m3fn),
                      (k_scales, torch.float32), (v_scales, torch.float32)):
            _at("8-bit cache", t, dt)
        token, head = (1, 2) if layout == "nhd" else (2, 1)
        self.k, self.v, self.k_scales, self.v_scales, self.layout = k, v, k_scales, v_scales, layout
        self.page, self.heads, self.D = k.shape[token], k.shape[head], k.shape[3]

        def stride(t, dim, least):  # a dimension of size 1 has no step; any valid one serves
            return t.stride(dim) if t.shape[dim] > 1 else least

        row = (self.D + 15) // 16 * 16
        self.c = Cache8(k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                        k.shape[0], self.page, self.heads, self.D,
                        *(stride(k, dim, row) for dim in (0, head, token)),
                        *(stride(k_scales, dim, 1) for dim in (0, head, token)))


def make_norm_dims(T, d, x_dtype, res_dtype, w_dtype, out_dtype, group=0, eps=1e-6, x_stride=None,
                   res_stride=None, res_out_stride=None, out_stride=None) -> NormDims:
    """Dims of lily_attn_add_rmsnorm; types are torch's, strides default to d."""
    dims = NormDims(T, d, _code(x_dtype), _code(res_dtype), _code(w_dtype), _code(out_dtype),
                    group, eps, *(d if s is None else s
                                  for s in (x_stride, res_stride, res_out_stride, out_stride)))
    dims.types = x_dtype, res_dtype, w_dtype, out_dtype
    return dims


def _norm_types(d):
    """dims.types of dims that were not made by make_norm_dims."""
    return tuple(next((t for t, c in _DTYPES.items() if c == code), None)
                 for code in (d.x_dtype, d.res_dtype, d.w_dtype, d.out_dtype))


def lily_attn_add_rmsnorm(dims: NormDims, x, residual, weight, residual_out, out, scales=None,
                          stream=None):
    """residual_out = x + residual; out = its RMSNorm (see the header)."""
    what = "lily_attn_add_rmsnorm"
    xt, rt, wt, ot = dims.types or _norm_types(dims)
    n_scales = 0
    if scales is not None:
        group = dims.group
        n_scales = dims.T * (dims.d // group) if group else dims.T
    rc = _L().lily_attn_add_rmsnorm(
        dims._at, _at(what, x, xt), _at(what, residual, rt), _at(what, weight, wt),
        _at(what, residual_out, rt), _at(what, out, ot),
        _array_at(what, scales, torch.float32, n_scales), _on(stream, x))
    if rc:
        _check(rc, what)


def _strides(t, what):
    """(token, head) strides of a [tokens][heads][D] tensor, or zeros for None."""
    if t is None:
        return 0, 0
    if t.dim() != 3 or t.stride(2) != 1:
        _refuse(f"{what}: [tokens][heads][D] with last stride 1")
    return (t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2],
            t.stride(1) if t.shape[1] > 1 else t.shape[2])


def make_rope_dims(q, k, v, q_out, rotary_dim, style=0) -> RopeDims:
    """Dims of lily_attn_rope_append from its [T][heads][D] tensors (q and q_out, or k and v,
    may be None)."""
    some = q if q is not None else k
    if some is None:
        _refuse("rope dims: neither q nor k")
    strides = (*_strides(q, "q"), *_strides(k, "k"), *_strides(v, "v"), *_strides(q_out, "q_out"))
    _alike("rope dims", q, q_out)
    _alike("rope dims", k, v)
    if q is not None and k is not None and q.shape[2] != k.shape[2]:
        _refuse("rope dims: heads of q and k differ in size")
    dims = RopeDims(some.shape[0], q.shape[1] if q is not None else 0, rotary_dim, style, *strides)
    dims.hkv, dims.D = k.shape[1] if k is not None else None, some.shape[2]
    return dims


def lily_attn_rope_append(dims: RopeDims, cache: PagedCache, q, k, v, positions, slots, inv_freq,
                          q_out, ws, stream=None):
    """Rotate q into q_out and k, append k and v at `slots` (see the header)."""
    what = "lily_attn_rope_append"
    dt, T = cache.dtype, dims.T
    if dims.D is not None and (dims.D != cache.D or dims.hkv not in (None, cache.heads)):
        _refuse(f"{what}: the dims' heads are not the cache's")
    rc = _L().lily_attn_rope_append(
        dims._at, cache.c._at, _at(what, q, dt), _at(what, k, dt), _at(what, v, dt),
        _array_at(what, positions, torch.int32, T), _array_at(what, slots, torch.int64, T),
        _array_at(what, inv_freq, torch.float64, dims.rotary_dim // 2), _at(what, q_out, dt),
        _at(what, ws, ws.dtype), ws.numel(), _on(stream, ws))
    if rc:
        _check(rc, what)


def make_attn_dims(q, out, n_seqs, max_q_len, prefix_len, max_seq_len, table_stride,
                   scale) -> AttnDims:
    """Dims of lily_attn_shared_prefix for [tokens][heads][D] tensors q and out."""
    strides = (*_strides(q, "q"), *_strides(out, "out"))
    _alike("attention dims", q, out)
    dims = AttnDims(q.shape[0], q.shape[1], n_seqs, max_q_len, prefix_len, max_seq_len,
                    table_stride, scale, *strides)
    dims.D = q.shape[2]
    return dims


def lily_attn_workspace_bytes(dims: AttnDims, cache: PagedCache) -> int:
    return int(_L().lily_attn_workspace_bytes(dims._at, cache.c._at))


def lily_attn_prefix_kernel(dims: AttnDims, cache: PagedCache) -> int:
    """Which kernel reads the shared prefix: LILY_PREFIX_NONE, _WARP or _TENSOR."""
    rc = _L().lily_attn_prefix_kernel(dims._at, cache.c._at)
    if rc < 0:
        _check(rc, "lily_attn_prefix_kernel")
    return rc


def lily_attn_shared_prefix(dims: AttnDims, cache: PagedCache, q, prefix_pages, q_start, seq_lens,
                            block_table, out, lse, ws, stream=None):
    """Attention over the shared prefix and each sequence's own pages (see the header)."""
    what = "lily_attn_shared_prefix"
    dt, i32, n = cache.dtype, torch.int32, dims.n_seqs
    if dims.D is not None and dims.D != cache.D:
        _refuse(f"{what}: the dims' heads are not the cache's")
    rc = _L().lily_attn_shared_prefix(
        dims._at, cache.c._at, _at(what, q, dt),
        _array_at(what, prefix_pages, i32, -(-dims.prefix_len // cache.page)),
        _array_at(what, q_start, i32, n + 1), _array_at(what, seq_lens, i32, n),
        _array_at(what, block_table, i32, n * dims.table_stride), _at(what, out, dt),
        _array_at(what, lse, torch.float32, dims.n_tokens * dims.n_q_heads),
        _at(what, ws, ws.dtype), ws.numel(), _on(stream, q))
    if rc:
        _check(rc, what)


def _step_type(what, *tensors):
    """The 16-bit type of the first of a call's tensors (None and addresses aside), which the
    others are held to."""
    for t in tensors:
        if t is not None and t.__class__ is not int:
            if t.dtype is torch.bfloat16 or t.dtype is torch.float16:
                return t.dtype
            _refuse(f"{what}: tensors of one 16-bit type belong here, not {t.dtype}")
    _refuse(f"{what}: tensors of one 16-bit type belong here")


def lily_attn_rope_append8(dims: RopeDims, cache: PagedCache8, q, k, v, positions, slots, inv_freq,
                           q_out, ws, stream=None):
    """Rotate q into q_out and k, append k and v as 8-bit codes at `slots` (see the header)."""
    what = "lily_attn_rope_append8"
    dt, T = _step_type(what, q, k, v, q_out), dims.T
    if dims.D is not None and (dims.D != cache.D or dims.hkv not in (None, cache.heads)):
        _refuse(f"{what}: the dims' heads are not the cache's")
    last, hq, hkv, D = T - 1, dims.n_q_heads - 1, cache.heads - 1, cache.D
    rc = _L().lily_attn_rope_append8(
        dims._at, cache.c._at, _DTYPES[dt],
        _reach_at(what, q, dt, last * dims.q_token_stride + hq * dims.q_head_stride + D),
        _reach_at(what, k, dt, last * dims.k_token_stride + hkv * dims.k_head_stride + D),
        _reach_at(what, v, dt, last * dims.v_token_stride + hkv * dims.v_head_stride + D),
        _array_at(what, positions, torch.int32, T), _array_at(what, slots, torch.int64, T),
        _array_at(what, inv_freq, torch.float64, dims.rotary_dim // 2),
        _reach_at(what, q_out, dt, last * dims.qo_token_stride + hq * dims.qo_head_stride + D),
        _at(what, ws, ws.dtype), ws.numel() * ws.element_size(), _on(stream, ws))
    if rc:
        _check(rc, what)


def lily_attn_decode8_workspace_bytes(dims: AttnDims, cache: PagedCache8) -> int:
    return int(_L().lily_attn_decode8_workspace_bytes(dims._at, cache.c._at))


def lily_attn_decode8(dims: AttnDims, cache: PagedCache8, q, q_start, seq_lens, block_table, out,
                      lse, ws, stream=None):
    """Attention of new tokens over an 8-bit paged cache (see the header); dims as
    make_attn_dims makes them, with prefix_len 0."""
    what = "lily_attn_decode8"
    dt, i32, n = _step_type(what, q, out), torch.int32, dims.n_seqs
    if dims.D is not None and dims.D != cache.D:
        _refuse(f"{what}: the dims' heads are not the cache's")
    last, heads, D = dims.n_tokens - 1, dims.n_q_heads - 1, cache.D
    rc = _L().lily_attn_decode8(
        dims._at, cache.c._at, _DTYPES[dt],
        _reach_at(what, q, dt, last * dims.q_token_stride + heads * dims.q_head_stride + D),
        _array_at(what, q_start, i32, n + 1), _array_at(what, seq_lens, i32, n),
        _array_at(what, block_table, i32, n * dims.table_stride),
        _reach_at(what, out, dt, last * dims.out_token_stride + heads * dims.out_head_stride + D),
        _array_at(what, lse, torch.float32, dims.n_tokens * dims.n_q_heads),
        _at(what, ws, ws.dtype), ws.numel() * ws.element_size(), _on(stream, q))
    if rc:
        _check(rc, what)


def lily_attn_set_wait_ns(ns: int) -> int:
    """Give-up limit of the waits inside lily_attn_shared_prefix's and lily_attn_decode8's
    kernels; returns the previous limit (nanoseconds)."""
    return int(_L().lily_attn_set_wait_ns(int(ns)))
