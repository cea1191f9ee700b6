"""ctypes binding of what a decode step needs beside attention and experts (the C ABI in
include/lily_decode.h): projections of a few rows by 4-bit weights, and token sampling.

Argument marshalling only, as in ``_lib``; the checks here are those the library cannot make
from addresses: that tensors live on the GPU, their element types, and that their memory reaches
as far as the call's dims do.  An int in a tensor's place is taken as an address, unchecked.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._attn import _array_at, _at, _code, _on, _reach_at, _refuse, _Struct
from ._lib import _check

# Every symbol include/lily_decode.h declares.
DECODE_EXPORTS = ("lily_decode_linear", "lily_decode_sample")


class LinearDims(_Struct):
    types = None  # torch's, of x and y (make_linear_dims)
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "K", "N", "group", "x_dtype", "out_dtype")]
                + [(n, ctypes.c_int64) for n in ("x_stride", "out_stride")])


class SampleDims(_Struct):
    type = None  # torch's, of the logits (make_sample_dims)
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "V", "logits_dtype", "reserved")]
                + [("stride", ctypes.c_int64)])


_decode = None


def _L():
    global _decode
    if _decode is None:
        L = _lib.lib()
        P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        sig = {
            "lily_decode_linear": (I, [P, P, P, P, P, P, P]),
            "lily_decode_sample": (I, [P, P, P, P, P, P, P, P, P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _decode = L
    return _decode


class W4Matrix:
    """A matrix [N][K] of 4-bit weights in the experts' format: q uint8 [N][K/2] (element 2j of a
    row in bits 0-3 of its byte j), scale and bias bf16 [N][K/group]; bias None: symmetric weights,
    scale * (q - 8).  Keeps the tensors alive."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor | None = None):
        if q.dim() != 2 or scale.dim() != 2 or q.shape[0] != scale.shape[0] or scale.shape[1] == 0:
            _refuse("4-bit matrix: q [N][K/2] and scale [N][K/group]")
        self.N, self.K = q.shape[0], 2 * q.shape[1]
        self.group = self.K // scale.shape[1]
        if self.group * scale.shape[1] != self.K:
            _refuse("4-bit matrix: the groups of scale do not divide a row")
        if bias is not None and bias.shape != scale.shape:
            _refuse("4-bit matrix: scale and bias differ in shape")
        self.q, self.scale, self.bias = q, scale, bias
        what, bf16 = "4-bit matrix", torch.bfloat16
        self._q = _array_at(what, q, torch.uint8, 0)
        self._s, self._b = _array_at(what, scale, bf16, 0), _array_at(what, bias, bf16, 0)


def _rows(t, what):
    """Elements from one row of a [rows][columns] tensor to the next."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        _refuse(f"{what}: [rows][columns] with last stride 1")
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def make_linear_dims(x, w: W4Matrix, y) -> LinearDims:
    """Dims of lily_decode_linear for x [T][K] and y [T][N]."""
    strides = _rows(x, "x"), _rows(y, "y")
    if x.shape[1] != w.K or y.shape[1] != w.N or x.shape[0] != y.shape[0]:
        _refuse(f"linear dims: x {tuple(x.shape)} by [{w.N}][{w.K}] into y {tuple(y.shape)}")
    dims = LinearDims(x.shape[0], w.K, w.N, w.group, _code(x.dtype), _code(y.dtype), *strides)
    dims.types = x.dtype, y.dtype
    return dims


def lily_decode_linear(dims: LinearDims, x, w: W4Matrix, y, stream=None):
    """y = x W^T with 4-bit weights (see the header)."""
    what = "lily_decode_linear"
    if (dims.K, dims.N, dims.group) != (w.K, w.N, w.group):
        _refuse(f"{what}: the dims are another matrix's")
    xt, yt = dims.types or (x.dtype, y.dtype)
    last = dims.T - 1
    rc = _L().lily_decode_linear(
        dims._at, _reach_at(what, x, xt, last * dims.x_stride + dims.K), w._q, w._s, w._b,
        _reach_at(what, y, yt, last * dims.out_stride + dims.N), _on(stream, x))
    if rc:
        _check(rc, what)


def make_sample_dims(logits) -> SampleDims:
    """Dims of lily_decode_sample for logits [B][V]."""
    stride = _rows(logits, "logits")
    dims = SampleDims(logits.shape[0], logits.shape[1], _code(logits.dtype), 0, stride)
    dims.type = logits.dtype
    return dims


def lily_decode_sample(dims: SampleDims, logits, temperature, top_k, top_p, min_p, u, tokens,
                       logprobs, ws, stream=None):
    """A token for each row of logits (see the header)."""
    what = "lily_decode_sample"
    f32, i32, n = torch.float32, torch.int32, dims.B
    rc = _L().lily_decode_sample(
        dims._at, _reach_at(what, logits, dims.type or logits.dtype, (n - 1) * dims.stride + dims.V),
        _array_at(what, temperature, f32, n),
        _array_at(what, top_k, i32, n), _array_at(what, top_p, f32, n),
        _array_at(what, min_p, f32, n), _array_at(what, u, f32, n),
        _array_at(what, tokens, i32, n), _array_at(what, logprobs, f32, n),
        _at(what, ws, ws.dtype), ws.numel() * ws.element_size(), _on(stream, logits))
    if rc:
        _check(rc, what)
