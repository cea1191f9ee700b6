"""The bindings of the decode step's operators refuse tensors whose memory ends before the call's dims do (no GPU: the
tensors only say that they are on one, and the library's functions only tell that they were called)."""
import pytest
import torch

import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import _attn, _decode

P = 1 << 20  # an address
BF = torch.bfloat16


class OnGpu:
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def called(monkeypatch):
    names = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: names.append(name) or 0
    monkeypatch.setattr(_attn, "_L", Lib)
    monkeypatch.setattr(_decode, "_L", Lib)
    return names


def tries(called, call, fits, short):
    """`call` takes each of `fits` and refuses each of `short`."""
    for t in fits:
        call(t)
        assert called
        called.clear()
    for t in short:
        with pytest.raises(lily.LilyError):
            call(t)
        assert not called


def gpu(*shape, dtype=BF):
    return OnGpu(torch.zeros(shape, dtype=dtype))


def test_linear(called):
    w = lily.W4Matrix.__new__(lily.W4Matrix)
    w.N, w.K, w.group, w._q, w._s, w._b = 40, 128, 64, P, P, None
    x, y = torch.zeros(6, 136, dtype=BF)[:, :128], torch.zeros(6, 48)[:, :40]
    dims = lily.make_linear_dims(x, w, y)
    assert (dims.x_stride, dims.out_stride) == (136, 48)
    tries(called, lambda t: lily.lily_decode_linear(dims, t, w, P, stream=0),
          [OnGpu(x), gpu(6, 136), gpu(1, 5 * 136 + 128), OnGpu(torch.zeros(7, 136, dtype=BF)[1:, :128])],
          [OnGpu(x[:5].clone()), gpu(5, 136), gpu(6, 128), OnGpu(torch.zeros(6, 136, dtype=BF)[1:, :128]),
           OnGpu(torch.zeros(1, 128, dtype=BF).expand(8, 128)), gpu(6, 136, dtype=torch.float16)])
    tries(called, lambda t: lily.lily_decode_linear(dims, P, w, t, stream=0),
          [OnGpu(y), gpu(5 * 48 + 40, dtype=torch.float32)], [gpu(6, 40, dtype=torch.float32), gpu(5, 48, dtype=torch.float32)])


def test_sample(called):
    dims = lily.make_sample_dims(torch.zeros(3, 50)[:, :41])
    ws = gpu(256, dtype=torch.uint8)
    tries(called, lambda t: lily.lily_decode_sample(dims, t, P, P, P, P, P, P, P, ws, stream=0),
          [OnGpu(torch.zeros(3, 50)[:, :41]), gpu(141, dtype=torch.float32)],
          [gpu(140, dtype=torch.float32), gpu(2, 50, dtype=torch.float32), OnGpu(torch.zeros(3, 50)[:, 10:])])


def _cache8(heads, D):
    c = lily.PagedCache8.__new__(lily.PagedCache8)
    c.heads, c.D, c.page, c.c = heads, D, 16, _attn.Cache8()
    return c


def test_append8(called):
    qkv = torch.zeros(4, 8 * 64, dtype=BF)
    q, k, v = (t.view(4, -1, 64) for t in qkv.split([256, 128, 128], 1))
    out = torch.zeros(4, 4, 64, dtype=BF)
    dims, cache, ws = lily.make_rope_dims(q, k, v, out, 64), _cache8(2, 64), gpu(256, dtype=torch.uint8)
    fewer = torch.zeros(3, 512, dtype=BF)

    def call(**other):
        a = {n: OnGpu(t) for n, t in (("q", q), ("k", k), ("v", v), ("out", out))} | other
        lily.lily_attn_rope_append8(dims, cache, a["q"], a["k"], a["v"], P, P, P, a["out"], ws, stream=0)
    for name, cols in (("q", slice(0, 256)), ("k", slice(256, 384)), ("v", slice(384, 512))):
        tries(called, lambda t: call(**{name: t}), [OnGpu(qkv[:, cols].view(4, -1, 64))],
              [OnGpu(fewer[:, cols].view(3, -1, 64)), OnGpu(qkv[:, cols].reshape(4, -1, 64).clone())])
    tries(called, lambda t: call(out=t), [gpu(4, 4, 64), gpu(5, 4, 64)], [gpu(3, 4, 64), gpu(4, 3, 64)])


def test_decode8(called):
    q = torch.zeros(5, 4, 64, dtype=BF)
    dims = lily.make_attn_dims(q, torch.zeros(5, 6, 64, dtype=BF)[:, :4], 5, 1, 0, 32, 2, 0.1)
    cache, ws = _cache8(2, 64), gpu(256, dtype=torch.uint8)
    out = OnGpu(torch.zeros(5, 6, 64, dtype=BF)[:, :4])
    tries(called, lambda t: lily.lily_attn_decode8(dims, cache, t, P, P, P, out, P, ws, stream=0), [OnGpu(q)],
          [gpu(4, 4, 64), gpu(5, 3, 64)])
    tries(called, lambda t: lily.lily_attn_decode8(dims, cache, OnGpu(q), P, P, P, t, P, ws, stream=0), [out],
          [gpu(5, 4, 64), gpu(4, 6, 64)])
