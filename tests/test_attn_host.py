"""The attention side of the C ABI on the host (no GPU): exports, workspace sizes, and refusals
before any launch."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import _attn

HEADER = Path(__file__).resolve().parent.parent / "include" / "lily_attn.h"
ARG, SHAPE, ALIGN, SMALL = (lily.LILY_ERR_INVALID_ARG, lily.LILY_ERR_UNSUPPORTED_SHAPE,
                            lily.LILY_ERR_MISALIGNED, lily.LILY_ERR_WORKSPACE_TOO_SMALL)
BIG = 1 << 40
P = 256  # an aligned address that no call reaches


@pytest.fixture(scope="module")
def L():
    from w4_grouped_gemm_gb300 import build
    build.build()
    return _attn._L()


def _with(s, **kw):
    c = type(s)()
    ctypes.memmove(c._at, s._at, ctypes.sizeof(s))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def no_device(rc):
    return rc in (lily.LILY_ERR_CUDA, lily.LILY_ERR_ARCH)


def test_header_functions_exported(L):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lily_attn_\w+)\s*\(", text)))
    assert names == sorted(lily.ATTN_EXPORTS)
    for n in names:
        assert hasattr(L, n)


def _norm(L, dims, x=P, res=P, w=P, res_out=P, out=P, scales=None):
    return L.lily_attn_add_rmsnorm(dims._at if dims else None, x, res, w, res_out, out,
                                   scales, None)


def test_norm_refusals(L):
    b, f = torch.bfloat16, torch.float32
    ok = lily.make_norm_dims(4, 256, b, f, f, b)
    q8 = lily.make_norm_dims(4, 256, b, f, f, torch.float8_e4m3fn, group=128)
    assert _norm(L, None) == ARG
    for name in ("x", "out"):
        assert _norm(L, ok, **{name: None}) == ARG
        assert _norm(L, ok, **{name: 24}) == ALIGN
    assert _norm(L, ok, w=8) == ALIGN
    for bad in (dict(T=0), dict(d=0), dict(x_stride=255), dict(out_stride=255),
                dict(res_stride=1), dict(res_out_stride=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x_stride=1 << 40)):
        assert _norm(L, _with(ok, **bad)) == ARG, bad
    for bad in (dict(d=16385, x_stride=20000, res_stride=20000, res_out_stride=20000,
                     out_stride=20000),
                dict(x_dtype=3), dict(res_dtype=9), dict(w_dtype=-1), dict(out_dtype=1),
                dict(group=64)):
        assert _norm(L, _with(ok, **bad)) == SHAPE, bad
    assert _norm(L, ok, scales=P) == ARG          # scales without 8 bits
    assert _norm(L, q8) == ARG                    # 8 bits without scales
    assert _norm(L, _with(q8, group=32), scales=P) == SHAPE
    assert _norm(L, _with(q8, d=192, group=128), scales=P) == SHAPE
    if not torch.cuda.is_available():
        assert no_device(_norm(L, ok)) and no_device(_norm(L, q8, scales=P))
        assert no_device(_norm(L, ok, res=None, w=None, res_out=None))


CACHE = _attn.Cache(P, P, lily.LILY_DTYPE_BF16, 10, 64, 2, 128, 64 * 256, 128, 256)
BAD_CACHES = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(n_pages=0), ARG),
              (dict(n_kv_heads=0), ARG), (dict(head_dim=0), ARG), (dict(page_stride=0), ARG),
              (dict(dtype=1), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=512), SHAPE), (dict(head_dim=100), SHAPE),
              (dict(head_dim=264), SHAPE), (dict(n_kv_heads=257), SHAPE),
              (dict(token_stride=260), SHAPE), (dict(page_stride=1 << 39), SHAPE),
              (dict(k=264), ALIGN), (dict(v=8), ALIGN)]


def _rope(L, dims, cache=CACHE, q=P, k=P, v=P, pos=P, slots=P, freq=P, qo=P, ws=P, n=256):
    return L.lily_attn_rope_append(dims._at if dims else None,
                                   cache._at if cache else None, q, k, v, pos, slots,
                                   freq, qo, ws, n, None)


def test_rope_refusals(L):
    ok = _attn.RopeDims(5, 16, 128, 0, 2048, 128, 256, 128, 256, 128, 2048, 128)
    assert _rope(L, None) == ARG and _rope(L, ok, cache=None) == ARG
    for bad, code in BAD_CACHES:
        assert _rope(L, ok, cache=_with(CACHE, **bad)) == code, bad
    for name in ("q", "k", "v", "pos", "slots", "freq", "qo", "ws"):
        assert _rope(L, ok, **{name: None}) == ARG, name
        assert _rope(L, ok, **{name: 258}) == ALIGN, name
    for name in ("q", "k", "v", "qo", "ws"):
        assert _rope(L, ok, **{name: 264}) == ALIGN, name
    assert _rope(L, ok, slots=260) == ALIGN and _rope(L, ok, freq=260) == ALIGN
    assert _rope(L, ok, q=None, qo=None) == ARG     # heads without q
    assert _rope(L, _with(ok, n_q_heads=0), q=None, qo=None, k=None, v=None) == ARG
    for bad in (dict(T=0), dict(n_q_heads=-1), dict(rotary_dim=-2)):
        assert _rope(L, _with(ok, **bad)) == ARG, bad
    for bad in (dict(rotary_dim=63), dict(rotary_dim=130), dict(style=2),
                dict(q_token_stride=2052), dict(k_head_stride=-8), dict(v_token_stride=1 << 40), dict(q_head_stride=1 << 31),
                dict(qo_head_stride=4)):
        assert _rope(L, _with(ok, **bad)) == SHAPE, bad
    assert _rope(L, ok, n=255) == SMALL
    if not torch.cuda.is_available():
        assert no_device(_rope(L, ok))
        assert no_device(_rope(L, _with(ok, n_q_heads=0), q=None, qo=None))
        assert no_device(_rope(L, ok, k=None, v=None, slots=None))
        assert no_device(_rope(L, _with(ok, rotary_dim=0), pos=None, freq=None))


ATTN = _attn.AttnDims(8, 16, 8, 1, 1000, 640, 10, 0.1, 2048, 128, 2048, 128)


def _attn_call(L, dims, cache=CACHE, q=P, pre=P, qs=P, lens=P, table=P, out=P, lse=P, ws=P, n=BIG):
    return L.lily_attn_shared_prefix(dims._at if dims else None,
                                     cache._at if cache else None, q, pre, qs, lens,
                                     table, out, lse, ws, n, None)


def test_attention_refusals(L):
    need = L.lily_attn_workspace_bytes(ATTN._at, CACHE._at)
    assert need > 256
    assert _attn_call(L, None) == ARG and _attn_call(L, ATTN, cache=None) == ARG
    assert L.lily_attn_workspace_bytes(None, CACHE._at) == 0
    for bad, code in BAD_CACHES:
        c = _with(CACHE, **bad)
        assert _attn_call(L, ATTN, cache=c) == code, bad
        assert L.lily_attn_workspace_bytes(ATTN._at, c._at) == 0
    for name in ("q", "pre", "lens", "table", "out", "ws"):
        assert _attn_call(L, ATTN, **{name: None}) == ARG, name
    for name in ("q", "pre", "qs", "lens", "table", "out", "lse", "ws"):
        assert _attn_call(L, ATTN, **{name: 258}) == ALIGN, name
    for name in ("q", "out", "ws"):
        assert _attn_call(L, ATTN, **{name: 264}) == ALIGN, name
    for bad in (dict(n_tokens=0), dict(n_q_heads=0), dict(n_seqs=0), dict(max_q_len=0),
                dict(prefix_len=-1), dict(max_seq_len=-1), dict(table_stride=-1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _attn_call(L, _with(ATTN, **bad)) == ARG, bad
    for bad in (dict(n_tokens=65537), dict(n_seqs=65537), dict(n_q_heads=15),
                dict(n_q_heads=130), dict(max_seq_len=641), dict(prefix_len=(1 << 31) - 1),
                dict(q_token_stride=2044), dict(out_head_stride=-8)):
        assert _attn_call(L, _with(ATTN, **bad)) == SHAPE, bad
    # no q_start: tokens must be n_seqs * max_q_len
    assert _attn_call(L, _with(ATTN, n_tokens=9), qs=None) == ARG
    assert _attn_call(L, ATTN, n=need - 1) == SMALL
    if not torch.cuda.is_available():
        assert no_device(_attn_call(L, ATTN, n=need))
        assert no_device(_attn_call(L, ATTN, qs=None, lse=None))
        # index arrays and lse need their own element's alignment only
        assert no_device(_attn_call(L, _with(ATTN, max_q_len=9), pre=260, qs=260, lens=260,
                                    table=260, lse=260))
        assert no_device(_attn_call(L, _with(ATTN, prefix_len=0), pre=None))
        assert no_device(_attn_call(L, _with(ATTN, max_seq_len=0), table=None))


def test_binding_refusals():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(lily.LilyError):
        lily.PagedCache(k, k, layout="dhn")
    with pytest.raises(lily.LilyError):
        lily.PagedCache(k, k.half())
    with pytest.raises(lily.LilyError):
        lily.PagedCache(k, k)                        # not on a GPU
    with pytest.raises(lily.LilyError):
        lily.make_norm_dims(1, 64, torch.float64, torch.float32, torch.float32, torch.bfloat16)
    d = lily.make_norm_dims(1, 64, torch.float32, torch.float32, torch.float32, torch.bfloat16)
    x = torch.zeros(1, 64)
    with pytest.raises(lily.LilyError):
        lily.lily_attn_add_rmsnorm(d, x, x, None, x, x.bfloat16())
    with pytest.raises(lily.LilyError):
        lily.make_rope_dims(k[0].transpose(1, 2), None, None, None, 64)
