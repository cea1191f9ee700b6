"""More of the attention side on the host (no GPU): settings, plans, and the binding's checks."""

import ctypes
import os
import random
import subprocess
import sys
from pathlib import Path
from types import SimpleNamespace

import pytest
import torch

import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import _attn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def L():
    from w4_grouped_gemm_gb300 import build
    build.build()
    return _attn._L()


def test_wait_limit_setter_returns_previous(L):
    """2 s by default; host state only."""
    prev = lily.lily_attn_set_wait_ns(12345)
    try:
        assert prev == 2_000_000_000
        assert lily.lily_attn_set_wait_ns(0) == 12345
    finally:
        assert lily.lily_attn_set_wait_ns(prev) == 0


# ------------------------------------------------------------------------------------ the binding's checks
B, H, F, Q = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


class OnGpu:
    """A CPU tensor that says it lives on a GPU: what the binding's checks see.  A call that passes
    them goes on to the library, which finds no device here (or is not made where there is one)."""
    is_cuda = True

    def __init__(self, *shape, dtype=B):
        self.t = torch.zeros(shape, dtype=dtype)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return 1 << 20


def _refused(f, *args):
    with pytest.raises(lily.LilyError) as e:
        f(*args)
    assert e.value.code == lily.LILY_ERR_INVALID_ARG, e.value


def _passes(f, *args):
    """The checks let it through (the library then has no device)."""
    if torch.cuda.is_available():
        return
    with pytest.raises(lily.LilyError) as e:
        f(*args)
    assert e.value.code in (lily.LILY_ERR_CUDA, lily.LILY_ERR_ARCH), e.value


def _swaps(f, args, swaps):
    """args are taken; args with any one of `swaps` (place: others in its place) are refused."""
    _passes(f, *args)
    for i, others in swaps.items():
        for other in others:
            _refused(f, *args[:i], other, *args[i + 1:])


def test_norm_binding_checks_types(L):
    T, d = 3, 256
    dims = lily.make_norm_dims(T, d, B, F, H, Q, group=128)
    x, r, w = OnGpu(T, d), OnGpu(T, d, dtype=F), OnGpu(d, dtype=H)
    out, scales = OnGpu(T, d, dtype=Q), OnGpu(T, 2, dtype=F)

    def call(*a):
        lily.lily_attn_add_rmsnorm(dims, *a, stream=0)
    args = (x, r, w, r, out, scales)
    _swaps(call, args, {
        0: [OnGpu(T, d, dtype=H), OnGpu(T, d, dtype=F), torch.zeros(T, d, dtype=B)],
        1: [x], 2: [OnGpu(d, dtype=F)], 3: [x], 4: [x, OnGpu(T, d, dtype=torch.uint8)],
        5: [OnGpu(T, 2), OnGpu(T, 1, dtype=F)]})
    # dims that were filled by hand are checked alike
    made = dims
    dims = _attn.NormDims(T, d, 0, 1, 2, 3, 128, 1e-6, d, d, d, d)
    _swaps(call, args, {0: [OnGpu(T, d, dtype=F)], 5: [OnGpu(T, 2)]})
    # the number of rows may change between calls
    dims = made
    dims.T = T + 1
    _refused(call, *args)
    dims.T = T - 1
    _passes(call, *args)
    dims = lily.make_norm_dims(T, d, B, F, F, B)
    _passes(call, x, None, None, None, x, None)


def _cache(dtype=B, heads=2, D=64, pages=6, page=16):
    return lily.PagedCache(OnGpu(pages, page, heads, D, dtype=dtype), OnGpu(pages, page, heads, D, dtype=dtype))


def test_rope_binding_checks_types_and_sizes(L):
    T = 5
    i32, i64, f64 = torch.int32, torch.int64, torch.float64
    q, k, v, qo = OnGpu(T, 4, 64), OnGpu(T, 2, 64), OnGpu(T, 2, 64), OnGpu(T, 4, 64)
    pos, slots, freq = OnGpu(T, dtype=i32), OnGpu(T, dtype=i64), OnGpu(32, dtype=f64)
    ws = OnGpu(256, dtype=torch.uint8)
    dims, cache = lily.make_rope_dims(q, k, v, qo, 64), _cache()

    def call(*a):
        lily.lily_attn_rope_append(dims, cache, *a, ws, stream=0)
    _swaps(call, (q, k, v, pos, slots, freq, qo), {
        0: [OnGpu(T, 4, 64, dtype=H)], 1: [OnGpu(T, 2, 64, dtype=F)], 2: [OnGpu(T, 2, 64, dtype=H)],
        3: [OnGpu(T, dtype=i64), OnGpu(T - 1, dtype=i32)], 4: [OnGpu(T, dtype=i32), OnGpu(T - 1, dtype=i64)],
        5: [OnGpu(32, dtype=F), OnGpu(31, dtype=f64)], 6: [OnGpu(T, 4, 64, dtype=H)]})


def test_attention_binding_checks_types_and_sizes(L):
    T, hq, D, seqs = 6, 4, 64, 3
    i32 = torch.int32
    q, out, lse = OnGpu(T, hq, D), OnGpu(T, hq, D), OnGpu(T, hq, dtype=F)
    pre, starts, lens, table = (OnGpu(n, dtype=i32) for n in (2, seqs + 1, seqs, seqs * 4))
    cache = _cache()
    dims = lily.make_attn_dims(q, out, seqs, 2, 20, 64, 4, 0.1)
    ws = OnGpu(max(16, lily.lily_attn_workspace_bytes(dims, cache)), dtype=torch.uint8)

    def call(*a):
        lily.lily_attn_shared_prefix(dims, cache, *a, ws, stream=0)
    _swaps(call, (q, pre, starts, lens, table, out, lse), {
        0: [OnGpu(T, hq, D, dtype=H)],
        1: [OnGpu(1, dtype=i32), OnGpu(2, dtype=torch.int64)],
        2: [OnGpu(seqs, dtype=i32)], 3: [OnGpu(seqs - 1, dtype=i32), OnGpu(seqs, dtype=F)],
        4: [OnGpu(seqs * 4 - 1, dtype=i32)], 5: [OnGpu(T, hq, D, dtype=F)],
        6: [OnGpu(T, hq), OnGpu(T, hq - 1, dtype=F)]})
    _passes(call, q, pre, None, lens, table, out, None)
    _passes(call, 4096, 4096, 4096, 4096, 4096, 4096, 4096)     # addresses are taken as they are


def test_dims_and_cache_have_the_same_heads(L):
    T, ws = 5, OnGpu(1 << 20, dtype=torch.uint8)
    x = {h: OnGpu(T, h, 64) for h in (1, 2, 4)}
    wide = OnGpu(T, 2, 128)
    _refused(lily.make_rope_dims, x[4], x[2], x[1], x[4], 64)     # k and v
    _refused(lily.make_rope_dims, x[4], x[2], x[2], x[2], 64)     # q and q_out
    _refused(lily.make_rope_dims, x[2], wide, wide, x[2], 64)     # q and k
    _refused(lily.make_attn_dims, x[4], x[2], 5, 1, 0, 16, 1, 0.1)
    i32, i64, f64 = torch.int32, torch.int64, torch.float64
    pos, slots, freq = OnGpu(T, dtype=i32), OnGpu(T, dtype=i64), OnGpu(32, dtype=f64)
    table = OnGpu(T, dtype=i32)
    for cache, q, k, good in ((_cache(), x[4], x[2], True), (_cache(), x[4], None, True),
                              (_cache(), None, x[2], True), (_cache(), x[4], x[1], False),
                              (_cache(D=128), x[4], x[2], False), (_cache(D=128), x[4], None, False)):
        dims = lily.make_rope_dims(q, k, k, q, 64)
        args = (dims, cache, q, k, k, pos, slots if k is not None else None, freq, q, ws, 0)
        (_passes if good else _refused)(lily.lily_attn_rope_append, *args)
    for cache, good in ((_cache(), True), (_cache(D=128), False)):
        dims = lily.make_attn_dims(x[4], x[4], T, 1, 0, 16, 1, 0.1)
        (_passes if good else _refused)(lily.lily_attn_shared_prefix, dims, cache, x[4], None, None, table,
                                        table, x[4], None, ws, 0)


# ------------------------------------------------------------------------------------ the example
@pytest.mark.parametrize("own", [20, 32, 33])
def test_example_tokens_past_a_sequences_room(own):
    """Slots of a decoder block's next tokens up to, at and past the room of their sequences: the last
    page is not passed (an index past the table would be a fault on the GPU)."""
    from decoder_block import DecoderBlock
    page, q_len, prefix = 16, 3, 40
    width = -(-own // page)
    b = SimpleNamespace(q_len=q_len, page=page, own=own, prefix=prefix,
                        table=torch.arange(5, 5 + 2 * width, dtype=torch.int32).view(2, width))
    for have in (0, own - 4, own - 3, own - 1, own, own + 1, own + 100):
        lens = torch.tensor([have, 0], dtype=torch.int32)
        slots, positions = DecoderBlock.slots_of(b, lens)
        for j in range(q_len):
            at = have + j
            want = int(b.table[0, at // page]) * page + at % page if at < own else -1
            assert int(slots[j]) == want and int(positions[j]) == prefix + at
            assert int(slots[q_len + j]) == int(b.table[1, 0]) * page + j


# ------------------------------------------------------------------------------------ the prefix's kernel
def test_kernel_of_the_prefix(L):
    """Few rows or few tiles of 64 rows and keys stay on mma.sync, many go to the tensor cores (256
    tiles, 512 for heads over 128)."""
    def kernel(tokens, hq, hkv, prefix, D):
        q = OnGpu(tokens, hq, D)
        dims = lily.make_attn_dims(q, q, tokens, 1, prefix, 16, 1, 0.1)
        return lily.lily_attn_prefix_kernel(dims, _cache(heads=hkv, D=D))
    none, warp, tensor = lily.LILY_PREFIX_NONE, lily.LILY_PREFIX_WARP, lily.LILY_PREFIX_TENSOR
    for D, tiles in ((64, 256), (128, 256), (136, 512), (256, 512)):
        assert kernel(8, 8, 1, 0, D) == none
        assert kernel(8, 8, 1, 1 << 20, D) == warp             # 64 rows
        assert kernel(65, 1, 1, 64 * (tiles // 2 - 1), D) == warp
        assert kernel(65, 1, 1, 64 * (tiles // 2 - 1) + 1, D) == tensor
        assert kernel(33, 8, 4, 64 * (tiles // 8 - 1), D) == warp       # 4 heads of 66 rows
        assert kernel(33, 8, 4, 64 * tiles // 8, D) == tensor
    q = OnGpu(4, 4, 64)
    _refused(lily.lily_attn_prefix_kernel, lily.make_attn_dims(q, q, 0, 1, 9, 16, 1, 0.1), _cache())


# ------------------------------------------------------------------------------------ places on the GPU
@pytest.fixture(scope="module")
def share(tmp_path_factory):
    """share_grid of the library's sources, compiled for the host: (CTAs of the prefix, of the own pages)."""
    at = tmp_path_factory.mktemp("share")
    csrc = Path(lily.__file__).resolve().parent / "csrc"
    (at / "s.cpp").write_text('#include "attn_share.h"\nextern "C" void share(int cap, int64_t A, int64_t B, '
                              'int wide, int* g) { lily::share_grid(cap, A, B, wide, g[0], g[1]); }\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{csrc}", str(at / "s.cpp"), "-o",
                    str(at / "s.so")], check=True)
    f = ctypes.CDLL(str(at / "s.so")).share
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]

    def call(cap, A, B, wide):
        g = (ctypes.c_int * 2)()
        f(cap, A, B, wide, g)
        return g[0], g[1]
    return call


def _up(n, by):
    return -(-n // by)


def test_places_are_shared_for_any_length_within_the_bound(share):
    """Whatever part b of its bound B the own pages use, the division is no slower than the two sets one
    after the other, in tiles: w per prefix tile, and three more for the second wave of CTAs."""
    rng = random.Random(1)
    split = 0
    for _ in range(20000):
        cap, wide = rng.choice([152, 304]), rng.random() < 0.5
        A, B = (int(2 ** rng.uniform(0, 18)) for _ in range(2))
        w = 2 if wide else 1
        ga, gb = share(cap, A, B, wide)
        a0, b0 = min(A, cap), min(B, cap)
        assert 1 <= ga <= a0 and 1 <= gb <= b0
        if (ga, gb) == (a0, b0):
            continue
        split += 1
        assert ga + gb <= cap
        for b in {0, 1, B // 100, B // 10, B // 3, B // 2, B - 1, B}:
            assert max(w * _up(A, ga), _up(b, gb)) <= w * _up(A, a0) + _up(b, b0) + 4, (cap, A, B, wide, b)
    assert split > 2000


def test_places_of_tight_and_loose_bounds(share):
    assert share(152, 4096, 40, True) == (147, 5)              # few own keys beside a long prefix
    assert share(304, 128, 896, True) == (128, 176)            # short runs beside a short prefix
    ga, _ = share(152, 4096, 8192, True)                       # room for as many own tiles as the prefix's
    assert ga >= 144
    ga, _ = share(304, 128, 65536, True)
    assert ga >= 64
    assert share(304, 0, 500, True) == (0, 304) and share(304, 500, 0, False) == (304, 0)
    assert share(304, 100, 200, True) == (100, 200)
