"""More of the attention side on the host (no GPU): settings, plans, and the binding's checks."""

import pytest
import torch

import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import _attn


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
