"""lily_decode_sample where top_k and top_p both cut among more than 256 tokens, near each other: the run that top_p
ends may share its last logits with the one that top_k ends."""
import numpy as np
import pytest
import torch

from test_gpu_decode_sample import BF, F16, F32, check, random

pytestmark = pytest.mark.gpu
U = [0.05, 0.5, 0.95, 0.999]


def _check(row, t, k, p, u=U):
    """One row with several u, a row each in one call, and alone: few rows and many take clusters of other sizes."""
    check(row[None].repeat(len(u), 1), [t] * len(u), [k] * len(u), [p] * len(u), None, u)
    check(row[None], [t], [k], [p], None, u[-1:])


# (rows found by emulating both searches on the host: 295 tokens were kept of 300, 487 of 500)
@pytest.mark.parametrize("V,seed,t,k", [(50021, 13, 1.0, 300), (131072, 25, 2.0, 500)])
def test_found_rows(V, seed, t, k):
    row = torch.from_numpy(2 * np.random.RandomState(seed).randn(V)).float()
    _check(row, t, k, 0.999)


def test_equal_steps():
    """Two values: the 1000 first hold 1000 equal logits, 990 of which are kept (of 897 by mistake, 852 was drawn)."""
    row = torch.full((16384,), -1.0)
    row[::8] = 0.0
    _check(row, 1.0, 1000, 0.99)


@pytest.mark.parametrize("k", [257, 300, 1000, 3000, 8000])
@pytest.mark.parametrize("p", [0.99, 0.995, 0.999, 0.9999])
def test_near_cuts(k, p):
    """Flat and steep rows, rows of few values, and one that is mostly masked."""
    V = 20021
    l, gen = random(5, V, F32, k + int(p * 1e4))
    for row, t in ((l[0], 1.0), (l[1], 3.0), (l[2].to(BF), 2.0), ((2 * l[3]).round().to(F16) / 2, 8.0)):
        _check(row, t, k, p, U[1:])
    masked = torch.where(torch.rand(V, generator=gen) < 0.5, -float("inf"), l[4])
    _check(masked, 1.5, k, p, U[2:])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_near_cuts_in_a_batch(dtype):
    """Each row its own k and p; more rows than clusters at once."""
    B, V = 200, 4099
    l, gen = random(B, V, dtype, 77, 1.0)
    k = [257 + (37 * b) % 3000 for b in range(B)]
    p = [(0.9, 0.99, 0.995, 0.999, 0.9999)[b % 5] for b in range(B)]
    check(l, [0.5 + b % 4 for b in range(B)], k, p, [0.0 if b % 3 else 0.001 for b in range(B)],
          torch.rand(B, generator=gen))
