"""What examples/token_step.py does without the library's kernels (no GPU)."""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_a_sequence_without_a_token():
    """The sampler's -1 (a row of nothing) is no index."""
    from token_step import TokenModel
    m = TokenModel.__new__(TokenModel)
    m.embedding = torch.arange(10.0).view(5, 2)
    m.tokens = torch.tensor([3, -1, 0, 4], dtype=torch.int32)
    m.residual = torch.empty(4, 2)
    m.embed()
    assert m.residual.tolist() == [[6.0, 7.0], [0.0, 1.0], [0.0, 1.0], [8.0, 9.0]]
