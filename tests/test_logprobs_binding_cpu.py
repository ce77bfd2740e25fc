"""Refusals of the log probabilities' binding that no kernel's call reaches."""
import os

import pytest
import torch

from ternary_packed_weight_amd import build


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def test_negative_top(tq2):
    x, t = torch.zeros((3, 100)), torch.zeros(3, dtype=torch.int64)
    for kw in ({}, {"top_tokens": torch.zeros((3, 1), dtype=torch.int64), "top_logprobs": torch.zeros((3, 1))}):
        with pytest.raises(ValueError, match="top must not be negative, got -1"):
            tq2.tq2_token_logprobs(x, t, top=-1, **kw)
