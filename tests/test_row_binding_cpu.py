"""What the row operators' binding refuses or passes on, seen on the CPU."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_40_gb300 as S


def test_checked_tensors_are_refused_by_place_and_type():
    x = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        S._checked(x, "workspace", torch.uint8, x.shape, 0)


@pytest.mark.parametrize("k,passed", [(0, 0), (5, 5), (100, 100), (101, 100), (2 ** 31, 100), (2 ** 32 + 5, 100), (2 ** 63, 100),
                                      (-1, -1), (-2 ** 32 + 5, -1)])
def test_counts_past_32_bits_do_not_wrap_around(k, passed):
    assert S._count(k, 100) == passed
