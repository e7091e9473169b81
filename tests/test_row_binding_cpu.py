"""What the row operators' binding refuses or passes on, seen on the CPU: the library's functions are stood in for by
one that notes its arguments."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_40_gb300 as S


def test_checked_tensors_are_refused_by_place_and_type():
    x = torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        S._checked(x, "workspace", torch.uint8, x.shape, 0)
