"""What the row operators' binding refuses or passes on, seen on the CPU."""
from __future__ import annotations

import gc

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


def test_an_outgrown_workspace_stays_allocated():
    # a graph captured with it still writes its error word there
    device = torch.device("cpu", 0)
    first = S.workspace_for(device, 4096)
    at = first.data_ptr()
    del first
    grown = S.workspace_for(device, 1 << 16)
    gc.collect()
    assert grown.numel() == 1 << 16 and grown.data_ptr() != at
    assert any(w.data_ptr() == at for w in S._WS_OUTGROWN)
    assert S.workspace_for(device, 100) is grown
