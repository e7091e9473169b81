"""What the row operators' binding refuses or passes on, seen on the CPU."""
from __future__ import annotations

import ctypes
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


AT = 1 << 20  # never dereferenced


def filtered(dtype=0, **kw):
    a = dict(l=0, u=0, t=0, k=0, p=0, m=0, tok=0, thr=0, logp=0) | kw
    q = {n: ctypes.c_void_p(AT + off) for n, off in a.items()}
    return S.lib.spec_sample_filtered(q["l"], dtype, q["u"], q["t"], q["k"], q["p"], q["m"], 1.0, 0, 1.0, 0.0, 3, 100,
                                      q["tok"], q["thr"], q["logp"], ctypes.c_void_p(AT), 4096, None)


def top(dtype=0, **kw):
    a = dict(l=0, v=0, i=0, lse=0) | kw
    q = {n: ctypes.c_void_p(AT + off) for n, off in a.items()}
    return S.lib.spec_top_logits(q["l"], dtype, 1.0, 3, 100, 5, q["v"], q["i"], q["lse"], None)


def distill(dtype=0, **kw):
    a = dict(s=0, v=0, i=0, lse=0, g=0, loss=0, stats=0, grad=1 << 20) | kw
    q = {n: ctypes.c_void_p(AT + off) for n, off in a.items()}
    shape = (1.0, 3, 100, 5)
    return (S.lib.spec_distill_forward(q["s"], dtype, q["v"], q["i"], q["lse"], *shape, q["loss"], q["stats"], None),
            S.lib.spec_distill_backward(q["s"], dtype, q["v"], q["i"], q["lse"], q["stats"], q["g"], *shape, q["grad"], None),
            S.lib.spec_distill_loss_grad(q["s"], dtype, q["v"], q["i"], q["lse"], q["g"], *shape, q["loss"], q["stats"],
                                         q["grad"], None))


@pytest.mark.parametrize("dtype,off", [(0, 1), (0, 2), (0, 3), (1, 1)])
def test_pointers_between_elements_are_refused(dtype, off):
    assert filtered(dtype, l=off) == 1 and top(dtype, l=off) == 1 and distill(dtype, s=off) == (1, 1, 1)
    assert distill(dtype, grad=(1 << 20) + off)[1:] == (1, 1)
    for name in ("u", "t", "k", "p", "m", "tok", "thr", "logp"):
        assert filtered(dtype, **{name: off}) == 1, name
    for name in ("v", "i", "lse"):
        assert top(dtype, **{name: off}) == 1, name
        assert distill(dtype, **{name: off}) == (1, 1, 1), name
    assert distill(dtype, g=off)[1:] == (1, 1) and distill(dtype, stats=off) == (1, 1, 1) and distill(dtype, loss=off)[::2] == (1, 1)
