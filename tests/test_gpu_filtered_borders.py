"""Filtered sampling next to its borders (GPU, against 64 bits): nuclei whose end is decided by the row's tail alone,
whatever path a row takes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_filtered import S, check, filters_of, logits_of, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu
V = 262144


def near_one(base, extra, lo, hi, n=6):
    """n pairs (b, p) of float32 with p (base + e^b + extra) - 1 between lo and hi and e^b about a third."""
    found = []
    b = np.float32(-np.log(3.0))
    while len(found) < n:
        b = np.nextafter(b, np.float32(0))
        total = base + np.exp(np.float64(b)) + extra
        p = np.float32(1 / total)
        for q in (np.nextafter(p, np.float32(0)), p, np.nextafter(p, np.float32(1))):
            if lo < np.float64(q) * total - 1 < hi:
                found.append((b, q))
    return found


@pytest.mark.parametrize("copies", [1, 20, 90])  # eight to one CTA per row
@pytest.mark.parametrize("u", [0.0, 0.9])
def test_a_flat_tail_of_small_weights_counts(S, copies, u):
    # 262142 tokens of five units of 2^-45 each, all alike, so that no list holds them: 3.7e-8 in all
    d = np.float32(np.log(5 * 2.0 ** -45))
    tail = (V - 2) * np.exp(np.float64(d))
    pairs = near_one(1.0, tail, 4e-9, 2e-8)  # with the tail the nucleus passes the first token, without it it does not
    x = torch.full((len(pairs), V), float(d))
    for r, (b, _) in enumerate(pairs):
        x[r, 600], x[r, 700] = 0.0, float(b)
    R = len(pairs) * copies
    logits = x.cuda().repeat(copies, 1)
    p = np.tile([q for _, q in pairs], copies)
    uu = torch.full((R,), u, device="cuda")
    n = len(pairs)
    f = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")  # noqa: E731
    got = S.sample_filtered(logits, uu, 1.0, 0, f(p), 0.0)
    check(S, logits[-n:], uu[-n:], np.ones(n), np.zeros(n, int), p[-n:], np.zeros(n), [t[-n:] for t in got], 0)
    assert all(torch.equal(t, t[-n:].repeat(copies)) for t in got)


@pytest.mark.parametrize("copies", [1, 20, 90])
@pytest.mark.parametrize("u", [0.0, 0.9])
def test_weights_below_the_smallest_unit_do_not_count(S, copies, u):
    # 3000 tokens that the list sees a part of, the rest 40 below the largest: the exact total decides the first cut
    x = torch.full((1, V), -40.0)
    at = torch.arange(3000) * 87 + 3
    x[0, at] = torch.linspace(-14.0, -9.0, 3000)
    base = 1.0 + np.exp(x[0, at].double().numpy()).sum()
    pairs = near_one(base, 0.0, -5e-9, -2e-9)  # the first token alone is the nucleus
    x = x.repeat(len(pairs), 1)
    for r, (b, _) in enumerate(pairs):
        x[r, 600], x[r, 500] = 0.0, float(b)
    logits = x.cuda().repeat(copies, 1)
    n = len(pairs)
    p = np.tile([q for _, q in pairs], copies)
    uu = torch.full((n * copies,), u, device="cuda")
    got = S.sample_filtered(logits, uu, 1.0, 0, torch.tensor(p, device="cuda"), 0.0)
    tokens = check(S, logits[-n:], uu[-n:], np.ones(n), np.zeros(n, int), p[-n:], np.zeros(n), [t[-n:] for t in got], 0)
    assert (tokens == 600).all() and all(torch.equal(t, t[-n:].repeat(copies)) for t in got)


@pytest.mark.parametrize("R", [3, 100, 330])  # eight to one CTA per row
@pytest.mark.parametrize("mask", [-1e4, -1e9, "lowest"])
@pytest.mark.parametrize("kind", ["block", "ends", "allowed", "few", "one", "levels"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_masked_by_finite_values(S, R, mask, kind, dtype):
    # the estimate that a row is streamed with must not take the mask's distance for the spread of its logits
    n, few = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (2.5 * torch.randn(R, n, device="cuda", generator=g)).to(dtype)
    low = torch.finfo(dtype).min if mask == "lowest" else mask
    if kind == "block":
        x[:, 9000:30000] = low
    elif kind == "ends":
        x[:, :8000] = low
        x[:, -15000:] = low
    elif kind == "levels":  # masks of several depths
        x[:, 5000:9000] = -50.0
        x[:, 9000:20000] = low
        x[:, 20000:33000] -= 300.0
    else:  # so many tokens are allowed, at places of each row's own
        allowed = {"allowed": 3000, "few": 300, "one": 1}[kind]
        at = torch.rand(R, n, device="cuda", generator=g).topk(allowed, dim=1).indices
        x = torch.full_like(x, low).scatter_(1, at, x.gather(1, at))
    u = torch.rand(R, device="cuda", generator=g)
    for kinds in ("k", "p", "k_p", "m", "none", "mixed"):
        T, k, p, m = filters_of(R, 7, kinds)
        got = S.sample_filtered(x, u, *on_gpu(T, k, p, m))
        check(S, x[-few:], u[-few:], T[-few:], k[-few:], p[-few:], m[-few:], [t[-few:] for t in got])
    for k in (1, 64, 700):
        v, i, _ = S.top_logits(x, k)
        want = torch.sort(x[-few:].float(), dim=1, descending=True, stable=True)
        assert torch.equal(v[-few:], want.values[:, :k]) and torch.equal(i[-few:].long(), want.indices[:, :k])
    assert S.check_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_log_sum_exp_past_the_range_of_float32(S, dtype):
    # the largest logit over T leaves float32: the log-sum-exp is infinite with its sign, the record as ever
    x = torch.full((4, 5000), -1e30, device="cuda", dtype=dtype)
    x[0, 7] = 3e30
    x[1, 9] = -2e29
    x[2, 11] = 100.0
    x[3] = torch.finfo(dtype).min
    v, i, lse = S.top_logits(x, 1, 2.0 ** -40)
    assert v[:, 0].tolist() == x.float().amax(1).tolist() and i[:, 0].tolist() == [7, 9, 11, 0]
    assert lse.tolist() == [float("inf"), -float("inf"), 2.0 ** 40 * 100, -float("inf")]


def test_workspaces_that_are_refused(S):
    # the kernels write the error word: a workspace on the host, of another type or with gaps is refused before the launch
    x, u = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    ok = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for bad, error in ((ok.cpu(), ValueError), (ok.int(), TypeError), (ok[::2], ValueError), (ok.cpu().pin_memory(), ValueError)):
        with pytest.raises(error, match="workspace"):
            S.sample_filtered(x, u, workspace=bad)
    assert S.sample_filtered(x, u, workspace=ok, check=True)[0].tolist() == [0, 0]


def test_top_k_past_32_bits_keeps_all(S):
    x = torch.linspace(-3, 0, 5000, device="cuda").repeat(64, 1)
    u = torch.linspace(0, 0.99, 64, device="cuda")
    want = S.sample_filtered(x, u)
    for k in (5000, 2 ** 31, 2 ** 32 + 5, 2 ** 40):
        assert all(torch.equal(a, b) for a, b in zip(S.sample_filtered(x, u, 1.0, k), want))
    with pytest.raises(S.SpecVerifyError):
        S.sample_filtered(x, u, 1.0, -2 ** 32 + 5)


@pytest.mark.parametrize("R", [4, 330])
@pytest.mark.parametrize("T", [2.0 ** -64, 1e-4, 50.0, 2.0 ** 64])
@pytest.mark.parametrize("shift", [0.0, -1e6])
def test_long_rows_at_extreme_temperatures_and_far_from_zero(S, R, T, shift):
    n, few = 40000, 4
    x = logits_of(R, n, "f32", 31) + shift
    u = torch.rand(R, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    for kinds in ("k", "p", "k_p", "m", "none"):
        _, k, p, m = filters_of(R, 8, kinds)
        t = np.full(R, T)
        got = S.sample_filtered(x, u, *on_gpu(t, k, p, m))
        check(S, x[-few:], u[-few:], t[-few:], k[-few:], p[-few:], m[-few:], [y[-few:] for y in got])
    assert S.check_status() == 0


@pytest.mark.parametrize("T,d", [(0.25, 21.75), (0.5, 43.5), (1.0, 87.0), (2.0, 174.0), (0.125, 10.875)])
@pytest.mark.parametrize("n", [500, 20000])
def test_a_weight_of_the_lowest_size_is_drawn_at_zero(S, n, T, d):
    # at u = 0 the first token of any weight: e^-87 of the largest is one, the next logit below it is not
    x = torch.full((2, n), -1e3, device="cuda")
    x[:, 300], x[:, 5] = 25.0, 25.0 - d
    x[:, 3] = torch.tensor([25.0 - d * 1.000001, -1e3], device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype) if dtype == torch.float32 else x.to(dtype).index_fill(1, torch.tensor([3], device="cuda"), -1e3)
        tokens = S.sample_filtered(y, torch.zeros(2, device="cuda"), T)[0].tolist()
        assert tokens == [5, 5], (dtype, tokens)
