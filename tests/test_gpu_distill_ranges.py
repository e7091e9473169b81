"""Distillation where the sums have to reach far: masked first logits, a student that is all but certain of the
record's tokens, sharp teachers, records that hold every token of weight (GPU, against 64 bits).

Tolerances.  A log-sum-exp is within a(V) = (V/256 + 84) 2^-24 of its value (test_gpu_distill.py).  A weight of distance
x from the largest of its kind (in nats) carries x 2^-24 from the scale's rounding, its own and that of the step
between two references, the hardware exponential's 2^-22, and a factor's few roundings: rel(x) = 2 a + 6 x 2^-24 +
2^-20.  The record's probabilities are kept to 2^-38 (1 + |lse| / 8): so is r = 1 - sum p, before one rounding.  The
loss adds p (ln p - z + lse) and r (ln r - lse_rest + lse), pairs of float32 until the last rounding.  The backward
pass takes both log-sum-exps from float32: 2 steps of 2^-24 of their size more.  Weights below 2^-126 of the largest of
the pass's reference are 0, which is at least 2^-60 of what they are divided by.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import filtered_ref as F
from test_gpu_filtered import S, logits_of  # noqa: F401

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
MIN = torch.finfo(torch.float32).min


def lse64(z):
    return z.max() + np.log(np.exp(z - z.max()).sum()) if z.size and np.isfinite(z.max()) else -np.inf


def reference(s, values, ids, T, lse):
    """(loss, [lse, lse outside], gradient, r, the record's probabilities over the vocabulary) of one valid row."""
    V = s.size
    on = ids != -1
    i, v = ids[on], values[on]
    z = s / T
    outside = np.ones(V, bool)
    outside[i] = False
    total, rest = lse64(z), lse64(z[outside])
    off = lse64(v / T) if lse is None else lse
    logp = v / T - off
    pi = np.exp(logp)
    r = 0.0 if lse is None else max(0.0, 1.0 - pi.sum())
    if total - rest > 87 and r <= 2.0 ** -21 * (1 + abs(off)):
        r = 0.0  # the rounding of lse, where the student has nothing beyond the record
    some = pi > 0
    with np.errstate(divide="ignore"):
        loss = (pi[some] * (logp[some] - z[i][some] + total)).sum() + (r * (np.log(r) - rest + total) if r > 0 else 0.0)
    p = np.zeros(V)
    p[i] = pi
    grad = (pi.sum() + r) * np.exp(z - total) - p
    if r > 0 and np.isfinite(rest):
        with np.errstate(over="ignore"):
            grad -= np.where(outside, r * np.exp(z - rest), 0.0)
    return loss, np.array([total, rest]), grad / T, r, p


def check(S, student, v, i, T, lse, rows=None, stats=None):
    """The three calls on a batch, `rows` of it against the reference; returns the losses and gradients."""
    N, V = student.shape
    loss, st = S.distill_forward(student, v, i, T, teacher_lse=lse)
    grad = S.distill_backward(student, v, i, T, st if stats is None else stats, teacher_lse=lse)
    loss2, grad2 = S.distill_loss_grad(student, v, i, T, teacher_lse=lse)
    eps = torch.finfo(student.dtype).eps
    T = float(np.float32(T))
    a = (V / 256 + 84) * HALF
    for r in range(N) if rows is None else sorted(set(rows)):
        s64, i64 = F.rows64(student[r]), i[r].cpu().numpy()
        off = None if lse is None else float(lse[r])
        L, want, G, tail, p = reference(s64, F.rows64(v[r]), i64, T, off)
        z = s64 / T
        outside = np.ones(V, bool)
        outside[i64[i64 >= 0]] = False
        some = p > 0
        size = np.abs(off) if off is not None else 0.0
        r_off = 2 * HALF * tail + 2.0 ** -38 * (1 + size / 8) * 2 if tail > 0 else 0.0
        gap = want[0] - want[1] if tail > 0 else 0.0
        log_r = np.abs(np.log(tail)) if tail > 0 else 0.0
        terms = p[some] * (np.abs(np.log(p[some])) + np.abs(z[some] - want[0]))
        tl = 3 * a + 8 * HALF * terms.sum() + tail * 2 * a + r_off * (log_r + gap + 2) + 8 * HALF * tail * (log_r + gap)
        most = float(np.finfo(np.float32).max)  # beyond it a float32 is infinite
        for x in (loss[r].item(), loss2[r].item()):
            assert x == L or (L > most * (1 - HALF) and x == np.inf) or abs(x - L) <= tl + HALF * min(L, most), (r, x, L, tl)
        got = st[r].tolist()
        for x, y in zip(got, want):
            assert x == y or (y < -most and x == -np.inf) or abs(x - y) <= a + HALF * abs(y), (r, got, want)
        rel = lambda x: 2 * a + 6 * HALF * x + 2.0 ** -20  # noqa: E731
        x_in, x_out = np.abs(np.where(np.isfinite(z), z - want[0], 0)), np.abs(np.where(np.isfinite(z), z - want[1], 0))
        x_out = np.where(np.isfinite(x_out), x_out, 0.0)
        out = np.where(outside & np.isfinite(z), np.exp(np.minimum(z - want[1], 1)), 0.0) if tail > 0 else np.zeros(V)
        q = np.exp(z - want[0])
        for k, x in enumerate((grad, grad2)):
            held = 2 * HALF * np.abs(want[0 if tail == 0 or np.isinf(want[1]) else [0, 1]]).sum() if k == 0 else 0.0
            tg = (q * (p.sum() + tail) * (rel(x_in) + held) + out * (tail * (rel(x_out) + held) + r_off) + 2 * HALF * p +
                  2.0 ** -60 * (p.sum() + tail)) / T + eps / 2 * np.abs(G) + 2.0 ** -126
            d = np.abs(F.rows64(x[r]) - G) - tg * 1.01
            at = int(np.argmax(np.where(np.isnan(d), np.inf, d)))
            assert d[at] <= 0, (r, k, at, F.rows64(x[r])[at], G[at], tg[at], outside[at])
    return loss, grad, loss2, grad2


def batch(N, V, K, dtype, T, seed, sigma=2.5):
    teacher = logits_of(N, V, "f32", seed, sigma)
    student = teacher + logits_of(N, V, "f32", seed + 1, 0.7, 0.0)
    v, i = torch.topk(teacher, K, dim=1)
    lse = torch.logsumexp(teacher.double() / T, 1).float()
    return student.to(torch.bfloat16 if dtype == "bf16" else torch.float32), v.contiguous(), i.to(torch.int32), lse


ROWS = pytest.mark.parametrize("N,V", [(1, 70000), (3, 20000), (700, 20000), (340, 70001)])  # eight to one CTA per row


@pytest.mark.parametrize("T", [0.5, 1.0, 1.3])
def test_record_values_of_the_types_lowest_value(S, T):
    # a teacher whose vocabulary is masked by a finite value and whose record is longer than what is left
    student, v, i, lse = batch(4, 9000, 40, "f32", T, 60)
    v[:, 25:] = MIN
    v[3, 1:] = MIN
    for l in (lse, None):
        check(S, student, v, i, T, l)


@ROWS
@pytest.mark.parametrize("T", [0.5, 1.0, 1.3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", ["lowest", -1e30, -1e12, -1e4, -float("inf")])
def test_masked_first_logits(S, N, V, T, dtype, mask):
    student, v, i, lse = batch(N, V, 30, dtype, T, 50)
    mask = torch.finfo(student.dtype).min if mask == "lowest" else mask
    # the row's start, the start of its second half (a slice's of any number of CTAs), all but its end
    for a, b in ((0, 8192 + 100), (V // 2 - 8, V // 2 + 8200), (0, V - 300)):
        x = student.clone()
        x[:, a:b] = mask
        outside = (i < a) | (i >= b)
        ids = torch.where(outside, i, -1)   # the teacher's tokens of the masked run left out
        ids[:, 0] = torch.where(outside.any(1), ids[:, 0], V - 1)
        rows = [0, N // 2, N - 1]
        for l in (lse, None):
            check(S, x, v, ids, T, l, rows)
            if mask > -1e9:  # and left in: their logits are the masked ones
                check(S, x, v, i, T, l, rows)


@ROWS
@pytest.mark.parametrize("T", [0.25, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_student_all_but_certain_of_the_record(S, N, V, T, dtype):
    # the mass outside the record is e^-peak of the whole
    student, v, i, lse = batch(N, V, 1, dtype, T, 52)
    lse = (v[:, 0].double() / T - np.log(0.9)).float()  # the teacher's tail is 0.1
    rows = sorted({0, N - 1})
    for noise in (0.0, 1.0):
        for peak in (30, 41, 60, 80, 87, 88, 90, 95, 99, 100, 102, 105, 130, 300, 4000):
            x = student * noise
            x.scatter_(1, i.long(), float(peak) * T)
            check(S, x, v, i, T, lse, rows)
            # statistics made in 64 bits
            z = x[rows].double() / T
            out = z.scatter(1, i[rows].long(), -float("inf"))
            stats = torch.stack([torch.logsumexp(z, 1), torch.logsumexp(out, 1)], 1).float()
            pick = [t[rows].contiguous() for t in (x, v, i, lse)]
            check(S, pick[0], pick[1], pick[2], T, pick[3], None, stats)


@ROWS
def test_record_far_below_the_rest(S, N, V):
    for T, low in ((1.0, -150.0), (0.3, -500.0), (1.0, -1e6)):
        student, v, i, lse = batch(N, V, 20, "f32", T, 54)
        student.scatter_(1, i.long(), low)
        for l in (lse, None):
            check(S, student, v, i, T, l, [0, N - 1])


@ROWS
@pytest.mark.parametrize("tail", [1e-3, 1e-5, 1e-6, 3e-7])
def test_sharp_teachers_and_students_near_them(S, N, V, tail):
    # r is the small difference of 1 and the record's probabilities
    K, T = 12, 1.0
    teacher = logits_of(N, V, "f32", 56, 1.0, 0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    i = torch.rand(N, V, device="cuda", generator=g).topk(K, dim=1).indices
    rest = torch.logsumexp(teacher.scatter(1, i, -float("inf")).double(), 1)
    top = torch.randn(N, K, device="cuda", generator=g).double()
    top += (rest + np.log(1 / tail - 1) - torch.logsumexp(top, 1))[:, None]
    teacher.scatter_(1, i, top.float())
    lse = torch.logsumexp(teacher.double(), 1).float()
    v = teacher.gather(1, i).contiguous()
    # (a record's probabilities sum to 1 - tail only as far as lse is exact: another lse says another tail)
    for near in (0.0, 1e-3, 0.1):
        student = teacher + near * logits_of(N, V, "f32", 57, 1.0, 0.0)
        check(S, student, v, i.to(torch.int32), T, lse, [0, N // 2, N - 1])
