"""Distillation where the sums have to reach far: masked first logits, a student that is all but certain of the
record's tokens, sharp teachers, records that hold every token of weight (GPU, against 64 bits).

Tolerances.  A log-sum-exp is within a(V) = (V/256 + 84) 2^-24 of its value (test_gpu_distill.py).  A weight of distance
x from the largest of its kind (in nats) carries x 2^-24 from the scale's rounding, its own and that of the step
between two references, the hardware exponential's 2^-22, and a factor's few roundings: rel(x) = 2 a + 6 x 2^-24 +
2^-20.  The record's probabilities are kept to 2^-38 (1 + |lse| / 8): so is r = 1 - sum p, before one rounding; in a
gradient p / T is within 2^-23 of p for expf (documented: one step), and three times 2^-24 (p's own rest, 1 / T, the product).  The
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


def softmax64(s, T):
    """(largest, ln of the sum relative to it, softmax) of logits; -inf, -inf and zeros if there is none."""
    top = s.max() if s.size else -np.inf
    if not np.isfinite(top):
        return -np.inf, -np.inf, np.zeros(s.size)
    e = np.exp((s - top) / T)  # (relative to the largest first: masks of 3e38 leave nothing of the rest in 64 bits)
    return top, np.log(e.sum()), e / e.sum()


def reference(s, values, ids, T, lse):
    """One valid row: loss, [lse, lse outside], gradient, r, and by token the record's probabilities, q, the shares of
    the mass outside the record, and -ln of the last two."""
    V = s.size
    on = ids != -1
    i, v = ids[on], values[on]
    outside = np.ones(V, bool)
    outside[i] = False
    top, total, q = softmax64(s, T)
    top_out, rest, share = softmax64(s[outside], T)
    if lse is None:
        top_v, off, pi = softmax64(v, T)
        logp, r = (v - top_v) / T - off, 0.0
    else:
        logp = v / T - lse
        pi = np.exp(logp)
        r = max(0.0, 1.0 - pi.sum())
    gap = (top - top_out) / T + total - rest if np.isfinite(top_out) else np.inf
    if gap > 60 and r <= 2.0 ** -21 * (1 + abs(lse or 0.0)):
        r = 0.0  # the rounding of lse, where the student has nothing beyond the record
    some = pi > 0
    far = total - (s - top) / T
    p, out, far_out = np.zeros(V), np.zeros(V), np.zeros(V)
    p[i] = pi
    out[outside] = share
    if np.isfinite(top_out):
        far_out[outside] = rest - (s[outside] - top_out) / T
    loss = (pi[some] * (logp[some] + far[i][some])).sum() + (r * (np.log(r) + gap) if r > 0 else 0.0)
    grad = ((pi.sum() + r) * q - p - r * out) / T
    stats = np.array([top / T + total, top_out / T + rest if np.isfinite(top_out) else -np.inf])
    return dict(loss=loss, stats=stats, grad=grad, r=r, p=p, q=q, out=out, far=far, far_out=far_out, gap=gap)


def check(S, student, v, i, T, lse, rows=None, stats=None):
    """The three calls on a batch, `rows` of it against the reference; returns the losses and gradients."""
    N, V = student.shape
    loss, st = S.distill_forward(student, v, i, T, teacher_lse=lse)
    grad = S.distill_backward(student, v, i, T, st if stats is None else stats, teacher_lse=lse)
    loss2, grad2 = S.distill_loss_grad(student, v, i, T, teacher_lse=lse)
    eps = torch.finfo(student.dtype).eps
    T = float(np.float32(T))
    a = (V / 256 + 84) * HALF
    most = float(np.finfo(np.float32).max)  # beyond it a float32 is infinite
    for n in range(N) if rows is None else sorted(set(rows)):
        off = None if lse is None else float(lse[n])
        w = reference(F.rows64(student[n]), F.rows64(v[n]), i[n].cpu().numpy(), T, off)
        L, G, r, p, far = w["loss"], w["grad"], w["r"], w["p"], w["far"]
        gap, log_r, r_off = 0.0, 0.0, 0.0
        if r > 0:
            gap, log_r = w["gap"], abs(np.log(r))
            r_off = 2 * HALF * r + 2.0 ** -37 * (1 + abs(off) / 8)
        some = p > 0
        terms = (p[some] * (np.abs(np.log(p[some])) + np.abs(far[some]))).sum()
        tl = 3 * a + 8 * HALF * terms + r * 2 * a + r_off * (log_r + gap + 2) + 8 * HALF * r * (log_r + gap)
        for x in (loss[n].item(), loss2[n].item()):
            assert x == L or (L > 1e38 and x == np.inf) or abs(x - L) <= tl + HALF * min(L, most), (n, x, L, tl)
        got = st[n].tolist()
        for x, y in zip(got, w["stats"]):
            nothing = y < -most or (r == 0 and w["gap"] > 60 and y == w["stats"][1])
            assert x == y or (nothing and x == -np.inf) or abs(x - y) <= a + HALF * abs(y), (n, got, w["stats"])
        rel = lambda x: 2 * a + 6 * HALF * np.where(np.isfinite(x), np.abs(x), 0.0) + 2.0 ** -20  # noqa: E731
        for k, x in enumerate((grad, grad2)):
            held = 2 * HALF * np.abs(w["stats"][0 if r == 0 or np.isinf(gap) else [0, 1]]).sum() if k == 0 else 0.0
            tg = (w["q"] * (p.sum() + r) * (rel(far) + held) + w["out"] * (r * (rel(w["far_out"]) + held) + r_off) +
                  5 * HALF * p + 2.0 ** -60 * (p.sum() + r)) / T + eps / 2 * np.abs(G) + 2.0 ** -126
            y = F.rows64(x[n])
            if k == 0 and abs(w["stats"][0]) >= 2.0 ** 22:  # float32 statistics that tell no weights
                assert np.isnan(y).all()
                continue
            if k == 0 and w["stats"][1] <= -2.0 ** 22:  # nor those outside the record
                y = y - r * w["out"] / T
            d = np.abs(y - G) - tg * 1.01
            at = int(np.argmax(np.where(np.isnan(d), np.inf, d)))
            assert d[at] <= 0, (n, k, at, y[at], G[at], tg[at])
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
@pytest.mark.parametrize("T", [0.7, 1.0, 1.3, 8.0, 2.0 ** 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_student_masked_by_its_types_lowest_value(S, N, V, T, dtype):
    # everywhere but at the record's tokens, which lie in the first half of the row
    student, v, i, lse = batch(N, V // 2, 20, dtype, T, 62)
    low = torch.finfo(student.dtype).min
    x = torch.full((N, V), low, device="cuda", dtype=student.dtype)
    x.scatter_(1, i.long(), student.gather(1, i.long()))
    for l in (None, lse):
        check(S, x, v, i, T, l, [0, N // 2, N - 1])
    x.fill_(low)  # all of them alike
    if T >= 1:
        check(S, x, v, i, T, None, [0, N - 1])
    else:  # 3.4e38 / 0.7 is no float32: the statistics are infinite
        loss, stats = S.distill_forward(x, v, i, T)
        assert torch.isfinite(loss).all() and (stats == -float("inf")).all()
        assert torch.isnan(S.distill_backward(x, v, i, T, stats)).all()
        assert torch.isfinite(S.distill_loss_grad(x, v, i, T)[1]).all()


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


@ROWS
@pytest.mark.parametrize("T", [0.7, 1.0])
@pytest.mark.parametrize("mask", [-float("inf"), MIN, -1e5])
def test_records_that_hold_every_token_of_weight(S, N, V, T, mask):
    # both models masked alike: at most K tokens are allowed
    K, allowed = 64, 40
    g = torch.Generator(device="cuda").manual_seed(2)
    i = torch.rand(N, V, device="cuda", generator=g).topk(K, dim=1).indices
    teacher = torch.full((N, V), mask, device="cuda")
    student = torch.full((N, V), mask, device="cuda")
    teacher.scatter_(1, i[:, :allowed], 3 * torch.randn(N, allowed, device="cuda", generator=g) + 10)
    student.scatter_(1, i[:, :allowed], 3 * torch.randn(N, allowed, device="cuda", generator=g))
    values, ids, lse = S.top_logits(teacher, K, T)
    for l in (lse, None):
        for made in (values, values.masked_fill(ids < 0, float("nan"))):
            out = check(S, student, made, ids, T, l, [0, N // 2, N - 1])
            assert all(torch.isfinite(t).all() for t in out) and out[0].abs().max() < 100
    # a teacher that gives real weight to what its student excludes: +inf where it is -inf
    other = (lse.double() + 0.01).float()
    loss = S.distill_forward(student, values, ids, T, teacher_lse=other)[0]
    assert (loss > 1).all() and (mask > -float("inf") or torch.isinf(loss).all())


@pytest.mark.parametrize("V", [1, 7, 300, 1000])
def test_records_of_the_whole_vocabulary(S, V):
    N = 64
    teacher, student = logits_of(N, V, "f32", 58), logits_of(N, V, "f32", 59)
    values, ids, lse = S.top_logits(teacher, V)
    out = check(S, student, values, ids, 1.0, lse)
    assert all(torch.isfinite(t).all() for t in out)


@pytest.mark.parametrize("T", [2.0 ** -64, 1e-6, 0.01, 100.0, 1e6, 2.0 ** 64])
@pytest.mark.parametrize("N,V", [(2, 40000), (400, 9001)])
def test_temperatures_at_their_ends(S, N, V, T):
    student, v, i, lse = batch(N, V, 25, "f32", T, 64)
    for l in (lse, None) if T >= 0.01 else (None,):  # (a float32 lse of 1e6 and more says nothing of p)
        check(S, student, v, i, T, l, [0, N - 1])
    # logits of the temperature's own size
    if 1e-6 <= T <= 1e6:
        check(S, student * T, v * T, i, T, (lse.double() * 0 + torch.logsumexp(v.double(), 1) + 0.1).float(), [0, N - 1])


@pytest.mark.parametrize("N,V", [(2, 40000), (400, 9001)])
@pytest.mark.parametrize("shift", [-3e4, 1e5, -1e6])
def test_logits_far_from_zero(S, N, V, shift):
    # a softmax does not see what its logits have in common (bfloat16 has no room for it)
    student, v, i, lse = batch(N, V, 25, "f32", 1.0, 66)
    for l in (lse, None):
        check(S, student + shift, v, i, 1.0, l, [0, N - 1])


@pytest.mark.parametrize("V", [1, 2, 3, 5, 9, 17, 1402])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0.0, 2992.0, -1e4])
def test_rows_whose_weight_lies_in_their_ends(S, V, dtype, shift):
    # the logits outside a row's 16-byte aligned body: a short row's all, a rising row's largest
    N = 40
    g = torch.Generator(device="cuda").manual_seed(V)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    for T in (1.0, 0.3):
        x = torch.sort(3 * torch.randn(N, V, device="cuda", generator=g), dim=1).values + shift
        buf = torch.empty(N * V + 3, device="cuda", dtype=t)
        for at in (0, 1, 3):  # (the ends differ from row to row where V is odd)
            student = buf[at:at + N * V].view(N, V).copy_(x)
            values, ids, lse = S.top_logits(2 * torch.randn(N, V, device="cuda", generator=g), 1, T)
            check(S, student, values, ids, T, None)
            check(S, student, values, ids, T, lse + 0.2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_that_only_the_first_reference_hides(S, dtype):
    # rows without a finite first load go by 0, far above their logits
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.tensor([[-7.0, -22.0, -40.0], [-100.0, -101.0, -115.0], [-4.0, -25.0, -25.0]], device="cuda", dtype=t)
    long = torch.full((3, 20000), -float("inf"), device="cuda", dtype=t)
    long[:, -300:] = x.repeat(1, 100)
    for s in (x, long):
        i = s.float().argmax(1, keepdim=True).to(torch.int32)
        v = s.float().gather(1, i.long())
        for T in (0.25, 0.5, 1.0):
            check(S, s, v, i, T, None)
            check(S, s, v, i, T, (v[:, 0].double() / T + 0.01).float())
            check(S, s, v, i, T, (v[:, 0] / T).clone())


@ROWS
@pytest.mark.parametrize("T", [0.01, 0.25, 0.7, 1.0])
def test_next_to_no_mass_on_a_masked_token(S, N, V, T):
    # p of e^-60 to e^-85 on tokens that the student masks by the type's lowest value: p times 3.4e38 / T is what counts
    student, v, i, _ = batch(N, V, 8, "f32", T, 68)
    v = (torch.tensor([0.0, -0.1, -0.5, -60.0, -70.0, -80.0, -84.0, -85.0], device="cuda") * T).repeat(N, 1)
    lse = torch.logsumexp(v.double() / T, 1).float()
    for first in (3, 5, 7):
        x = student.clone().scatter_(1, i[:, first:].long(), MIN)
        for l in (lse, None):
            check(S, x, v, i, T, l, [0, N - 1])
