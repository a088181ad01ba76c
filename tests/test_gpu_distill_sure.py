"""lmhead_distill where the loss or its gradient is far below 1: a student that is sure of
its teacher's token, or at its teacher's distribution.

Tolerances, derived before any run (u = 2^-24, t = the logits' error as test_gpu_distill
derives it, S = 4096 the longest chain of float32 sums):
  A logit off by t moves p_n by p_n (1 - p_n) 2 t at most, so with P = min(p, 1 - p):
  p - q   P_j (4 t + S u) for a teacher's token + 2^-22 |p_j - q_j| + 2^-22 min(q, 1 - q);
          p_n (4 t + (N + S) u + c) for another, c = 2^-20 (float32) or 2^-10 (two
          roundings to binary16 of 16-bit types), and 2^-38 of the largest of them.
  dx      temperature |g| times those times |T|, + half a step.
  loss    sum |p - q| 4 t (the loss's own slope in the logits), S u of the sum's share: of
          1 - p of the teacher's likeliest token, + 2 u |loss| and 2^-50 of a difference
          of logarithms."""

import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_distill as D
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24


def reference(w, x, ids, logits, temp):
    """(loss, its tolerance, dx, its tolerance, p of the teacher's likeliest) in float64, with
    1 - p and 1 - q as sums of the others."""
    n, x6 = w.shape[0], x.double()
    l, b = x6 @ w.t() / temp, x6.abs() @ w.abs().t() / temp
    t = ((x.shape[1] + 64) * U * b + 2.0 ** -20 * b + 2 * U * l.abs()).amax(1, keepdim=True)
    at = ids.long()
    e = logits.double() / temp
    e = (e - e.amax(1, keepdim=True)).exp()
    likely = e.argmax(1, keepdim=True)
    rest_q = e.scatter(1, likely, 0.0).sum(1, keepdim=True)
    q = e / (1 + rest_q)
    star = at.gather(1, likely)
    # relative to the likeliest token's logit: its probability is 1 / (1 + others)
    d = l - l.gather(1, star)
    f = d.exp()
    others = f.scatter(1, star, 0.0).sum(1, keepdim=True)
    p = f / (1 + others)
    pj = p.gather(1, at)
    rest_p = others / (1 + others)
    full_q, diff = torch.zeros_like(l).scatter(1, at, q), None
    diff = p - full_q
    diff.scatter_(1, star, rest_q / (1 + rest_q) - rest_p)
    logq = torch.where(e > 0, e.clamp(min=1e-300).log(), 0.0) - torch.log1p(rest_q)
    logp = d.gather(1, at) - torch.log1p(others)
    loss = temp ** 2 * (q * (logq - logp)).sum(1)
    chain = 4096 * U
    tl = temp ** 2 * ((diff.abs() * 4 * t).sum(1) + chain * rest_p.squeeze(1)
                      + 2.0 ** -50 * (q * (logq.abs() + logp.abs())).sum(1)) + 2 * U * loss.abs()
    c = 2.0 ** -20 if x.dtype == F32 else 2.0 ** -10
    small = torch.minimum(p, (1 - p).clamp(min=0)).scatter(1, star, torch.minimum(p.gather(1, star), rest_p))
    qs = torch.minimum(full_q, 1 - full_q).scatter(1, star, torch.minimum(q.gather(1, likely), rest_q / (1 + rest_q)))
    mark = torch.zeros_like(l, dtype=torch.bool).scatter(1, at, True)
    err = torch.where(mark, small * (4 * t + chain) + 2.0 ** -22 * (diff.abs() + qs), p * (4 * t + (n + 4096) * U + c))
    tx = temp * (err @ w.abs() + 2.0 ** -38 * (p * ~mark).amax(1, keepdim=True) * w.abs().sum(0))
    dx = temp * diff @ w
    return loss, tl, dx, tx + D.half_step(x.dtype, dx.abs() + tx) + 1e-37, pj.gather(1, likely).squeeze(1)


def lean(w, at, margins, gen, noise=0.3):
    """Rows of x whose logit at token at[m] is some margins[m] above the others'."""
    rows = w[at]
    x = margins[:, None] * rows / (rows * rows).sum(1, keepdim=True)
    return x + noise * torch.randn(x.shape, device="cuda", generator=gen, dtype=torch.float64)


# (rows, table, columns, entries): to 64 rows straight from the table, above through unpacked codes
SHAPES = [(12, 700, 256, 1), (40, 3000, 320, 1), (90, 1200, 256, 1), (5, 131072, 512, 1), (12, 700, 256, 9),
          (64, 5000, 352, 33), (120, 2000, 256, 64), (3, 200, 20032, 5), (70, 300, 1280, 256)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k,top", SHAPES)
def test_student_sure_of_its_teachers_token(m, n, k, top, dtype):
    """Others' probabilities from 1e-2 down to 1e-17 and below: the gradient and the loss shrink
    with them, not to what is left of a rounded 1."""
    wq, w = D.table(n, k, 500 + m)
    gen = torch.Generator(device="cuda").manual_seed(m + top)
    ids = torch.stack([torch.randperm(n, device="cuda", generator=gen)[:top] for _ in range(m)]).to(torch.int32)
    margin = torch.linspace(12.0, 50.0, m, device="cuda", dtype=torch.float64)
    x = lean(w, ids[:, 0].long(), margin, gen).to(dtype)
    logits = torch.randn((m, top), device="cuda", generator=gen)
    logits[:, 0] = margin.float() + 1.0
    for temp in (1.0, 1.5):
        announce(f"lmhead_distill sure {m}x{n}x{k} top {top} {dtype} temperature {temp}")
        loss, lse, dx = q4.lmhead_distill(wq, x, ids, logits, temperature=temp, grad=True)
        torch.cuda.synchronize()
        want, tl, wx, tx, _ = reference(w, x, ids, logits, temp)
        D.assert_close(loss, want, tl, "loss")
        D.assert_close(dx, wx, tx, "dx")
    if top == 1:  # the cross entropy of the head is the same function
        l2, lse2, dx2 = q4.lmhead_xent(wq, x, ids[:, 0].contiguous(), grad=True)
        loss, lse, dx = q4.lmhead_distill(wq, x, ids, logits, grad=True)
        want, tl, wx, tx, _ = reference(w, x, ids, logits, 1.0)
        D.assert_close(loss, l2.double(), 2 * tl, "loss against the cross entropy's")
        D.assert_close(dx, dx2.double(), 2 * tx, "dx against the cross entropy's")
        assert torch.allclose(lse, lse2, rtol=2 ** -20, atol=0)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k,top", SHAPES)
def test_sure_students_loss_alone(m, n, k, top, dtype):
    wq, w = D.table(n, k, 500 + m)
    gen = torch.Generator(device="cuda").manual_seed(m + top)
    ids = torch.stack([torch.randperm(n, device="cuda", generator=gen)[:top] for _ in range(m)]).to(torch.int32)
    margin = torch.linspace(12.0, 50.0, m, device="cuda", dtype=torch.float64)
    x = lean(w, ids[:, 0].long(), margin, gen).to(dtype)
    logits = torch.randn((m, top), device="cuda", generator=gen)
    logits[:, 0] = margin.float() + 1.0
    for temp in (1.0, 1.5):
        announce(f"lmhead_distill sure, loss alone {m}x{n}x{k} top {top} {dtype} temperature {temp}")
        loss, lse, _ = q4.lmhead_distill(wq, x, ids, logits, temperature=temp)
        torch.cuda.synchronize()
        want, tl, _, _, _ = reference(w, x, ids, logits, temp)
        D.assert_close(loss, want, tl, "loss alone")


def at_teacher(m, n, k, top, temp, dtype, seed):
    """A student at its teacher: the teacher's logits are the student's best, all that matter."""
    wq, w = D.table(n, k, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((m, k), device="cuda", generator=gen) * 20).to(dtype)
    best = (x.double() @ w.t()).topk(top, 1)
    return wq, w, x, best.indices.to(torch.int32), best.values.float().contiguous()


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("m,n,k,top,temp,dtype", [(24, 256, 256, 256, 1.0, F32), (24, 200, 256, 200, 4.0, F32),
                                                  (90, 256, 512, 256, 2.0, F32), (70, 180, 96, 180, 16.0, BF16),
                                                  (7, 250, 1280, 250, 8.0, F16)])
def test_student_at_its_teacher_has_no_loss(m, n, k, top, temp, dtype, grad):
    """Every token is a teacher's, p = q up to float32's logits: the loss is of second order in
    their errors and never below 0 by more than float32 sums of the others' share."""
    wq, w, x, ids, logits = at_teacher(m, n, k, top, temp, dtype, 600 + m)
    announce(f"lmhead_distill at its teacher {m}x{n}x{k} temperature {temp} {dtype} grad {grad}")
    loss, _, _ = q4.lmhead_distill(wq, x, ids, logits, temperature=temp, grad=grad)
    torch.cuda.synchronize()
    want, tl, _, _, likely = reference(w, x, ids, logits, temp)
    D.assert_close(loss, want, tl, "loss")
    # with the gradient every term is one of the teacher's, in float64; alone, sums of a few
    # hundred float32 exponentials, each within a few u, make up 1 - p
    below = temp ** 2 * (2.0 ** -45 if grad else 8 * U * (1 - likely))
    assert (loss.double() >= -below).all(), float((loss.double() / below).min())


@pytest.mark.parametrize("temp", [2.0 ** -60, 2.0 ** -20, 1e-3, 64.0, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("m", [6, 70])
def test_any_temperature(m, temp):
    """The ends of the range, with and without the gradient (the checks of test_gpu_distill)."""
    n, k, top = 900, 96, 17
    wq, w = D.table(n, k, 700)
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), device="cuda", generator=gen) * 4
    ids, logits = D.teacher(m, n, top, 12)
    D.check(wq, w, x, ids, logits, temp)
