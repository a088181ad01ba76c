"""Distillation of a teacher's best logits through the Q4_0 head (lmhead_distill)
against a float64 form on the oracle's decoded weights.

Tolerances, derived before any run (u = 2^-24, half a float32 step; B = sum |x w|):
  logits  t = ((K + 64) u B + 2^-20 B) / temperature, + 2 u |l| for the temperature.
          A shift of the logits by at most t moves lse by max t and log p by 2 max t.
  lse     max t + S u, S = 4096 the longest chain of a piece's sums, + 4 u |lse|.
  loss    temperature^2 sum q (2 max t + S u + 8 u (|log q| + |l| + |lse|)).
  dx      temperature |g| (sum_n p |T_n| (4 max t + (N + S) u + c)
          + sum_j (p_j + q_j) |T_j| (4 max t + S u + 2^-20)
          + 2^-38 max_n p sum_n |T_n|), n over the other tokens, j over the teacher's;
          c = 2^-20 for float32, 2^-10 where probabilities and weights are rounded to
          binary16 (16-bit types); + half a step."""

import numpy as np
import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu
from oracle import q4_oracle as O
from q4_quantized_speech_amd import synth

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24
INF = float("inf")


def table(n, k, seed, ramp=False):
    """(bytes on the GPU, float64 weights on the GPU)."""
    w = synth.weights(n, k, seed)
    if ramp:  # later rows larger: the running maximum grows from piece to piece
        w *= np.linspace(0.2, 4.0, n, dtype=np.float32)[:, None]
    qb = O.quantize_q4_0(w)
    return torch.from_numpy(qb).cuda(), torch.from_numpy(O.dequantize_q4_0(qb, n, k)).double().cuda()


def half_step(dtype, want):
    f = torch.finfo(dtype)
    return f.eps / 2 * want.abs() * (1 + 2.0 ** -10) + f.tiny * f.eps


def assert_close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(0.0).max()))


def teacher(m, n, top, seed, ragged=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(n, generator=g)[:top] if n <= 200000 and top <= n else
                       torch.randint(0, n, (top,), generator=g) for _ in range(m)]).to(torch.int32)
    logits = 3 * torch.randn((m, top), generator=g)
    if ragged and m > 2:
        ids[0] = -1                      # no teacher
        ids[1, top // 2:] = n            # outside the table
        ids[2, :top // 3] = -100
    return ids.cuda(), logits.cuda()


def reference(w, x, ids, logits, temp, dloss):
    n = w.shape[0]
    x6 = x.double()
    l, b = x6 @ w.t() / temp, x6.abs() @ w.abs().t() / temp
    t = ((x.shape[1] + 64) * U * b + 2.0 ** -20 * b + 2 * U * l.abs()).amax(1, keepdim=True)
    lse = torch.logsumexp(l, 1, keepdim=True)
    here = (ids >= 0) & (ids < n)
    at = torch.where(here, ids, 0).long()
    b = torch.where(here, logits.double() / temp, -INF)
    used = (b > -INF).any(1)
    q = torch.softmax(torch.where(used[:, None], b, 0.0), 1) * (here & used[:, None])
    # entries of one token add up
    full = torch.zeros_like(l).scatter_add_(1, at, q)
    mark = torch.zeros_like(l).scatter_add_(1, at, (here & used[:, None]).double()) > 0
    logq = torch.where(full > 0, full.log(), 0.0)
    p = (l - lse).exp()
    loss = temp ** 2 * (full * torch.where(full > 0, logq - (l - lse), 0.0)).sum(1)
    chain = 4096 * U
    tl = temp ** 2 * (full * (2 * t + chain + 8 * U * (logq.abs() + l.abs() + lse.abs()))).sum(1)
    g = temp * (dloss.double() if dloss is not None else 1.0) * used
    dx = ((p - full) * g.reshape(-1, 1)) @ w
    c = 2.0 ** -20 if x.dtype == F32 else 2.0 ** -10
    rest = p * ~mark
    tol = (rest @ w.abs()) * (4 * t + (n + 4096) * U + c)
    tol += ((p + full) * mark) @ w.abs() * (4 * t + chain + 2.0 ** -20)
    tol += 2.0 ** -38 * rest.amax(1, keepdim=True) * w.abs().sum(0)
    tol = tol * g.reshape(-1, 1).abs()
    return (lse.squeeze(1), (t + chain + 4 * U * lse.abs()).squeeze(1), loss, tl + 4 * U * loss.abs() + 1e-30, dx,
            tol + half_step(x.dtype, dx.abs() + tol) + 1e-30)


def check(wq, w, x, ids, logits, temp, dloss=None):
    announce(f"lmhead_distill {tuple(x.shape)} of {w.shape[0]} top {ids.shape[1]} {x.dtype} temperature {temp}")
    loss, lse, dx = q4.lmhead_distill(wq, x, ids, logits, temperature=temp, grad=True, dloss=dloss)
    torch.cuda.synchronize()
    rl, tl, rs, ts, rx, tx = reference(w, x, ids, logits, temp, dloss)
    assert_close(lse, rl, tl, "lse")
    assert_close(loss, rs, ts, "loss")
    assert_close(dx, rx, tx, "dx")
    loss2, lse2, none = q4.lmhead_distill(wq, x, ids, logits, temperature=temp)
    torch.cuda.synchronize()
    assert none is None
    assert_close(lse2, rl, tl, "lse alone")
    assert_close(loss2, rs, ts, "loss alone")
    again = q4.lmhead_distill(wq, x, ids, logits, temperature=temp, grad=True, dloss=dloss)
    assert torch.equal(again[2], dx) and torch.equal(again[0], loss)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k,top", [(1, 1, 32, 1), (1, 100, 64, 3), (3, 65, 96, 64), (4, 1000, 128, 7),
                                       (16, 333, 160, 256), (17, 2000, 1280, 16), (64, 500, 96, 33),
                                       (65, 1031, 64, 64), (130, 64, 320, 5), (200, 5000, 256, 32)])
def test_shapes(m, n, k, top, dtype):
    wq, w = table(n, k, 100 + m)
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = (torch.randn((m, k), device="cuda", generator=gen) * 4).to(dtype)
    ids, logits = teacher(m, n, top, 7 + m)
    dloss = torch.rand(m, device="cuda", generator=gen)
    check(wq, w, x, ids, logits, 1.0 if m % 2 else 2.5, dloss)


@pytest.mark.parametrize("m,n,k,top,dtype", [(8, 131072, 1280, 16, F32), (375, 32768, 1280, 32, F32),
                                             (96, 70001, 512, 64, BF16), (40, 66000, 96, 8, F16)])
def test_pieces(m, n, k, top, dtype):
    """Several pieces of the vocabulary, later ones with the larger logits."""
    wq, w = table(n, k, 300 + m, ramp=True)
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), device="cuda", generator=gen).to(dtype)
    ids, logits = teacher(m, n, top, 9 + m)
    check(wq, w, x, ids, logits, 1.5)


def test_student_at_its_teacher():
    """p - q nearly cancels: the teacher's logits are the student's own, of all the tokens
    that matter.  The gradient is what is left, to the precision of the difference."""
    n, k, m = 300, 256, 24
    wq, w = table(n, k, 400)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((m, k), device="cuda", generator=gen) * 20
    l = x.double() @ w.t()
    best = l.topk(200, 1)
    check(wq, w, x, best.indices.to(torch.int32), best.values.float().contiguous(), 1.0)


def test_teacher_holds_the_whole_table():
    """Every column is a teacher's: nothing is left of the sum over the others."""
    n, k, m = 96, 64, 70
    wq, w = table(n, k, 410)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for rows in (m, 20):
        x = torch.randn((rows, k), device="cuda", generator=gen) * 8
        ids = torch.arange(n, dtype=torch.int32, device="cuda").repeat(rows, 1)
        check(wq, w, x, ids, torch.randn((rows, n), device="cuda", generator=gen), 0.7)


def test_one_token_twice_and_masked_entries():
    n, k, m, top = 200, 96, 40, 12
    wq, w = table(n, k, 420)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((m, k), device="cuda", generator=gen) * 4
    ids = torch.randint(0, 6, (m, top), device="cuda", generator=gen, dtype=torch.int32)
    logits = torch.randn((m, top), device="cuda", generator=gen)
    logits[:, 3] = -INF
    logits[5] = -INF       # nothing left: no teacher
    logits[6, 1:] = -INF   # one certain token
    logits[7, 2] = float("nan")
    ids[7, 2] = -1         # an absent entry's logit does not matter
    logits[8] *= 1e30      # certain, by far
    check(wq, w, x, ids, logits, 1.0)
    loss, _, dx = q4.lmhead_distill(wq, x, ids, logits, grad=True)
    assert loss[5] == 0 and (dx[5] == 0).all()


def test_rows_apart():
    """NaN and infinities in x or in a teacher's logits stay in their row."""
    n, k, top = 700, 64, 9
    wq, _ = table(n, k, 430)
    for m in (40, 90):
        gen = torch.Generator(device="cuda").manual_seed(m)
        x = torch.randn((m, k), device="cuda", generator=gen)
        ids, logits = teacher(m, n, top, 3)
        want = q4.lmhead_distill(wq, x, ids, logits, grad=True)
        alone = q4.lmhead_distill(wq, x, ids, logits)
        x2, l2 = x.clone(), logits.clone()
        x2[4, 3], x2[9, 0], x2[0, 1] = float("nan"), INF, float("nan")
        l2[12, 8], l2[20, 0] = float("nan"), INF
        got = q4.lmhead_distill(wq, x2, ids, l2, grad=True)
        got_alone = q4.lmhead_distill(wq, x2, ids, l2)
        ok = torch.ones(m, dtype=torch.bool, device="cuda")
        ok[[0, 4, 9, 12, 20]] = False
        for a, b in zip(want, got):
            assert torch.equal(a[ok], b[ok])
        for a, b in zip(alone[:2], got_alone[:2]):
            assert torch.equal(a[ok], b[ok])
        for r in (4, 9, 12, 20):
            assert not got[0][r].isfinite() and not got_alone[0][r].isfinite()
            assert not got[2][r].isfinite().any()
        # row 0 has no teacher, whatever it holds
        assert got[0][0] == 0 and got_alone[0][0] == 0 and (got[2][0] == 0).all()


def test_gradient_against_differences():
    """The float32 gradient against central differences of the float64 loss."""
    n, k, m, top = 150, 64, 5, 8
    wq, w = table(n, k, 440)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((m, k), device="cuda", generator=gen) * 4
    ids, logits = teacher(m, n, top, 5, ragged=False)
    _, _, dx = q4.lmhead_distill(wq, x, ids, logits, temperature=2.0, grad=True)
    q = torch.softmax(logits.double() / 2, 1)

    def loss(y):
        logp = torch.log_softmax(y @ w.t() / 2, 1).gather(1, ids.long())
        return 4 * (q * (q.log() - logp)).sum(1)

    for seed in range(4):
        v = torch.randn((m, k), device="cuda", generator=gen).double()
        h = 1e-4
        slope = (loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)
        # differences: h^2 / 6 times the third derivative, below |v w|^3 / temperature
        err = (slope - (dx.double() * v).sum(1)).abs()
        tol = h * h * (v @ w.t()).abs().amax(1) ** 3 + 1e-5 * (dx.double().abs() * v.abs()).sum(1) + 1e-9
        assert (err <= tol).all(), (err, tol)
