"""Verification of drafted tokens (verify_draft) against a float64 form written out per
sequence.  Its results are whole numbers: they have to be equal.  Random numbers that lie
within 1e-10 of a border are moved by 1e-6 before the call, so that no rounding decides."""

import math

import numpy as np
import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


def distribution(l, temp):
    """p of a row of logits (float64), or None."""
    top = l.max() if l.size else -INF
    if np.isnan(l).any() or not math.isfinite(top):
        return None
    if temp == 0:
        p = np.zeros_like(l)
        p[int(np.argmax(l == top))] = 1.0
        return p
    e = np.exp((l - top) / temp)
    return e / e.sum()


def expect(logits, draft, u, probs, length, temp):
    """(tokens, accepted, smallest distance of a random number to its border) of a sequence."""
    d, n = draft.shape[0], logits.shape[1]
    tokens, near = [-1] * (d + 1), 1.0
    for i in range(d + 1):
        p = distribution(logits[i], temp)
        if i < length:
            t = int(draft[i])
            inside = 0 <= t < n
            q = np.zeros(n) if probs is None else probs[i]
            qt = 1.0 if probs is None else (float(q[t]) if inside else 1.0)
            pt = float(p[t]) if p is not None and inside else 0.0
            if p is not None and inside and qt > 0:
                near = min(near, abs(float(u[i]) - pt / qt))
            if p is not None and float(u[i]) * qt < pt:
                tokens[i] = t
                continue
            if p is not None:
                if probs is None and inside:
                    q[t] = 1.0
                rest = np.maximum(p - q, 0.0)
                if rest.sum() > 0:
                    p = rest
        if p is not None:
            c = np.cumsum(p)
            goal = float(u[d]) * c[-1]
            near = min(near, float(np.abs(c / c[-1] - float(u[d])).min()))
            hit = np.nonzero((c > goal) & (p > 0))[0]
            tokens[i] = int(hit[0]) if hit.size else int(np.nonzero(p > 0)[0][-1])
        return tokens, i, near
    raise AssertionError


def check(logits, draft, u, probs=None, lens=None, temp=1.0):
    s, rows, n = logits.shape
    d = rows - 1
    l6, p6 = logits.double().cpu().numpy(), None if probs is None else probs.double().cpu().numpy()
    dn, ln = draft.cpu().numpy(), None if lens is None else lens.cpu().numpy()
    want, count = [], []
    u = u.clone()
    for i in range(s):
        length = d if ln is None else int(min(max(ln[i], 0), d))
        for _ in range(20):
            t, a, near = expect(l6[i], dn[i], u[i].double().cpu().numpy(), None if probs is None else p6[i], length, temp)
            if near > 1e-10:
                break
            u[i] = (u[i] + 1e-6) % 1.0
        want.append(t)
        count.append(a)
    announce(f"verify_draft {s} x {d} of {n} {logits.dtype} temperature {temp} probs {probs is not None}")
    tokens, accepted = q4.verify_draft(logits, draft, u, probs=probs, lens=lens, temperature=temp)
    torch.cuda.synchronize()
    assert accepted.tolist() == count
    assert tokens.tolist() == want
    again = q4.verify_draft(logits, draft, u, probs=probs, lens=lens, temperature=temp)
    assert torch.equal(again[0], tokens) and torch.equal(again[1], accepted)
    return tokens, accepted


def case(s, d, n, dtype, seed, sharp=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = (sharp * torch.randn((s, d + 1, n), device="cuda", generator=g)).to(dtype)
    q = torch.softmax(l[:, :d].float() + 0.7 * torch.randn((s, d, n), device="cuda", generator=g), 2).to(dtype)
    draft = torch.zeros((s, d), dtype=torch.int32, device="cuda")
    if d:
        draft = torch.multinomial(q.float().view(s * d, n), 1, generator=g).view(s, d).to(torch.int32)
    u = torch.rand((s, d + 1), device="cuda", generator=g)
    return l, draft, u, q


SHAPES = [(1, 0, 1), (1, 1, 1), (3, 2, 2), (2, 4, 63), (5, 3, 257), (1, 4, 4096), (2, 5, 4097), (7, 1, 5000),
          (4, 7, 12289), (2, 63, 300), (40, 2, 1000), (1, 0, 131072), (3, 5, 131071)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("s,d,n", SHAPES)
def test_shapes(s, d, n, dtype):
    l, draft, u, q = case(s, d, n, dtype, s + d + n)
    for temp in (1.0, 0.6, 0.0):
        check(l, draft, u, q, temp=temp)
        check(l, draft, u, None, temp=temp)
    lens = torch.randint(-1, d + 2, (s,), device="cuda", dtype=torch.int32)
    check(l, draft, u, q, lens=lens)


def test_masked_rows_and_tokens():
    s, d, n = 12, 3, 5000
    l, draft, u, q = case(s, d, n, F32, 1)
    l[0, 0] = -INF                       # no distribution at once
    l[1, 1, 77] = float("nan")
    l[2, 2, 5] = INF
    l[3, :, 1:] = -INF                   # one token left
    draft[3] = 0
    l[4, :, 4096:] = -INF                # a whole chunk masked
    l[5, :, :4096] = -INF
    l[6, 0, int(draft[6, 0])] = -INF     # the drafted token is masked
    l[7] = 0                             # all alike
    draft[8, 0], draft[9, 0], draft[10, 1] = -1, n, -2**31
    u[:8, :d] = 1e-9                     # whatever may stand does
    for temp in (1.0, 0.0):
        check(l, draft, u, q, temp=temp)
        check(l, draft, u, None, temp=temp)


def test_random_numbers_at_the_ends():
    l, draft, u, q = case(6, 2, 9000, F32, 2)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    u[2, :2], u[2, 2] = 0.0, 1 - 2.0 ** -24
    tokens, accepted = q4.verify_draft(l, draft, u, probs=q)
    assert accepted[0] == 2 and accepted[2] == 2  # 0 q < p
    assert ((tokens >= -1) & (tokens < 9000)).all()
    # out of the stated range: refused tokens and some token, never a bad index
    u[3], u[4], u[5] = 1.0, 7.0, float("nan")
    tokens, accepted = q4.verify_draft(l, draft, u, probs=q)
    assert (accepted[4:] == 0).all()
    assert (tokens[3:, 0] >= 0).all() and (tokens < 9000).all()


def test_draft_equal_to_the_target():
    """p = q: everything stands while u < 1 (up to rounding), and where probabilities above p
    refuse a token nothing is left, so p itself is drawn from."""
    s, d, n = 4, 3, 1000
    l, draft, u, _ = case(s, d, n, F32, 3)
    q = torch.softmax(l[:, :d], 2)
    u[:, :d] *= 0.999
    tokens, accepted = q4.verify_draft(l, draft, u, probs=q.contiguous())
    assert (accepted == d).all() and torch.equal(tokens[:, :d], draft)
    check(l, draft, u, (4 * q).contiguous())
    u[:, :d] = 0.9
    check(l, draft, u, (4 * q).contiguous())


def test_greedy_ties_go_to_the_lowest():
    s, d, n = 3, 2, 9000
    l = torch.zeros((s, d + 1, n), device="cuda", dtype=BF16)
    l[0, :, [8999, 4500, 123]] = 3.0
    l[1, :, [8999, 4096, 4095]] = 3.0
    draft = torch.tensor([[123, 4500], [4095, 4095], [0, 0]], dtype=torch.int32, device="cuda")
    u = torch.rand((s, d + 1), device="cuda")
    tokens, accepted = check(l, draft, u, None, temp=0.0)
    assert accepted.tolist() == [1, 2, 2]
    assert tokens.tolist() == [[123, 123, -1], [4095, 4095, 4095], [0, 0, 0]]


def test_drawn_tokens_have_the_targets_distribution():
    """Whatever the draft, a first token is distributed as p: 20000 sequences over 8 tokens.
    The counts' distances from 20000 p, squared over the expected, are chi-squared with 7
    degrees of freedom: above 40 once in 10^6 runs, and the seed is fixed."""
    s, n = 20000, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    row = torch.randn(n, device="cuda", generator=g)
    q = torch.softmax(torch.randn(n, device="cuda", generator=g), 0)
    l = row.expand(s, 2, n).contiguous()
    probs = q.expand(s, 1, n).contiguous()
    draft = torch.multinomial(probs.view(s, n), 1, generator=g).to(torch.int32)
    u = torch.rand((s, 2), device="cuda", generator=g)
    p = torch.softmax(row.double(), 0)
    for pr, dr in ((probs, draft), (None, torch.full_like(draft, 3))):
        tokens, accepted = q4.verify_draft(l, dr, u, probs=pr)
        counts = torch.bincount(tokens[:, 0].long(), minlength=n).double()
        chi = float(((counts - s * p) ** 2 / (s * p)).sum())
        assert chi < 40, (chi, counts.tolist(), (s * p).tolist())
