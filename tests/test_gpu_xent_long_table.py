"""The loss alone for a few rows of a table with more logits than are kept at a time (2^26):
the direct kernel takes it in pieces.  Rows but the last 96 are zero, so the reference
stays small."""

import math

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24


@pytest.mark.parametrize("m,n", [(1, (1 << 26) - 7), (4, (1 << 24) + 65), (3, 40000001)])
def test_few_rows_of_a_long_table(m, n):
    """2^26 logits and less at once, and more in pieces."""
    k, tail = 64, 96
    g = torch.Generator(device="cuda").manual_seed(m)
    wq = torch.zeros((n, k // 32, 18), device="cuda", dtype=torch.uint8)  # scale 0
    q = torch.randint(0, 16, (tail, k // 32, 32), device="cuda", generator=g)
    d = torch.full((tail, k // 32, 1), 0.05, device="cuda", dtype=torch.float16)
    wq[n - tail:, :, :2] = d.view(torch.uint8).view(tail, k // 32, 2)
    wq[n - tail:, :, 2:] = (q[..., :16] | (q[..., 16:] << 4)).to(torch.uint8)
    w = ((q - 8).double() * d.double()).view(tail, k)
    x = torch.randn((m, k), device="cuda", generator=g) * 3
    t = torch.randint(n - tail, n, (m,), device="cuda", generator=g, dtype=torch.int32)
    t[-1] = n - 1
    announce(f"xent {m}x{n}x{k}")
    loss, lse, _ = q4.lmhead_xent(wq.view(n, -1), x, t)
    torch.cuda.synchronize()
    l = x.double() @ w.t()
    zeros = torch.full((m, 1), math.log(n - tail), device="cuda", dtype=torch.float64)
    ref = torch.logsumexp(torch.cat([l, zeros], 1), 1)
    want = ref - l.gather(1, (t.long() - (n - tail)).unsqueeze(1)).squeeze(1)
    # a logit: float32 sums of k products, x good to 2^-21; the sum of exponentials: entries of
    # 64 (or 4096) columns summed 256 apart, at most 4200 additions in a row
    tl = ((k + 64) * U + 2.0 ** -20) * (x.double().abs() @ w.abs().t()).amax(1)
    ts = 4200 * U + 2.0 ** -21 * (1 + l.abs().amax(1))
    assert ((lse.double() - ref).abs() <= tl + ts + U * ref).all()
    assert ((loss.double() - want).abs() <= 2 * tl + ts + 4 * U * (want.abs() + ref)).all()
