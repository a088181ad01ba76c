"""verify_draft on logits and probabilities past 2^32 elements.  Sequences at the borders of
31- and 32-bit offsets hold logits of their own, so that an offset cut to 31 or 32 bits
reads another sequence's; they are compared with the float64 form of test_gpu_verify."""

import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_verify as V
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sequences_at_the_borders(dtype):
    s, d, n = 2060, 15, 131071  # odd: rows start at any element
    rows = (d + 1) * n
    gen = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.full((s, d + 1, n), -4.0, device="cuda", dtype=dtype)
    probs = torch.full((s, d, n), 1.0 / n, device="cuda", dtype=dtype)
    draft = torch.zeros((s, d), dtype=torch.int32, device="cuda")
    u = torch.rand((s, d + 1), device="cuda", generator=gen)
    # where bytes or elements of either tensor pass 2^31 and 2^32, what a cut offset of those
    # would read (the first), and the last ones
    edges = {0, s - 1}
    for size in (rows, d * n):
        for bits in (30, 31, 32):  # 2^30 elements are 2^31 bytes
            edges |= {e for e in (2 ** bits // size - 1, 2 ** bits // size, 2 ** bits // size + 1) if e < s}
    edges = sorted(edges)
    for e in edges:
        l, t, _, q = V.case(1, d, n, dtype, 100 + e, sharp=1.5)
        best = l[0, :d].argmax(1).to(torch.int32)
        logits[e], probs[e] = l[0], q[0]
        # a few drafted tokens that stand, then one that the draft drew
        keep = torch.arange(d, device="cuda") < e % 7
        draft[e] = torch.where(keep, best, t[0])
    at = torch.tensor(edges, device="cuda")
    for temp, p in ((0.0, None), (0.5, probs), (0.5, None)):
        announce(f"verify_draft {s} x {d} of {n} {dtype} temperature {temp} probs {p is not None}")
        tokens, accepted = q4.verify_draft(logits, draft, u, probs=p, temperature=temp)
        torch.cuda.synchronize()
        alone = V.check(logits[at], draft[at], u[at], None if p is None else p[at], temp=temp)
        assert torch.equal(tokens[at], alone[0]) and torch.equal(accepted[at], alone[1])
        assert len(set(map(tuple, tokens[at].tolist()))) == len(edges)  # each its own
