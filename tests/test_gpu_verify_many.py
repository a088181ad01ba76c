"""verify_draft with more chunks of 4096 columns than one launch takes workgroups (2^23; a
dimension of 256 threads cannot have 2^24): the whole against its parts, whose launches are
small, and against the float64 form of test_gpu_verify."""

import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_verify as V
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("s,d,n,dtype", [(1 << 18, 63, 3, torch.float32), (1 << 20, 15, 4, torch.bfloat16),
                                         ((1 << 17) + 40, 63, 1, torch.float16), (520, 63, 300, torch.float32)])
def test_many_sequences(s, d, n, dtype):
    """2^24 chunks, 2^24, a few more than 2^23, and one launch."""
    gen = torch.Generator(device="cuda").manual_seed(d + n)
    logits = torch.randn((s, d + 1, n), device="cuda", generator=gen).to(dtype)
    draft = torch.randint(0, n, (s, d), device="cuda", generator=gen, dtype=torch.int32)
    # drafts that stand for a while: the best token, mostly
    best = logits[:, :d].argmax(2).to(torch.int32)
    draft = torch.where(torch.rand((s, d), device="cuda", generator=gen) < 0.9, best, draft)
    u = torch.rand((s, d + 1), device="cuda", generator=gen)
    lens = torch.randint(0, d + 1, (s,), device="cuda", generator=gen, dtype=torch.int32)
    for temp in (0.25, 0.0):
        announce(f"verify_draft {s} x {d} of {n} {dtype} temperature {temp}")
        tokens, accepted = q4.verify_draft(logits, draft, u, lens=lens, temperature=temp)
        torch.cuda.synchronize()
        part = s // 8
        for at in (0, 3 * part, s - part):
            rows = slice(at, at + part)
            t, a = q4.verify_draft(logits[rows], draft[rows].clone(), u[rows].clone(), lens=lens[rows].clone(), temperature=temp)
            assert torch.equal(tokens[rows], t) and torch.equal(accepted[rows], a), (at, temp)
    for at in (0, s // 2 - 10, s - 20):
        rows = slice(at, at + 20)
        some = V.check(logits[rows].contiguous(), draft[rows].contiguous(), u[rows].contiguous(), lens=lens[rows].contiguous(), temp=0.0)
        assert torch.equal(some[0], tokens[rows]) and torch.equal(some[1], accepted[rows])
