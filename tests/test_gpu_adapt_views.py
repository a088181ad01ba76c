"""Vectors that start in the middle of a 16-byte word: next-token targets are tokens[1:]."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


def shifted(t, by):
    """t's values in a view `by` elements into a buffer."""
    buf = torch.empty(t.numel() + by, device=t.device, dtype=t.dtype)
    buf[by:] = t
    assert buf[by:].data_ptr() % 16
    return buf[by:]


@pytest.mark.parametrize("by", [1, 2, 3])
def test_vectors_from_any_element(by):
    g = torch.Generator(device="cuda").manual_seed(by)
    m, n, k, r, na = 37, 300, 64, 8, 5
    wq = q4.quantize(torch.randn((n, k), device="cuda", generator=g) * 0.05)
    x = torch.randn((m, k), device="cuda", generator=g)
    dy = torch.randn((m, n), device="cuda", generator=g)
    t = torch.randint(0, n, (m,), device="cuda", generator=g, dtype=torch.int32)
    dloss = torch.rand(m, device="cuda", generator=g)
    a, b = torch.randn((na, r, k), device="cuda", generator=g), torch.randn((na, n, r), device="cuda", generator=g)
    ids = torch.randint(-1, na, (m,), device="cuda", generator=g, dtype=torch.int32)
    scale = torch.rand(na, device="cuda", generator=g)
    announce(f"vectors from element {by}")
    t2, dloss2, ids2, scale2 = (shifted(v, by) for v in (t, dloss, ids, scale))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for grad in (False, True):
            want = q4.lmhead_xent(wq, x, t, grad=grad, dloss=dloss)
            got = q4.lmhead_xent(wq, x, t2, grad=grad, dloss=dloss2, stream=stream)
            torch.cuda.synchronize()
            assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))
        want, got = q4.lora(x, a, b, ids, scale=scale), q4.lora(x, a, b, ids2, scale=scale2, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        want = q4.lora_grad(x, dy, a, b, ids, scale=scale)
        got = q4.lora_grad(x, dy, a, b, ids2, scale=scale2, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_captured():
    """The copy is part of a captured call: a replay sees the targets of the moment."""
    g = torch.Generator(device="cuda").manual_seed(9)
    m, n, k = 20, 300, 64
    wq = q4.quantize(torch.randn((n, k), device="cuda", generator=g) * 0.05)
    x = torch.randn((m, k), device="cuda", generator=g)
    tokens = torch.randint(0, n, (m + 1,), device="cuda", generator=g, dtype=torch.int32)
    loss, lse, dx = (torch.empty(s, device="cuda") for s in ((m,), (m,), (m, k)))
    q4.lmhead_xent(wq, x, tokens[1:], loss=loss, lse=lse, dx=dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.lmhead_xent(wq, x, tokens[1:], loss=loss, lse=lse, dx=dx)
    for rep in range(3):
        tokens.copy_(torch.randint(0, n, (m + 1,), device="cuda", generator=g, dtype=torch.int32))
        want = q4.lmhead_xent(wq, x, tokens[1:].clone(), grad=True)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((loss, lse, dx), want)), rep


def test_outputs_from_any_element_are_refused():
    x = torch.randn((4, 64), device="cuda")
    wq = q4.quantize(torch.randn((32, 64), device="cuda"))
    t = torch.zeros(4, device="cuda", dtype=torch.int32)
    for name in ("loss", "lse"):
        with pytest.raises(q4.Q4Error) as e:
            q4.lmhead_xent(wq, x, t, **{name: torch.empty(5, device="cuda")[1:]})
        assert e.value.status == q4.Q4_ERR_ALIGN
