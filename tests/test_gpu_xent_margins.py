"""The gradient of the Q4_0 head's cross entropy for rows the model is sure of: targets far
above the other logits, table rows that share a component (the sum over the others and the
target's row then cancel), one piece of the vocabulary and several, against float64.

Tolerance of dx, derived before any run (u = 2^-24; o = the largest logit but the target's;
g = dloss): the bounds of the head's own tests, relative to the terms that are summed,
  |g| sum_{n != t} p_n (|T_n| + |T_t|) (4 tl + (N + 4096) u + c),
tl = (K + 64) u B + 2^-20 B the error of a logit, c = 2^-10 (16-bit types: probabilities and
weights as one binary16 number) or 2^-20, and for the probabilities' fixed step
  |g| p_o 2^-39 sum |T|
since they are kept relative to the largest of the others (half of binary16's smallest step,
2^-25, under a scale of 2^14), + half a step of the output, + the smallest normal number
for a probability below it.  dloss is exp(the margin), up to e^80, so that every row's
gradient is as large as the table's rows and no type's range hides an error."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: 0, F16: 1, BF16: 30}
U = 2.0 ** -24


def table(n, k, seed, shared):
    """n rows of Q4_0 with a common pattern `shared` times as large as their own part, and
    their float64 values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    own = torch.randint(-3, 4, (n, k // 32, 32), device="cuda", generator=g)
    common = torch.randint(-4, 5, (1, k // 32, 32), device="cuda", generator=g) if shared else 0
    q = (8 + own + common).clamp_(0, 15)
    d = (torch.rand((n, k // 32, 1), device="cuda", generator=g) * 0.001 + 0.006).half()
    raw = torch.empty((n, k // 32, 18), dtype=torch.uint8, device="cuda")
    raw[..., :2] = d.view(torch.uint8).view(n, k // 32, 2)
    raw[..., 2:] = (q[..., :16] | (q[..., 16:] << 4)).to(torch.uint8)
    return raw.view(n, -1), ((q - 8).double() * d.double()).view(n, k)


def workspace(dtype, m, n, k):
    return int(q4.lib().q4_lmhead_xent_workspace_bytes(CODE[dtype], 1, m, n, k))


def case(m, n, k, dtype, seed, shared, targets=()):
    wq, w = table(n, k, seed, shared)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, n, (m,), device="cuda", generator=g, dtype=torch.int32)
    if targets:
        t[: len(targets)] = torch.tensor(targets, dtype=torch.int32)
    margin = torch.linspace(0, 64, m, device="cuda", dtype=torch.float64)
    margin[-2:] = torch.tensor([90.0, 130.0], dtype=torch.float64)
    # x: noise, and along the target's own part as much as the margin takes
    v = w[t.long()] - w.mean(0)
    lead = v @ w.t()
    at = t.long().unsqueeze(1)
    gap = lead.gather(1, at).squeeze(1) - lead.scatter(1, at, -1e30).amax(1)
    x = torch.randn((m, k), device="cuda", generator=g).double() + (margin / gap).unsqueeze(1) * v
    x = x.to(dtype)
    dl = torch.exp(margin.clamp(max=80.0)).float()
    announce(f"xent margins {m}x{n}x{k} {dtype} shared={shared}")
    loss, lse, dx = q4.lmhead_xent(wq, x, t, grad=True, dloss=dl)
    torch.cuda.synchronize()

    x6 = x.double()
    l, b = x6 @ w.t(), (x6.abs() @ w.abs().t()).amax(1)
    ref_lse = torch.logsumexp(l, 1)
    lt = l.gather(1, at).squeeze(1)
    p = (l - ref_lse.unsqueeze(1)).exp_().scatter_(1, at, 0.0)
    rest, top = p.sum(1), p.amax(1)
    ref_loss = torch.where(rest < 0.5, -torch.log1p(-rest), ref_lse - lt)
    gr = dl.double()
    want = gr.unsqueeze(1) * (p @ w - rest.unsqueeze(1) * w[t.long()])
    terms = gr.unsqueeze(1) * (p @ w.abs() + rest.unsqueeze(1) * w[t.long()].abs())
    tl = ((k + 64) * U + 2.0 ** -20) * b
    c = 2.0 ** -20 if dtype == F32 else 2.0 ** -10
    f = torch.finfo(dtype)
    tol = terms * (4 * tl + (n + 4096) * U + c).unsqueeze(1)
    tol += (gr * (top * 2.0 ** -39 + 2.0 ** -126)).unsqueeze(1) * w.abs().sum(0)
    tol += f.eps / 2 * want.abs() * (1 + 2.0 ** -10) + f.tiny * f.eps
    for row in range(0, m, 8):  # margins of the rows: what a failure prints
        e = ((dx[row].double() - want[row]).norm() / want[row].norm()).item()
        print(f"margin {(lt[row] - l.scatter(1, at, -1e30).amax(1)[row]).item():7.2f} relative error {e:.1e}")
    err = (dx.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    size = 2.0 ** -21 * (1 + l.abs().amax(1))
    for loss, lse in ((loss, lse), q4.lmhead_xent(wq, x, t)[:2]):  # with the gradient, and alone
        assert ((loss.double() - ref_loss).abs()
                <= rest * (2 * tl + 4096 * U + size) + 2.0 ** -21 * ref_loss + n * 2.0 ** -126).all()
        assert ((lse.double() - ref_lse).abs() <= tl + 4096 * U + size).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("m,n,k", [(40, 700, 128), (64, 1001, 96), (70, 700, 128), (130, 515, 160), (9, 2, 64),
                                   (80, 2, 64)])
def test_margins(m, n, k, shared, dtype):
    """Straight from the Q4_0 bytes (up to 64 rows) and unpacked."""
    case(m, n, k, dtype, 6000 + m + n + shared, shared)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("k", [64, 96])
def test_margins_unpacked_pieces(k, dtype):
    """Three pieces of an unpacked table, targets at their first and last columns."""
    m, n = 70, 66000
    assert workspace(dtype, m, n, k) < n * k * 2 * (3 if dtype == F32 else 2)  # one piece's copies at a time
    piece = (n // 3 + 255) // 256 * 256
    case(m, n, k, dtype, 6200 + k, True,
         [0, piece - 1, piece, 2 * piece - 1, 2 * piece, n - 1] * 10)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("k", [64, 96])
def test_margins_direct_pieces(k, dtype):
    """Two pieces of the bytes, whose size the rows decide."""
    m, n = 64, (1 << 20) + 777
    # one piece's logits and probabilities at a time
    assert workspace(dtype, m, n, k) < 0.75 * m * n * (8 if dtype == F32 else 6)
    piece = ((n + 1) // 2 + 255) // 256 * 256
    case(m, n, k, dtype, 6300 + k, True, [0, piece - 1, piece, n - 1] * 14)


def test_one_column():
    """A table of one row: the loss and the gradient are zero, lse is its logit."""
    for m in (5, 70):
        wq, w = table(1, 64, 6400, False)
        x = torch.randn((m, 64), device="cuda")
        t = torch.zeros(m, device="cuda", dtype=torch.int32)
        t[1] = -1
        loss, lse, dx = q4.lmhead_xent(wq, x, t, grad=True)
        want = (x.double() @ w.t()).squeeze(1)
        assert (loss == 0).all() and (dx == 0).all()
        tl = (128 * U + 2.0 ** -20) * (x.double().abs() @ w.abs().t()).squeeze(1)
        assert ((lse.double() - want).abs() <= tl + U * want.abs()).all()
