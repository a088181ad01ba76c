"""The gradient of a Q4_0 projection (matmul_dx) and the cross entropy of the Q4_0
head with its gradient (lmhead_xent) against float64 forms on the oracle's decoded
weights.

Tolerances, derived before any run (u = 2^-24, half a float32 step; B = the sum of
the terms' magnitudes):
  matmul_dx    N u B for the float32 sum of N products, + 2^-20 B for the operands
               (two binary16 parts: each lo rounds at 2^-22, the dropped lo lo
               products are below 2^-22), or + 2^-11 B where the weight is rounded
               to binary16 (bfloat16), + 2^-40 max|dy| sum|w| for values far below
               their row's largest, + half a step of the output.
  logits       tl = (K + 64) u B + 2^-20 B (the few-row route splits x in two
               binary16 parts).  A shift of the logits by at most tl moves lse by
               tl and p_n by a factor of at most exp(2 tl).
  loss         its error is (1 - p_t) (2 tl + S u), S = 4096 the longest chain of a
               piece's partial sums, + 2^-21 (1 + |l|max) (1 - p_t) + 2^-21 loss.
  dx           (sum p |T| + (1 - p_t) |T_t|) |g| (4 tl + (N + S) u + c) with c = 2^-10
               where probabilities and weights are rounded to binary16 (16-bit types:
               two roundings of 2^-11), 2^-20 for float32, + half a step.
A norm-wise check beside the element-wise one: errors of random sign leave float32
results within 2 sqrt(terms) u + 2^-20 of the result's 2-norm."""

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


# ------------------------------------------------------------------ matmul_dx

def dx_case(m, n, k, dtype, seed, scale=1.0):
    wq, w = table(n, k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn((m, n), device="cuda", generator=g) * scale
    dy *= 10.0 ** torch.empty((m, 1), device="cuda").uniform_(-3, 3, generator=g)
    dy = dy.to(dtype)
    announce(f"matmul_dx {m}x{n}x{k} {dtype} scale {scale}")
    got = q4.matmul_dx(wq, dy)
    torch.cuda.synchronize()
    d = dy.double()
    want, b = d @ w, d.abs() @ w.abs()
    c = 2.0 ** -11 if dtype == BF16 else 2.0 ** -20
    tol = (n * U + c) * b + 2.0 ** -40 * d.abs().amax(1, keepdim=True) * w.abs().sum(0)
    assert_close(got, want, tol + half_step(dtype, want) + 1e-300, "dx")
    if dtype == F32:
        rows = (got.double() - want).norm(dim=1) / want.norm(dim=1).clamp_min(1e-300)
        assert float(rows.max()) <= 2 * n ** 0.5 * U + 2.0 ** -20, float(rows.max())
    assert torch.equal(q4.matmul_dx(wq, dy), got)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 70, 64), (3, 64, 96), (16, 257, 160), (17, 33, 288),
                                   (33, 1000, 1280), (64, 96, 32), (130, 131, 416), (300, 640, 320),
                                   (513, 320, 1056)])
def test_dx_shapes(m, n, k, dtype):
    # float16 gradients stay inside its range
    dx_case(m, n, k, dtype, 1000 + m + n, 0.1 if dtype == F16 else 1.0)


@pytest.mark.parametrize("m,n,k,dtype", [(16, 3072, 4096, F32), (375, 1280, 5120, F32), (1500, 5120, 1280, BF16),
                                         (76, 18432, 3072, F16), (2, 3072, 9216, F32)])
def test_dx_model_shapes(m, n, k, dtype):
    dx_case(m, n, k, dtype, 2000 + m, 0.01)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e20])
def test_dx_range(scale):
    dx_case(20, 200, 96, F32, 3000, scale)
    dx_case(20, 200, 96, BF16, 3001, scale)


def test_dx_rows_apart():
    """Zero rows, rows with infinities and NaN: nothing crosses rows."""
    wq, w = table(130, 64, 3100)
    dy = torch.randn((40, 130), device="cuda")
    want = q4.matmul_dx(wq, dy)
    bad = dy.clone()
    bad[3] = 0
    bad[7, 5] = float("nan")
    bad[21, 100] = float("inf")
    got = q4.matmul_dx(wq, bad)
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[[3, 7, 21]] = False
    assert torch.equal(got[ok], want[ok]) and (got[3] == 0).all()
    assert got[7].isnan().all() and not got[21].isfinite().any()


def test_dx_subnormal_scales():
    """Block scales that are binary16 subnormals: the two parts of a weight stay exact."""
    n, k = 96, 64
    g = np.random.Generator(np.random.PCG64(9))
    qb = O.quantize_q4_0(synth.weights(n, k, 3200)).reshape(n, k // 32, 18)
    bits = g.integers(1, 1024, (n, k // 32)).astype(np.uint16)
    qb[..., :2] = bits[..., None].view(np.uint8)
    qb = np.ascontiguousarray(qb.reshape(n, -1))
    w = torch.from_numpy(O.dequantize_q4_0(qb, n, k)).double().cuda()
    dy = torch.randn((24, n), device="cuda")
    got = q4.matmul_dx(torch.from_numpy(qb).cuda(), dy)
    d = dy.double()
    assert_close(got, d @ w, (n * U + 2.0 ** -20) * (d.abs() @ w.abs()), "subnormal")


# ------------------------------------------------------------------ lmhead_xent

def reference(w, x, targets, dloss):
    n = w.shape[0]
    x6, t = x.double(), targets.long()
    l, b = x6 @ w.t(), x6.abs() @ w.abs().t()
    lse = torch.logsumexp(l, 1)
    valid = (t >= 0) & (t < n)
    at = torch.where(valid, t, 0).unsqueeze(1)
    p = (l - lse.unsqueeze(1)).exp_()
    p.scatter_(1, at, torch.where(valid.unsqueeze(1), 0.0, p.gather(1, at)))
    rest = p.sum(1)
    # log(1 + rest / p_t), the loss of a sure row to full precision
    lt = l.gather(1, at).squeeze(1)
    loss = torch.where(valid, torch.where(rest < 0.5, -torch.log1p(-rest), lse - lt), 0.0)
    g = (dloss.double() if dloss is not None else torch.ones_like(lse)) * valid
    q = p.scatter(1, at, -rest.unsqueeze(1))
    dx, bx = g.unsqueeze(1) * (q @ w), g.abs().unsqueeze(1) * (q.abs() @ w.abs())
    return dict(l=l, b=b, lse=lse, valid=valid, rest=rest, loss=loss, dx=dx, bx=bx, g=g)


def xent_case(m, n, k, dtype, seed, grad=True, ramp=False, xscale=1.0, dloss=True, targets=None):
    wq, w = table(n, k, seed, ramp)
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, n, (m,), device="cuda", generator=g, dtype=torch.int32)
    x = torch.randn((m, k), device="cuda", generator=g) * xscale
    x += torch.rand((m, 1), device="cuda", generator=g) * w[t.long()].float() * (40000.0 / k)
    x = x.to(dtype)
    if targets is not None:
        t[: len(targets)] = torch.tensor(targets[:m], dtype=torch.int32)
    dl = torch.rand(m, device="cuda", generator=g) if dloss else None
    announce(f"xent {m}x{n}x{k} {dtype} grad={grad} ramp={ramp} xscale={xscale}")
    loss, lse, dx = q4.lmhead_xent(wq, x, t, grad=grad, dloss=dl)
    torch.cuda.synchronize()
    r = reference(w, x, t, dl)
    top = r["l"].abs().amax(1)
    tl = ((k + 64) * U + 2.0 ** -20) * r["b"].amax(1)
    s = 4096 * U
    assert_close(lse, r["lse"], tl + s + 2.0 ** -21 * (1 + top), "lse")
    rest = torch.where(r["valid"], r["rest"], 0.0)
    # terms of the sum below the smallest normal float32 relative to the row's
    # maximum (2^-126 each) may vanish: a loss is a sum of n such terms
    tiny = n * 2.0 ** -126
    assert_close(loss, r["loss"],
                 rest * (2 * tl + s + 2.0 ** -21 * (1 + top)) + 2.0 ** -21 * r["loss"].abs() + tiny, "loss")
    if not grad:
        assert dx is None
        return
    c = 2.0 ** -20 if dtype == F32 else 2.0 ** -10
    tol = r["bx"] * (4 * tl + (n + 4096) * U + c).unsqueeze(1)
    tol += (r["g"].abs() * 2.0 ** -38).unsqueeze(1) * w.abs().sum(0)
    assert_close(dx, r["dx"], tol + half_step(dtype, r["dx"]) + 1e-300, "dx")
    if dtype == F32 and xscale <= 1:
        err = float((dx.double() - r["dx"]).norm() / r["dx"].norm().clamp_min(1e-300))
        assert err <= 2 * float(tl.max()) + 2 * n ** 0.5 * U + 2.0 ** -20, err
    loss2, lse2, dx2 = q4.lmhead_xent(wq, x, t, grad=True, dloss=dl)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dx, dx2)


ODD = [-100, 0, -1, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 2, 64), (2, 63, 96), (5, 65, 32), (16, 300, 160),
                                   (17, 64, 64), (40, 1000, 1280), (130, 4097, 288), (300, 700, 416)])
def test_xent_shapes(m, n, k, dtype):
    xent_case(m, n, k, dtype, 4000 + m + n, targets=ODD if m > 5 else None)
    xent_case(m, n, k, dtype, 4500 + m + n, grad=False, targets=ODD if m > 5 else None)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 31, 128), (5, 300, 128), (15, 513, 256), (16, 512, 384), (17, 1025, 128),
                                   (32, 700, 640), (33, 2000, 256), (48, 511, 128), (49, 65, 256), (64, 3000, 384),
                                   (65, 600, 128), (7, 100, 64), (40, 900, 192), (64, 129, 320), (20, 1300, 448)])
def test_xent_few_rows(m, n, k, dtype):
    """Up to 64 rows with K a multiple of 64: straight from the Q4_0 bytes; one row more."""
    xent_case(m, n, k, dtype, 4700 + m + n, targets=ODD if m > 5 else None)
    xent_case(m, n, k, dtype, 4800 + m + n, grad=False, targets=ODD if m > 5 else None)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_xent_pieces(dtype):
    """Several pieces of the vocabulary, a short last one, the maximum growing through them;
    targets in the first and last rows of pieces."""
    for n in (32769, 40001, 70000):
        t = [0, n - 1, 32767, 32768, n // 2, -1]
        xent_case(20, n, 64, dtype, 5000 + n, ramp=True, targets=t)
        xent_case(20, n, 64, dtype, 5000 + n, ramp=True, targets=t, grad=False)
    xent_case(3000, 45000, 32, dtype, 5100, ramp=True, targets=ODD)


def test_xent_few_rows_pieces():
    """The direct form's pieces are of 2^26 / M columns: 64 rows over a table past one of them."""
    n = (1 << 20) + 777
    xent_case(64, n, 128, BF16, 5150, ramp=True, targets=[0, n - 1, (n + 1) // 2 // 256 * 256, -1])
    xent_case(64, n, 128, F32, 5150, ramp=True, grad=False)


@pytest.mark.parametrize("grad", [False, True])
def test_xent_head(grad):
    xent_case(3, 131072, 3072, F32, 5200, grad=grad)
    xent_case(70, 131072, 1280, BF16, 5201, grad=grad)


@pytest.mark.parametrize("m", [2, 40])
def test_xent_extremes(m):
    """Huge logits of either sign (a softmax that is one token), tiny ones (a flat one), no
    dloss, every row padding."""
    xent_case(m, 500, 64, F32, 5300, xscale=3e4)
    xent_case(m, 500, 64, F32, 5301, xscale=1e-20, dloss=False)
    xent_case(m, 500, 64, BF16, 5302, xscale=1e3, dloss=False)
    wq, w = table(300, 64, 5303)
    x = torch.randn((m, 64), device="cuda")
    t = torch.full((m,), -100, dtype=torch.int32, device="cuda")
    loss, lse, dx = q4.lmhead_xent(wq, x, t, grad=True)
    assert (loss == 0).all() and (dx == 0).all()
    assert torch.allclose(lse.double(), torch.logsumexp(x.double() @ w.t(), 1), atol=1e-5)


def test_xent_rows_apart():
    wq, _ = table(700, 64, 5400)
    for m in (9, 40):
        x = torch.randn((m, 64), device="cuda")
        t = torch.randint(0, 700, (m,), device="cuda", dtype=torch.int32)
        a = q4.lmhead_xent(wq, x, t, grad=True)
        b = q4.lmhead_xent(wq, x, t)
        x2 = x.clone()
        x2[4, 3], x2[6] = float("nan"), float("inf")
        ok = torch.ones(m, dtype=torch.bool, device="cuda")
        ok[[4, 6]] = False
        for want, got in ((a, q4.lmhead_xent(wq, x2, t, grad=True)), (b, q4.lmhead_xent(wq, x2, t))):
            for p, q in zip(want, got):
                if p is not None:
                    assert torch.equal(p[ok], q[ok])
            assert got[0][4].isnan() and got[1][4].isnan()


def test_xent_gradient_by_differences():
    """Central differences of the float64 loss with steps of 1e-4: their truncation is
    h^2 / 6 times the third derivative, below 1e-8 of the weights' scale here."""
    n, k, m = 50, 32, 24
    wq, w = table(n, k, 5500)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m, k), device="cuda", generator=g)
    t = torch.randint(0, n, (m,), device="cuda", generator=g, dtype=torch.int32)
    dx = q4.lmhead_xent(wq, x, t, grad=True)[2].double()
    f = lambda v: torch.nn.functional.cross_entropy(v @ w.t(), t.long(), reduction="sum")  # noqa: E731
    for i in range(0, m, 5):
        for j in range(0, k, 7):
            a, b = x.double(), x.double()
            a[i, j] += 1e-4
            b[i, j] -= 1e-4
            assert abs(float((f(a) - f(b)) / 2e-4 - dx[i, j])) <= 1e-6 * float(dx.abs().max()) + 1e-8


# ------------------------------------------------------------------ streams, graphs, a step

def test_side_stream_and_graph():
    wq, _ = table(3000, 96, 5600)
    x = torch.randn((50, 96), device="cuda")
    t = torch.randint(0, 3000, (50,), device="cuda", dtype=torch.int32)
    dy = torch.randn((50, 3000), device="cuda", dtype=BF16)
    few = x[:3].to(BF16).contiguous()
    want = [*q4.lmhead_xent(wq, x, t, grad=True), *q4.lmhead_xent(wq, few, t[:3].contiguous())[:2],
            q4.matmul_dx(wq, dy)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t3 = t[:3].contiguous()
    got = [*q4.lmhead_xent(wq, x, t, grad=True, stream=s), *q4.lmhead_xent(wq, few, t3, stream=s)[:2],
           q4.matmul_dx(wq, dy, stream=s)]
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    out = [torch.empty_like(p) for p in want]
    need = [int(q4.lib().q4_lmhead_xent_workspace_bytes(0, 1, 50, 3000, 96)),
            int(q4.lib().q4_lmhead_xent_workspace_bytes(30, 0, 3, 3000, 96)),
            int(q4.lib().q4_matmul_dx_workspace_bytes(30, 50, 3000, 96))]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q4.lmhead_xent(wq, x, t, loss=out[0], lse=out[1], dx=out[2], workspace=ws)
        q4.lmhead_xent(wq, few, t3, loss=out[3], lse=out[4], workspace=ws)
        q4.matmul_dx(wq, dy, out=out[5], workspace=ws)
    for rep in range(3):
        for p in out:
            p.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), rep


def test_training_step():
    """A step as it is used: an adapted projection, the head's loss, and the gradients back
    to the adapters and the input, against float64 through torch's autograd."""
    m, d, hid, v, r = 40, 64, 96, 500, 8
    wq, w = table(hid, d, 5700)
    tq, tab = table(v, hid, 5701)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((m, d), device="cuda", generator=gen)
    a = torch.randn((2, r, d), device="cuda", generator=gen) * d ** -0.5
    b = torch.randn((2, hid, r), device="cuda", generator=gen) * 0.3
    scale = torch.tensor([1.5, 0.5], device="cuda")
    ids = (torch.arange(m, device="cuda") % 3 - 1).to(torch.int32)
    t = torch.randint(0, v, (m,), device="cuda", generator=gen, dtype=torch.int32)
    # the projection runs with binary16 operands from five rows up: its own
    # tolerance (2e-3 of the terms) is what the step is held to
    y = q4.lora(x, a, b, ids, scale=scale)
    y = q4.matmul_residual(wq, x, y, out=y)
    loss, _, dy = q4.lmhead_xent(tq, y, t, grad=True, dloss=torch.full((m,), 1 / m, device="cuda"))
    dx = q4.matmul_dx(wq, dy)
    dx, da, db = q4.lora_grad(x, dy, a, b, ids, scale=scale, r=dx, dx=dx)
    x6, a6, b6 = (p.double().requires_grad_() for p in (x, a, b))
    ok = ids >= 0
    sel = torch.where(ok, ids, 0).long()
    h = torch.bmm(a6[sel], x6.unsqueeze(2))
    low = torch.bmm(b6[sel], h).squeeze(2) * (scale.double()[sel] * ok).unsqueeze(1)
    y6 = x6 @ w.t() + low
    loss6 = torch.nn.functional.cross_entropy(y6 @ tab.t(), t.long(), reduction="none")
    loss6.mean().backward()
    assert float((loss.double() - loss6).abs().max()) <= 2e-3 * float(y6.detach().abs().max())
    for got, want in ((dx, x6.grad), (da, a6.grad), (db, b6.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 2e-3


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_xent_pieces_unpacked(dtype):
    """Several pieces of an unpacked table: more than 64 rows, and K an odd multiple of 32."""
    for m, n, k in ((70, 40001, 64), (20, 70000, 96)):
        t = [0, n - 1, 32767, 32768, n // 2, -1]
        xent_case(m, n, k, dtype, 5300 + n, ramp=True, targets=t)
        xent_case(m, n, k, dtype, 5300 + n, ramp=True, targets=t, grad=False)


@pytest.mark.parametrize("m,n,k", [(4, 1000, 2048), (5, 1000, 2048), (16, 16384, 2112), (16, 16385, 2048),
                                   (17, 500, 2048), (16, 300, 1984), (1, 40000, 96), (2, 40000, 96),
                                   (16, 21845, 96), (16, 21846, 96), (16, 1985, 1056), (16, 1986, 1056),
                                   (3, 500, 1056), (3, 500, 992)])
def test_xent_loss_routes(m, n, k):
    """Losses alone on both sides of the sizes that choose between the kernels."""
    for dtype in (F32, BF16):
        xent_case(m, n, k, dtype, 5400 + m, grad=False, targets=ODD if m > 5 else None)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(2, 1, 32), (2, 3, 96), (5, 31, 32), (17, 33, 160), (33, 63, 224), (49, 65, 288),
                                   (64, 129, 352), (64, 128, 416), (20, 2001, 1056), (70, 301, 160), (16, 515, 480)])
def test_odd_blocks(m, n, k, dtype):
    """K an odd multiple of 32 (every other row of the weights starts in the middle of a
    dword), with an odd or even last row: the head's loss and gradient, and dx."""
    xent_case(m, n, k, dtype, 5500 + m + n, targets=ODD if m > 5 else None)
    xent_case(m, n, k, dtype, 5600 + m + n, grad=False, targets=ODD if m > 5 else None)
    dx_case(m, n, k, dtype, 5700 + m + n)
    dx_case(300, n, k, dtype, 5800 + m + n)


@pytest.mark.parametrize("n", [(1 << 20) + 777, (1 << 20) + 2048])
def test_odd_blocks_pieces(n):
    """K an odd multiple of 32 and more columns than one piece of the direct form."""
    t = [0, n - 1, (n + 1) // 2 // 256 * 256, n // 2, -1]
    xent_case(64, n, 96, BF16, 5900, ramp=True, targets=t)
    xent_case(64, n, 96, F32, 5900, ramp=True, grad=False, targets=t)
