"""Low-rank adapters of many requests (lora) and their gradient (lora_grad)
against plain float64 forms, one row at a time.

Tolerances, derived before any run.  Every output element is a float32 sum of
products whose terms the reference also gives in magnitude: with B the same
expression over absolute values (two chained sums for y, dx; the rows' sum of
such for da, db), L the longest chain of roundings, |err| <= L 2^-24 B, plus
half a step of the output type relative to the value.  A sum of n float32
products in any order has at most n roundings per term, and the two chained
sums add: L = K + R + 40 (the slices, the scale, the residual) for the sums
over K and R; errors of random sign grow with sqrt(L), so L 2^-24 is generous
and still catches a lost term (relative size 1 / n of B) for every n here
below 4096 = sqrt(2^24)."""

import numpy as np
import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def make(m, n, k, r, na, dtype, atype, seed, ids="mixed"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g).to(dtype)
    dy = (torch.randn((m, n), generator=g) * 0.1).to(dtype)
    a = (torch.randn((na, r, k), generator=g) * k ** -0.5).to(atype)
    b = (torch.randn((na, n, r), generator=g) * 0.1).to(atype)
    scale = torch.rand(na, generator=g) + 0.5
    if ids == "mixed":          # every row its own, some without
        i = torch.randint(-1, na + 1, (m,), generator=g)
    elif ids == "runs":
        i = torch.arange(m) * min(m, 5) // m % na
    elif ids == "none":
        i = torch.full((m,), -1)
    else:
        i = torch.full((m,), na - 1)
    return x, dy, a, b, scale, i.to(torch.int32)


def reference(x, dy, a, b, scale, ids, res_y, res_x):
    """float64: y, dx, da, db and the same sums over absolute values."""
    out = []
    for f in (lambda t: t, torch.abs):
        x6, dy6, a6, b6 = (f(t.double()) for t in (x, dy, a, b))
        y, dx = f(res_y.double()).clone(), f(res_x.double()).clone()
        da, db = torch.zeros_like(a6), torch.zeros_like(b6)
        s = scale.double()
        for j in range(a.shape[0]):
            rows = (ids == j).nonzero().squeeze(1)
            h, g = x6[rows] @ a6[j].t(), s[j] * (dy6[rows] @ b6[j])
            y[rows] += s[j] * (h @ b6[j].t())
            dx[rows] += g @ a6[j]
            da[j] = g.t() @ x6[rows]
            db[j] = s[j] * (dy6[rows].t() @ h)
        out.append((y, dx, da, db))
    return out


def check(got, want, bound, chain, what):
    got = got.cpu()
    half = torch.finfo(got.dtype).eps / 2
    # a subnormal result (float16) rounds by half of the smallest step instead
    tol = chain * 2.0 ** -24 * bound + half * want.abs() * (1 + 2.0 ** -10)
    tol += torch.finfo(got.dtype).tiny * half * 2 + 1e-30
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol).max()))


def run_case(m, n, k, r, na, dtype, atype, seed, ids="mixed"):
    x, dy, a, b, scale, i = make(m, n, k, r, na, dtype, atype, seed, ids)
    g = torch.Generator().manual_seed(seed + 1)
    ry, rx = torch.randn((m, n), generator=g).to(dtype), torch.randn((m, k), generator=g).to(dtype)
    (y, dx, da, db), (by, bx, ba, bb) = reference(x, dy, a, b, scale, i, ry, rx)
    cu = [t.cuda() for t in (x, dy, a, b, scale, i, ry, rx)]
    announce(f"lora {m}x{n}x{k} r={r} adapters={na} {dtype} {atype} {ids}")
    got = q4.lora(cu[0], cu[2], cu[3], cu[5], scale=cu[4], r=cu[6])
    torch.cuda.synchronize()
    check(got, y, by, k + r + 40, "y")
    announce("lora_grad")
    gx, ga, gb = q4.lora_grad(cu[0], cu[1], cu[2], cu[3], cu[5], scale=cu[4], r=cu[7])
    torch.cuda.synchronize()
    check(gx, dx, bx, n + r + 40, "dx")
    check(ga, da, ba, n + m + 40, "da")
    check(gb, db, bb, k + m + 40, "db")
    # again: the same bits
    assert torch.equal(q4.lora(cu[0], cu[2], cu[3], cu[5], scale=cu[4], r=cu[6]), got)
    for p, q in zip(q4.lora_grad(cu[0], cu[1], cu[2], cu[3], cu[5], scale=cu[4], r=cu[7]), (gx, ga, gb)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype,atype", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16),
                                         (F16, F32), (BF16, BF16), (BF16, F32)])
def test_types(dtype, atype):
    run_case(21, 200, 96, 16, 3, dtype, atype, 11)
    run_case(37, 203, 160, 24, 4, dtype, atype, 12)   # odd width: element loads and stores


@pytest.mark.parametrize("m,n,k,r,na,ids", [
    (1, 64, 32, 8, 1, "one"), (1, 1, 32, 8, 2, "one"), (1, 3072, 1280, 16, 8, "one"),
    (2, 5, 64, 8, 3, "mixed"), (15, 66, 32, 32, 2, "mixed"), (16, 64, 256, 64, 40, "mixed"),
    (17, 129, 288, 128, 2, "runs"), (64, 1000, 1280, 16, 48, "mixed"), (65, 256, 512, 72, 3, "runs"),
    (300, 644, 320, 40, 5, "runs"), (257, 130, 96, 8, 2, "none"), (700, 72, 64, 16, 700, "mixed"),
    (1000, 96, 96, 120, 2, "one")])
def test_shapes(m, n, k, r, na, ids):
    run_case(m, n, k, r, na, F32, BF16, 100 + m + n, ids)
    run_case(m, n, k, r, na, BF16, BF16, 200 + m + n, ids)


def test_long_axes():
    run_case(5, 18432, 3072, 16, 3, F32, F32, 31)
    run_case(40, 3072, 9216, 64, 2, F16, F16, 32, "runs")


def test_in_place_and_defaults():
    x, dy, a, b, scale, i = make(33, 130, 64, 8, 3, F32, F32, 41)
    one = torch.ones(3)
    (y, dx, _, _), (by, bx, _, _) = reference(x, dy, a, b, one, i, torch.zeros(33, 130),
                                              torch.zeros(33, 64))
    x, dy, a, b, i = (t.cuda() for t in (x, dy, a, b, i))
    check(q4.lora(x, a, b, i), y, by, 200, "no residual, no scale")
    r = torch.randn((33, 130), device="cuda")
    want = q4.lora(x, a, b, i, r=r)
    without = (i < 0) | (i >= 3)
    assert without.any() and torch.equal(want[without], r[without])
    buf = r.clone()
    assert q4.lora(x, a, b, i, r=buf, out=buf) is buf and torch.equal(buf, want)
    check(q4.lora_grad(x, dy, a, b, i)[0], dx, bx, 250, "dx")
    rx = torch.randn((33, 64), device="cuda")
    want = q4.lora_grad(x, dy, a, b, i, r=rx)
    buf = rx.clone()
    got = q4.lora_grad(x, dy, a, b, i, r=buf, dx=buf)
    for p, q in zip(got, want):
        assert torch.equal(p, q)


def test_strangers_do_not_leak():
    """Infinities and NaN in rows without an adapter, and in rows and parameters of other
    adapters, reach nobody else's results."""
    x, dy, a, b, scale, i = make(40, 100, 64, 8, 4, F32, F32, 51)
    x, dy, a, b, scale, i = (t.cuda() for t in (x, dy, a, b, scale, i))
    r, rx = torch.randn((40, 100), device="cuda"), torch.randn((40, 64), device="cuda")
    y = q4.lora(x, a, b, i, scale=scale, r=r)
    dx, da, db = q4.lora_grad(x, dy, a, b, i, scale=scale, r=rx)
    bad = (i == 2) | (i < 0) | (i >= 4)
    assert bad.any() and not bad.all()
    x2, dy2, a2, b2 = x.clone(), dy.clone(), a.clone(), b.clone()
    x2[bad], dy2[bad] = float("nan"), float("inf")
    a2[2], b2[2] = float("nan"), float("inf")
    y2 = q4.lora(x2, a2, b2, i, scale=scale, r=r)
    dx2, da2, db2 = q4.lora_grad(x2, dy2, a2, b2, i, scale=scale, r=rx)
    assert torch.equal(y2[~bad], y[~bad]) and torch.equal(dx2[~bad], dx[~bad])
    without = (i < 0) | (i >= 4)
    assert torch.equal(y2[without], r[without]) and torch.equal(dx2[without], rx[without])
    for j in (0, 1, 3):
        assert torch.equal(da2[j], da[j]) and torch.equal(db2[j], db[j])


def test_gradient_by_differences():
    """The gradient against central differences of the forward's float64 form.  The function is
    trilinear, so a central difference along one operand is exact but for rounding: with float64
    differences and an h of 1 the only error is the kernel's own."""
    m, n, k, r, na = 9, 20, 32, 8, 2
    x, dy, a, b, scale, i = make(m, n, k, r, na, F32, F32, 61)
    dx, da, db = (t.cpu().double() for t in q4.lora_grad(*(t.cuda() for t in (x, dy, a, b, i)),
                                                         scale=scale.cuda()))

    def f(x, a, b):
        tot = 0.0
        for row in range(m):
            j = int(i[row])
            if 0 <= j < na:
                tot += float(scale[j]) * float(dy[row].double() @ (b[j] @ (a[j] @ x[row])))
        return tot

    g = np.random.Generator(np.random.PCG64(3))
    p = [x.double(), a.double(), b.double()]
    for which, grad in ((0, dx), (1, da), (2, db)):
        size = float(grad.abs().max())
        for _ in range(12):
            at = tuple(int(g.integers(0, s)) for s in grad.shape)
            val = []
            for h in (1.0, -1.0):
                q = [t.clone() for t in p]
                q[which][at] += h
                val.append(f(*q))
            assert abs((val[0] - val[1]) / 2 - float(grad[at])) <= 1e-5 * size


def test_side_stream_and_graph():
    x, dy, a, b, scale, i = (t.cuda() for t in make(70, 256, 128, 16, 5, F32, BF16, 71))
    want = q4.lora(x, a, b, i, scale=scale)
    wantg = q4.lora_grad(x, dy, a, b, i, scale=scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q4.lora(x, a, b, i, scale=scale, stream=s)
    gotg = q4.lora_grad(x, dy, a, b, i, scale=scale, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(p, q) for p, q in zip(gotg, wantg))
    y, dx, da, db = (torch.empty_like(t) for t in (want, *wantg))
    ws = torch.empty(int(q4.lib().q4_lora_grad_workspace_bytes(70, 256, 128, 16)), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q4.lora(x, a, b, i, scale=scale, out=y, workspace=ws)
        q4.lora_grad(x, dy, a, b, i, scale=scale, dx=dx, da=da, db=db, workspace=ws)
    for rep in range(3):
        for t in (y, dx, da, db):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((y, dx, da, db), (want, *wantg)):
            assert torch.equal(p, q), rep
