"""The operators that adapt a frozen model where offsets pass 32 bits, and called from two
threads at once.  Large operands are zero, or repeat, outside a few rows, so that the
references (64 bits) stay small."""

import math
import threading

import pytest
import torch

import q4_quantized_speech_amd as q4

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of float32
BF16 = 2.0 ** -8  # half a step of bfloat16


def announce(what):
    print(what, flush=True)


def table(n, k, seed):
    """n random rows of Q4_0 (uint8 [n, 18 k / 32]) and their values (float64)."""
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (n, k // 32, 18), generator=g, dtype=torch.uint8)
    d = (torch.rand((n, k // 32, 1), generator=g) * 0.01 + 0.001).half()
    raw[..., :2] = d.view(torch.uint8).reshape(n, k // 32, 2)
    codes = raw[..., 2:].to(torch.int64)
    q = torch.cat([codes & 15, codes >> 4], dim=2) - 8
    return raw.reshape(n, -1).contiguous(), (q.double() * d.double()).reshape(n, k)


def test_lora_offsets_past_32_bits():
    """A and its gradient hold 2.4e9 elements; the last adapter and the first are used."""
    adapters, r, k, n, m = 2300, 128, 8192, 64, 70
    assert adapters * r * k > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    announce(f"lora {m}x{n}x{k} rank {r} of {adapters}")
    a = torch.zeros((adapters, r, k), device="cuda", dtype=torch.bfloat16)
    b = torch.zeros((adapters, n, r), device="cuda", dtype=torch.bfloat16)
    for i in (0, adapters - 1):
        a[i] = torch.randn((r, k), device="cuda", generator=g) / math.sqrt(k)
        b[i] = torch.randn((n, r), device="cuda", generator=g) / math.sqrt(r)
    x = torch.randn((m, k), device="cuda", generator=g).bfloat16()
    dy = torch.randn((m, n), device="cuda", generator=g).bfloat16()
    ids = torch.full((m,), adapters - 1, device="cuda", dtype=torch.int32)
    ids[::3] = 0
    y = q4.lora(x, a, b, ids).double().cpu()
    dx, da, db = q4.lora_grad(x, dy, a, b, ids)
    torch.cuda.synchronize()
    ids, xs, dys = ids.cpu(), x.double().cpu(), dy.double().cpu()
    for i in (0, adapters - 1):
        rows = ids == i
        ai, bi, xi, di = a[i].double().cpu(), b[i].double().cpu(), xs[rows], dys[rows]
        h, gr = xi @ ai.T, di @ bi
        habs, gabs = xi.abs() @ ai.abs().T, di.abs() @ bi.abs()
        # float32 sums of C terms: C U of the absolute sum; a rank vector as two bfloat16
        # parts: 2^-16 of it; the 16-bit result's rounding
        eh, eg = (k + 64) * U * habs + 2.0 ** -16 * h.abs(), (n + 64) * U * gabs + 2.0 ** -16 * gr.abs()
        ref = h @ bi.T
        tol = BF16 * ref.abs() + 1.01 * (eh @ bi.abs().T + (r + 64) * U * h.abs() @ bi.abs().T)
        assert ((y[rows] - ref).abs() <= tol).all()
        ref = gr @ ai
        tol = BF16 * ref.abs() + 1.01 * (eg @ ai.abs() + (r + 64) * U * gr.abs() @ ai.abs())
        assert ((dx[rows.cuda()].double().cpu() - ref).abs() <= tol).all()
        ref = gr.T @ xi
        tol = 1.01 * (eg.T @ xi.abs() + (m + 64) * U * gr.abs().T @ xi.abs())
        assert ((da[i].double().cpu() - ref).abs() <= tol).all()
        ref = di.T @ h
        tol = 1.01 * (di.abs().T @ eh + (m + 64) * U * di.abs().T @ h.abs())
        assert ((db[i].double().cpu() - ref).abs() <= tol).all()
    assert not da[1:-1].any() and not db[1:-1].any()


def test_matmul_dx_offsets_past_32_bits():
    """dx holds 2^32 elements and more: 64 rows of dy over and over."""
    reps, n, k = 8193, 64, 8192
    assert 64 * reps * k > 1 << 32
    wq, w = table(n, k, 2)
    g = torch.Generator().manual_seed(2)
    dy = torch.randn((64, n), generator=g).bfloat16()
    announce(f"dx {64 * reps}x{n}x{k}")
    dx = q4.matmul_dx(wq.cuda(), dy.cuda().repeat(reps, 1)).view(reps, 64, k)
    for i in range(0, reps, 1024):
        part = dx[i:i + 1024]
        assert torch.equal(part, dx[:1].expand_as(part)), i
    ref = dy.double() @ w
    absum = dy.double().abs() @ w.abs()
    # weights rounded to binary16 (2^-11), float32 sums, the result's rounding
    tol = BF16 * ref.abs() + 1.01 * (2.0 ** -11 + (n + 64) * U) * absum
    assert ((dx[0].double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("m,grad", [(2, False), (5, True), (70, True)])
def test_xent_offsets_past_32_bits(m, grad):
    """A table of 4.8 GB whose rows are zero but for the last 64."""
    n, k, tail = 1 << 21, 4096, 64
    g = torch.Generator().manual_seed(m)
    last, w = table(tail, k, 3)
    wq = torch.zeros((n, k // 32 * 18), device="cuda", dtype=torch.uint8)
    assert wq.numel() > 1 << 32
    wq[n - tail:] = last.cuda()
    x = torch.randn((m, k), generator=g) * 2
    t = torch.randint(n - tail, n, (m,), generator=g, dtype=torch.int32)
    t[0] = n - 1
    t[1] = 7  # a zero row
    announce(f"xent {m}x{n}x{k} grad={grad}")
    loss, lse, dx = q4.lmhead_xent(wq, x.cuda(), t.cuda(), grad=grad)
    torch.cuda.synchronize()
    l = x.double() @ w.T
    ref = torch.logsumexp(torch.cat([l, torch.full((m, 1), math.log(n - tail), dtype=torch.float64)], 1), 1)
    lt = torch.where(t < n - tail, torch.zeros(m, dtype=torch.float64),
                     l.gather(1, (t.long() - (n - tail)).clamp(min=0)[:, None])[:, 0])
    bound = (x.double().abs() @ w.abs().T).max(1).values
    # logits: float32 sums of k terms over operands good to 2^-21; their sum of exponentials is
    # made of at most 1100 additions in a row
    tl = ((k + 64) * U + 2.0 ** -20) * bound
    ts = 2.0 ** -13
    assert ((lse.double().cpu() - ref).abs() <= tl + ts + U * ref.abs()).all()
    want = ref - lt
    assert ((loss.double().cpu() - want).abs() <= 2 * tl + ts + 4 * U * (want.abs() + lt.abs())).all()
    if not grad:
        return
    p = torch.exp(l - ref[:, None])
    wt = torch.where((t < n - tail)[:, None], torch.zeros(1, dtype=torch.float64),
                     w[(t.long() - (n - tail)).clamp(min=0)])
    want = p @ w - wt
    size = p @ w.abs() + wt.abs()
    tol = 1.01 * (2 * tl + 2 * ts)[:, None] * size + U * want.abs()
    assert ((dx.double().cpu() - want).abs() <= tol).all()


def test_two_threads_at_once():
    """Two host threads, each on a stream of its own: the same bits as one after the other."""
    wq, _ = table(1000, 256, 4)
    wq = wq.cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    jobs = []
    for m in (33, 300):
        x = torch.randn((m, 256), device="cuda", generator=g).bfloat16()
        dy = torch.randn((m, 1000), device="cuda", generator=g).bfloat16()
        a = torch.randn((3, 16, 256), device="cuda", generator=g).bfloat16()
        b = torch.randn((3, 1000, 16), device="cuda", generator=g).bfloat16()
        ids = torch.randint(-1, 3, (m,), device="cuda", generator=g, dtype=torch.int32)
        t = torch.randint(0, 1000, (m,), device="cuda", generator=g, dtype=torch.int32)

        def job(x=x, dy=dy, a=a, b=b, ids=ids, t=t):
            return [q4.matmul_dx(wq, dy), *q4.lmhead_xent(wq, x, t, grad=True),
                    q4.lora(x, a, b, ids), *q4.lora_grad(x, dy, a, b, ids)]
        jobs.append(job)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    bad, errors = [], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                with torch.cuda.stream(stream):
                    got = jobs[i]()
                stream.synchronize()
                bad.extend((i, j) for j, (u, v) in enumerate(zip(got, want[i])) if not torch.equal(u, v))
        except Exception as e:  # reported by the main thread
            errors.append(e)

    announce("two threads")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and not bad
