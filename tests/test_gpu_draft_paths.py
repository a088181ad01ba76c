"""A draft model's operators along the paths a program takes them: long rows, values of
any magnitude, rows that must not see each other, outputs in place of inputs, halves of
one tensor, captured and replayed graphs, streams, offsets past 32 bits, and a run of them
together.  Tolerances are those of test_gpu_gated and test_gpu_distill; where bits are
compared, the same kernel does the same sums."""

import numpy as np
import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_distill as D
import test_gpu_gated as G
from gpu_util import announce, needs_gpu
from oracle import q4_oracle as O
from q4_quantized_speech_amd import synth

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")


# ------------------------------------------------------------------ the gated block

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 40, 4128), (4, 4200, 4160), (6, 33, 9216), (8, 64, 4352), (13, 50, 8224),
                                   (16, 4100, 4384), (16, 17, 4096), (3, 9, 4096), (30, 70, 4128), (64, 20, 9216)])
def test_forward_long_rows(m, n, k, dtype):
    qg, wg = G.weights(n, k, 30 * m + 1)
    qu, wu = G.weights(n, k, 30 * m + 2)
    x, res = G.inputs(m, n, k, dtype, m + n, m % 2 == 0)
    announce(f"gated_ffn {m}x{n}x{k} {dtype}")
    h, z = q4.gated_ffn(qg, qu, x, r=res, keep=True)
    torch.cuda.synchronize()
    want, tol, wz, tz = G.forward(wg, wu, x, res, "silu", dtype)
    G.assert_close(z, wz, tz, "z")
    G.assert_close(h, want, tol, "h")


@pytest.mark.parametrize("m", [1, 3, 16, 40, 100])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e15, 1e30])
def test_forward_any_magnitude(m, scale):
    """Rows of any magnitude keep their relative precision (float32 and bfloat16)."""
    n, k = 70, 320
    qg, wg = G.weights(n, k, 41)
    qu, wu = G.weights(n, k, 42)
    for dtype in (F32, BF16):
        gen = torch.Generator(device="cuda").manual_seed(m)
        x = (torch.randn((m, k), device="cuda", generator=gen) * scale).to(dtype)
        announce(f"gated_ffn {m} rows of magnitude {scale} {dtype}")
        _, z = q4.gated_ffn(qg, qu, x, keep=True)
        torch.cuda.synchronize()
        _, _, wz, tz = G.forward(wg, wu, x, None, "silu", dtype)
        # results below float32's (and so bfloat16's) normal numbers are as coarse as those
        G.assert_close(z, wz, tz + 2.0 ** -133, "z")


@pytest.mark.parametrize("m", [4, 8, 16, 40, 90])
def test_forward_rows_apart(m):
    n, k = 100, 256
    qg, _ = G.weights(n, k, 51)
    qu, _ = G.weights(n, k, 52)
    for dtype in (F32, F16, BF16):
        gen = torch.Generator(device="cuda").manual_seed(m)
        x = torch.randn((m, k), device="cuda", generator=gen).to(dtype)
        want, wz = q4.gated_ffn(qg, qu, x, keep=True)
        bad = x.clone()
        bad[0, 7], bad[2, 200], bad[m - 1] = NAN, INF, 0.0
        got, z = q4.gated_ffn(qg, qu, bad, keep=True)
        ok = torch.ones(m, dtype=torch.bool, device="cuda")
        ok[[0, 2, m - 1]] = False
        assert torch.equal(got[ok], want[ok]) and torch.equal(z[ok], wz[ok])
        assert not z[0].isfinite().any() and not z[2].isfinite().any()
        assert (got[m - 1] == 0).all() and (z[m - 1] == 0).all()


@pytest.mark.parametrize("m", [5, 20, 80])
def test_gradient_rows_apart(m):
    n, k = 90, 128
    qg, _ = G.weights(n, k, 53)
    qu, _ = G.weights(n, k, 54)
    for dtype in (F32, F16, BF16):
        gen = torch.Generator(device="cuda").manual_seed(m)
        z = torch.randn((m, 2 * n), device="cuda", generator=gen).to(dtype)
        dh = torch.randn((m, n), device="cuda", generator=gen).to(dtype)
        want, wz = q4.gated_ffn_grad(qg, qu, z, dh, keep=True)
        z2, d2 = z.clone(), dh.clone()
        d2[0, 3], z2[1, 5], d2[2], z2[3] = NAN, INF, 0.0, 0.0
        got, dz = q4.gated_ffn_grad(qg, qu, z2, d2, keep=True)
        assert torch.equal(got[4:], want[4:]) and torch.equal(dz[4:], wz[4:])
        assert not got[0].isfinite().any() and not got[1].isfinite().any()
        assert (got[2:4] == 0).all() and (dz[2:4] == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_far_out(act):
    """Pre-activations of any size: large ones pass or vanish, nothing turns into NaN."""
    n, k, m = 64, 32, 66
    qg, wg = G.weights(n, k, 61)
    qu, wu = G.weights(n, k, 62)
    zero = torch.zeros((m, k), device="cuda")
    r = torch.empty((m, 2 * n), device="cuda")
    r[:, :n] = torch.linspace(-1, 1, n, device="cuda") * (10.0 ** torch.linspace(-6, 30, m, device="cuda"))[:, None]
    r[:, n:] = 1.0
    for rows in (7, 40, m):
        h, z = q4.gated_ffn(qg, qu, zero[:rows], act=act, r=r[:rows].contiguous(), keep=True)
        want, tol, _, _ = G.forward(wg, wu, zero[:rows], r[:rows], act, F32)
        assert torch.equal(z, r[:rows])
        a, _, _, _, _ = G.gate(r[:rows, :n].double(), act)
        G.assert_close(h, want.nan_to_num(0.0), tol.nan_to_num(1e-30) + (a > 80) * 1e-30, act)
        dx, dz = q4.gated_ffn_grad(qg, qu, r[:rows].contiguous(), torch.ones((rows, n), device="cuda"), act=act, keep=True)
        assert dz.isfinite().all() and dx.isfinite().all()


def test_in_place_and_halves_of_one_tensor():
    n, k = 96, 160
    both, w = G.weights(2 * n, k, 71)
    for m in (3, 24, 70):
        x, res = G.inputs(m, n, k, F32, m, True)
        want, wz = q4.gated_ffn(both[:n], both[n:], x, r=res, keep=True)
        z = res.clone()
        got, same = q4.gated_ffn(both[:n], both[n:], x, r=z, z=z)
        assert same is z and torch.equal(got, want) and torch.equal(z, wz)
        full, tol, _, _ = G.forward(w[:n], w[n:], x, res, "silu", F32)
        G.assert_close(got, full, tol, "halves")
        dh = torch.randn((m, n), device="cuda")
        dx, dz = q4.gated_ffn_grad(both[:n], both[n:], wz, dh, keep=True)
        dx2, same = q4.gated_ffn_grad(both[:n], both[n:], z, dh, dz=z)
        assert same is z and torch.equal(dx2, dx) and torch.equal(z, dz)
    # rows that do not start at a 16-byte address are refused, not read wrongly
    odd, _ = G.weights(3, 32, 72)
    with pytest.raises(q4.Q4Error):
        q4.gated_ffn(odd[:1], odd[1:2], torch.zeros((1, 32), device="cuda"))


def test_rows_of_a_batch_alone():
    """A row's result does not depend on the other rows of its route."""
    n, k = 200, 512
    qg, _ = G.weights(n, k, 81)
    qu, _ = G.weights(n, k, 82)
    for lo, hi in ((9, 16), (33, 48), (130, 200)):
        x, _ = G.inputs(hi, n, k, F32, 1, False)
        assert torch.equal(q4.gated_ffn(qg, qu, x)[0][:lo], q4.gated_ffn(qg, qu, x[:lo].contiguous())[0])


def test_offsets_past_32_bits():
    """70000 rows of 2 x 16384: z has 2.3 G elements; the rows around 2^31 and the last ones."""
    m, n, k = 70000, 16384, 32
    qg, wg = G.weights(n, k, 91)
    qu, wu = G.weights(n, k, 92)
    x = torch.randn((m, k), device="cuda").to(BF16)
    announce(f"gated_ffn {m}x{n}x{k}")
    h, z = q4.gated_ffn(qg, qu, x, keep=True)
    dh = (h * 0.5)
    announce(f"gated_ffn_grad {m}x{n}x{k}")
    dx, dz = q4.gated_ffn_grad(qg, qu, z, dh, keep=True)
    torch.cuda.synchronize()
    edge = 2 ** 31 // (2 * n)
    for rows in (slice(0, 20), slice(edge - 10, edge + 10), slice(m - 20, m)):
        want, tol, wz, tz = G.forward(wg, wu, x[rows], None, "silu", BF16)
        G.assert_close(z[rows], wz, tz, "z")
        G.assert_close(h[rows], want, tol, "h")
        want, tol, wz, tz = G.gradient(wg, wu, z[rows], dh[rows], "silu", BF16)
        G.assert_close(dz[rows], wz, tz, "dz")
        G.assert_close(dx[rows], want, tol, "dx")


def test_verify_offsets_past_32_bits():
    """2060 sequences of 16 rows of 131072: 4.3 G logits.  The last sequences alone give the
    same tokens."""
    s, d, n = 2060, 15, 131072
    base = (2 * torch.randn((1, d + 1, n), device="cuda")).to(BF16)
    logits = base.expand(s, d + 1, n).contiguous()
    best = base[0, :, :].argmax(1).to(torch.int32)
    draft = best[:d].repeat(s, 1).contiguous()
    u = torch.rand((s, d + 1), device="cuda")
    announce(f"verify_draft {s} x {d} of {n}")
    for temp in (0.0, 0.3):
        tokens, accepted = q4.verify_draft(logits, draft, u, temperature=temp)
        for rows in (slice(0, 4), slice(s - 4, s)):
            t, a = q4.verify_draft(logits[rows], draft[rows], u[rows].contiguous(), temperature=temp)
            assert torch.equal(tokens[rows], t) and torch.equal(accepted[rows], a)
    assert (accepted < d).any() and (accepted >= 0).all()


@pytest.mark.parametrize("m", [1, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("k", [3840, 3872, 4064, 4096])
def test_forward_longest_rows_of_the_persistent_kernel(m, k):
    """Fifteen and sixteen waves, with as much LDS as their rows of x take."""
    n = 40
    qg, wg = G.weights(n, k, 95)
    qu, wu = G.weights(n, k, 96)
    for dtype in (F32, BF16, F16):
        x, _ = G.inputs(m, n, k, dtype, m, False)
        announce(f"gated_ffn {m}x{n}x{k} {dtype}")
        h, z = q4.gated_ffn(qg, qu, x, keep=True)
        want, tol, wz, tz = G.forward(wg, wu, x, None, "silu", dtype)
        G.assert_close(z, wz, tz, "z")
        G.assert_close(h, want, tol, "h")


@pytest.mark.parametrize("temp", [2.0 ** -60, 1e-9, 1e-6, 1e-3, 50.0, 2.0 ** 60])
def test_verify_any_temperature(temp):
    """From one token of each row to all of them alike; logits near and far from 0."""
    import test_gpu_verify as V
    l, draft, u, q = V.case(6, 3, 9000, F32, 17)
    l[1] += 3000.0
    l[2] *= 1e-6
    l[3] -= 1e6
    l[4, :, 100:] = -INF
    draft[4] %= 100
    l[5] *= 1e20
    best = l[:, :3].argmax(2).to(torch.int32)
    draft[::2] = best[::2]
    V.check(l, draft, u, q, temp=temp)
    V.check(l, draft, u, None, temp=temp)


def test_verify_more_chunks_than_threads():
    """A table of 2.6 million tokens: 640 chunks of a row."""
    import test_gpu_verify as V
    for dtype in (F32, BF16):
        l, draft, u, q = V.case(2, 1, 2621441, dtype, 18, sharp=1.0)
        l[1, 0, 2621440] = 30.0
        draft[1, 0] = 2621440
        V.check(l, draft, u, q)
        V.check(l, draft, u, None)
        u[:, 1] = 1 - 2.0 ** -24
        V.check(l, draft, u, q, temp=1.3)


# ------------------------------------------------------------------ graphs and streams

def calls(gen):
    """(name, function of the stream, output tensors, input tensors that may be refilled)."""
    out = []
    for m, n, k, dtype in ((1, 300, 512, F32), (7, 300, 512, BF16), (40, 200, 320, F32), (80, 150, 256, F16)):
        qg, _ = G.weights(n, k, 5)
        qu, _ = G.weights(n, k, 6)
        x = torch.randn((m, k), device="cuda", generator=gen).to(dtype)
        dh = torch.randn((m, n), device="cuda", generator=gen).to(dtype)
        h, z = torch.empty((m, n), dtype=dtype, device="cuda"), torch.empty((m, 2 * n), dtype=dtype, device="cuda")
        dx, dz = torch.empty_like(x), torch.empty_like(z)
        t = q4._TYPES[dtype]
        ws = torch.empty(max(16, q4._scratch_bytes("q4_gated_ffn_workspace_bytes", 0, t, m, n, k),
                             q4._scratch_bytes("q4_gated_ffn_grad_workspace_bytes", 0, t, m, n, k)),
                         dtype=torch.uint8, device="cuda")

        def block(st, qg=qg, qu=qu, x=x, dh=dh, h=h, z=z, dx=dx, dz=dz, ws=ws):
            q4.gated_ffn(qg, qu, x, out=h, z=z, workspace=ws, stream=st)
            q4.gated_ffn_grad(qg, qu, z, dh, act="gelu", dx=dx, dz=dz, workspace=ws, stream=st)
        out.append((f"gated {m}x{n}x{k}", block, [h, z, dx, dz], [x, dh]))
    for m, n, k, top, dtype in ((5, 900, 64, 9, F32), (90, 40000, 96, 17, BF16)):
        wq, _ = D.table(n, k, 7)
        x = torch.randn((m, k), device="cuda", generator=gen).to(dtype)
        ids, logits = D.teacher(m, n, top, 3)
        loss, lse = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        loss2, lse2 = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        dx = torch.empty_like(x)
        t = q4._TYPES[dtype]
        ws = torch.empty(max(q4._scratch_bytes("q4_lmhead_distill_workspace_bytes", 0, t, g, m, n, k, top) for g in (0, 1)),
                         dtype=torch.uint8, device="cuda")

        def loss_of(st, wq=wq, x=x, ids=ids, logits=logits, loss=loss, lse=lse, loss2=loss2, lse2=lse2, dx=dx, ws=ws):
            q4.lmhead_distill(wq, x, ids, logits, 2.0, loss=loss, lse=lse, dx=dx, workspace=ws, stream=st)
            q4.lmhead_distill(wq, x, ids, logits, 2.0, loss=loss2, lse=lse2, workspace=ws, stream=st)
        out.append((f"distill {m}x{n}x{k}", loss_of, [loss, lse, dx, loss2, lse2], [x, logits]))
    for s, d, n, temp in ((3, 4, 9000, 1.0), (40, 2, 500, 0.7), (2, 3, 5000, 0.0)):
        l = 3 * torch.randn((s, d + 1, n), device="cuda", generator=gen)
        q = torch.softmax(l[:, :d] + torch.randn((s, d, n), device="cuda", generator=gen), 2)
        draft = torch.multinomial(q.view(s * d, n), 1, generator=gen).view(s, d).to(torch.int32)
        u = torch.rand((s, d + 1), device="cuda", generator=gen)
        tokens = torch.empty((s, d + 1), dtype=torch.int32, device="cuda")
        accepted = torch.empty(s, dtype=torch.int32, device="cuda")
        ws = torch.empty(q4._scratch_bytes("q4_verify_draft_workspace_bytes", 0, s, d, n), dtype=torch.uint8, device="cuda")

        def verify(st, l=l, q=q, draft=draft, u=u, tokens=tokens, accepted=accepted, ws=ws, temp=temp):
            q4.verify_draft(l, draft, u, probs=q, temperature=temp, tokens=tokens, accepted=accepted, workspace=ws, stream=st)
        out.append((f"verify {s}x{d}x{n}", verify, [tokens, accepted], [l, u]))
    return out


def refill(tensors, gen):
    for t in tensors:
        t.copy_(torch.rand(t.shape, device="cuda", generator=gen) if t.shape[-1] < 10 and t.dim() == 2
                else 2 * torch.randn(t.shape, device="cuda", generator=gen))


def test_graph_replays_match_eager():
    """Captured calls whose workspaces are shared by several calls, replayed on new inputs with
    the outputs overwritten between, against eager calls; every replay is checked."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        todo = calls(gen)
        for name, call, _, _ in todo:
            announce(f"graph: {name}")
            call(st)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for _, call, _, _ in todo:
                call(st)
        for replay in range(4):
            for _, _, outs, ins in todo:
                refill(ins, gen)
                for t in outs:
                    t.fill_(-7 if t.dtype == torch.int32 else NAN)
            graph.replay()
            got = [[t.clone() for t in outs] for _, _, outs, _ in todo]
            for (name, call, outs, _), kept in zip(todo, got):
                for t in outs:
                    t.fill_(-7 if t.dtype == torch.int32 else NAN)
                call(st)
                st.synchronize()
                for a, b in zip(kept, outs):
                    assert torch.equal(a, b), (name, replay)


def test_two_streams_at_once():
    """The same calls on two streams, each with outputs and workspaces of its own."""
    gen = torch.Generator(device="cuda").manual_seed(22)
    first, second = calls(gen), calls(gen)
    want = []
    for todo in (first, second):
        for _, call, outs, _ in todo:
            call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([[t.clone() for t in outs] for _, _, outs, _ in todo])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (name, a, _, _), (_, b, _, _) in zip(first, second):
            announce(f"two streams: {name}")
            a(streams[0])
            b(streams[1])
    torch.cuda.synchronize()
    for todo, kept in zip((first, second), want):
        for (name, _, outs, _), old in zip(todo, kept):
            for x, y in zip(outs, old):
                assert torch.equal(x, y), name


def test_vectors_at_any_element():
    """ids, teacher logits, draft tokens and random numbers that are slices of larger tensors."""
    n, k, m, top = 300, 64, 6, 5
    wq, _ = D.table(n, k, 8)
    x = torch.randn((m, k), device="cuda")
    ids, logits = D.teacher(m, n, top, 4)
    want = q4.lmhead_distill(wq, x, ids, logits, grad=True)
    shifted = torch.zeros(m * top + 1, dtype=torch.int32, device="cuda")
    shifted[1:] = ids.flatten()
    floats = torch.zeros(m * top + 3, device="cuda")
    floats[3:] = logits.flatten()
    got = q4.lmhead_distill(wq, x, shifted[1:].view(m, top), floats[3:].view(m, top), grad=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    l = torch.randn((2, 4, 50), device="cuda")
    u = torch.rand(9, device="cuda")
    draft = torch.randint(0, 50, (7,), device="cuda", dtype=torch.int32)
    a = q4.verify_draft(l, draft[1:].view(2, 3), u[1:].view(2, 4))
    b = q4.verify_draft(l, draft[1:].view(2, 3).clone(), u[1:].view(2, 4).clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ together

def test_training_step_of_a_draft():
    """An adapted gated block and a down projection under the head, distilled from a teacher:
    the loss and the gradients of x and of both adapters against float64 autograd."""
    d, f, vocab, m, rank, top = 128, 192, 500, 20, 8, 16
    gen = torch.Generator(device="cuda").manual_seed(31)
    (qgu, wgu), (qd, wd), (qt, wt) = (G.weights(a, b, s) for a, b, s in ((2 * f, d, 1), (d, f, 2), (vocab, d, 3)))
    x = torch.randn((m, d), device="cuda", generator=gen)
    a = torch.randn((1, rank, d), device="cuda", generator=gen) / 8
    b = torch.randn((1, 2 * f, rank), device="cuda", generator=gen) / 8
    ids = torch.zeros(m, dtype=torch.int32, device="cuda")
    tids, tl = D.teacher(m, vocab, top, 5, ragged=False)
    dloss = torch.full((m,), 1.0 / m, device="cuda")

    r = q4.lora(x, a, b, ids)
    h, z = q4.gated_ffn(qgu[:f], qgu[f:], x, r=r, z=r)
    y = q4.matmul_residual(qd, h, x)
    loss, _, dy = q4.lmhead_distill(qt, y, tids, tl, temperature=2.0, grad=True, dloss=dloss)
    dh = q4.matmul_dx(qd, dy)
    dx, dz = q4.gated_ffn_grad(qgu[:f], qgu[f:], z, dh, dz=z)
    dx, da, db = q4.lora_grad(x, dz, a, b, ids, r=dx + dy)

    x6, a6, b6 = (t.double().requires_grad_() for t in (x, a[0], b[0]))
    z6 = x6 @ wgu.t() + x6 @ a6.t() @ b6.t()
    y6 = x6 + (z6[:, :f] * torch.sigmoid(z6[:, :f]) * z6[:, f:]) @ wd.t()
    logp = torch.log_softmax(y6 @ wt.t() / 2, 1).gather(1, tids.long())
    q = torch.softmax(tl.double() / 2, 1)
    loss6 = 4 * (q * (q.log() - logp)).sum(1)
    (loss6 * dloss.double()).sum().backward()
    # matmul_residual rounds x and weights to binary16 (2^-11 of each term): some 2^-10 of
    # the hidden state, and the results move with it by a few times that
    for got, want, what in ((loss, loss6.detach(), "loss"), (dx, x6.grad, "dx"), (da[0], a6.grad, "da"), (db[0], b6.grad, "db")):
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 4 * 2.0 ** -10, (what, err)


def test_greedy_drafts_change_nothing():
    """Decoding with drafted tokens gives the tokens that decoding without them gives: a target
    of one Q4_0 block and head, drafts that are right only now and then."""
    d, f, vocab, steps, draft_len = 96, 128, 300, 40, 4
    (qg, _), (qu, _), (qd, _), (qt, _) = (G.weights(a, b, s) for a, b, s in ((f, d, 11), (f, d, 12), (d, f, 13), (vocab, d, 14)))
    mix = torch.randn((d, d), device="cuda") / d ** 0.5

    def logits(tokens):
        """The target's logits after each token of [S, L]."""
        shape = tokens.shape
        e = 30 * q4.embed_rows(qt, tokens.flatten().contiguous())
        e = (e @ mix).contiguous()
        h, _ = q4.gated_ffn(qg, qu, e)
        y = q4.matmul_residual(qd, h, e)
        return (y.double() @ table.t()).float().view(*shape, vocab)

    table = torch.from_numpy(O.dequantize_q4_0(qt.cpu().numpy(), vocab, d)).double().cuda()
    plain = [5]
    for _ in range(steps):
        plain.append(int(logits(torch.tensor([[plain[-1]]], dtype=torch.int32, device="cuda"))[0, 0].argmax()))
    gen = torch.Generator().manual_seed(3)
    out, calls_made = [5], 0
    u = torch.rand((1, draft_len + 1), device="cuda")
    while len(out) <= steps:
        at = len(out)
        guess = [plain[at + i] if at + i < len(plain) and torch.rand((), generator=gen) < 0.7 else 7 for i in range(draft_len)]
        seq = torch.tensor([[out[-1]] + guess], dtype=torch.int32, device="cuda")
        draft = torch.tensor([guess], dtype=torch.int32, device="cuda")
        tokens, accepted = q4.verify_draft(logits(seq), draft, u, temperature=0.0)
        new = tokens[0, :int(accepted[0]) + 1].tolist()
        assert tokens[0, int(accepted[0]) + 1:].eq(-1).all() and new
        out += new
        calls_made += 1
    assert out[:steps + 1] == plain[:steps + 1]
    assert calls_made < steps
