"""Measured cases of the gated feed-forward block on Q4_0 weights (gated_ffn) and its
gradient (gated_ffn_grad), the distillation of a teacher's top logits through the Q4_0
LM head (lmhead_distill), and the verification of drafted tokens (verify_draft).

Shapes are the speech model's: decoder width 3072 with 9216 gated units, encoder width
1280 with 5120, the 131072-row table, the 38- and 76-token prefixes, 375 and 1500
positions.  Weights are Gaussians of deviation 0.02 encoded to Q4_0 blocks (binary16
scale, then 16 bytes: weight j of a block in the low nibble of byte j, weight j + 16 in
the high).
"""

import math

import torch

own = False

VOCAB, DEC, ENC, FFN = 131072, 3072, 1280, 9216
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the block of one decoder layer for one streamed token
        {"name": "ffn_decode_1", "op": "ffn", "m": 1, "n": FFN, "k": DEC, "act": "silu", "type": "f32", "res": False,
         "keep": False},
        # seven streams decoded together, with their adapters' share of the projections
        {"name": "ffn_decode_7", "op": "ffn", "m": 7, "n": FFN, "k": DEC, "act": "silu", "type": "bf16", "res": True,
         "keep": False},
        # the 38-token decoder prefix
        {"name": "ffn_prefix_38", "op": "ffn", "m": 38, "n": FFN, "k": DEC, "act": "silu", "type": "f32", "res": False,
         "keep": False},
        # forward of a training step, 1500 positions, projections kept for the backward pass
        {"name": "ffn_train_1500", "op": "ffn", "m": 1500, "n": FFN, "k": DEC, "act": "silu", "type": "bf16",
         "res": False, "keep": True},
        # backward of the 76-token prefix, the projections' gradients returned for their adapters
        {"name": "ffn_grad_76", "op": "ffn_grad", "m": 76, "n": FFN, "k": DEC, "act": "silu", "type": "f32",
         "keep": True},
        # backward of 1500 frames through an encoder-sized block
        {"name": "ffn_grad_1500", "op": "ffn_grad", "m": 1500, "n": 5120, "k": ENC, "act": "gelu", "type": "bf16",
         "keep": False},
        # distance of eight streamed tokens from their teacher
        {"name": "distill_score_8", "op": "distill", "m": 8, "n": VOCAB, "k": ENC, "top": 16, "temp": 1.0,
         "type": "f32", "grad": False},
        # training step of a draft as wide as the encoder, kept in float32
        {"name": "distill_train_375", "op": "distill", "m": 375, "n": VOCAB, "k": ENC, "top": 32, "temp": 2.0,
         "type": "f32", "grad": True},
        # training step at the decoder's width over 1500 positions
        {"name": "distill_train_1500", "op": "distill", "m": 1500, "n": VOCAB, "k": DEC, "top": 64, "temp": 1.0,
         "type": "bf16", "grad": True},
        # four drafted tokens of one stream, the draft's distribution at hand
        {"name": "verify_1x4", "op": "verify", "s": 1, "d": 4, "n": VOCAB, "temp": 1.0, "type": "f32", "probs": True,
         "ragged": False},
        # 48 streams, drafts that carry no distribution (a lookup of earlier text), of any length up to seven
        {"name": "verify_48x7", "op": "verify", "s": 48, "d": 7, "n": VOCAB, "temp": 0.7, "type": "bf16",
         "probs": False, "ragged": True},
        # 64 streams of five drafted tokens
        {"name": "verify_64x5", "op": "verify", "s": 64, "d": 5, "n": VOCAB, "temp": 1.0, "type": "f32", "probs": True,
         "ragged": False},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "distill", "distill", "verify", "verify"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "verify":
        s, d = _log(rng, 1, 64), rng.randint(0, 7)
        while s * (d + 1) > 384:
            d -= 1
        return {"op": op, "s": s, "d": d, "n": _log(rng, 500, VOCAB), "temp": rng.choice([0.0, 0.7, 1.0, 1.3]),
                "type": kind, "probs": rng.random() < 0.6, "ragged": rng.random() < 0.5}
    if op == "distill":
        grad = rng.random() < 0.6
        return {"op": op, "m": _log(rng, 1, 375 if kind == "f32" else 1500), "n": _log(rng, 500, VOCAB),
                "k": 32 * _log(rng, 4, DEC // 32), "top": _log(rng, 1, 64), "temp": rng.choice([1.0, 1.5, 2.0, 4.0]),
                "type": kind, "grad": grad}
    c = {"op": op, "m": _log(rng, 1, 375 if kind == "f32" else 1500), "n": _log(rng, 64, FFN),
         "k": 32 * _log(rng, 4, DEC // 32), "act": rng.choice(["silu", "gelu"]), "type": kind}
    if op == "ffn":
        c["res"] = rng.random() < 0.4
    c["keep"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs

def _q4(n, k, gen):
    """n rows of k Gaussian weights as Q4_0 blocks."""
    w = torch.randn((n, k // 32, 32), device="cuda", generator=gen).mul_(0.02)
    at = w.abs().argmax(-1, keepdim=True)
    d = w.gather(-1, at).div_(-8.0).to(torch.float16)
    inv = torch.where(d == 0, torch.zeros_like(d, dtype=torch.float32), 1.0 / d.float())
    q = w.mul_(inv).add_(8.5).floor_().clamp_(0, 15).to(torch.uint8)
    out = torch.empty((n, k // 32, 18), dtype=torch.uint8, device="cuda")
    out[..., :2] = d.view(torch.uint8)
    out[..., 2:] = q[..., :16] | (q[..., 16:] << 4)
    return out.view(n, k // 32 * 18)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    t, n, op = TYPES[case["type"]], case["n"], case["op"]
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=t):
        return torch.randn(shape, device="cuda", generator=gen).mul_(std).to(dtype)

    if op == "ffn":
        s["gate"], s["up"] = _q4(n, case["k"], gen), _q4(n, case["k"], gen)
        s["x"] = normal(case["m"], case["k"])  # after the norm
        if case["res"]:
            s["r"] = normal(case["m"], 2 * n, std=0.2)
    elif op == "ffn_grad":
        s["gate"], s["up"] = _q4(n, case["k"], gen), _q4(n, case["k"], gen)
        s["z"] = normal(case["m"], 2 * n)
        # a gradient: small, rows of different sizes
        size = torch.rand((case["m"], 1), device="cuda", generator=gen).mul_(0.02)
        s["dh"] = (torch.randn((case["m"], n), device="cuda", generator=gen) * size).to(t)
    elif op == "distill":
        m, k, top = case["m"], case["k"], case["top"]
        s["w"] = _q4(n, k, gen)
        # the teacher's best tokens, distinct, its logits falling from the first to the last
        ids = torch.randint(0, n, (m, 1), device="cuda", generator=gen)
        step = max(1, n // top)
        ids = (ids + torch.arange(top, device="cuda") * step) % n
        logits = 14.0 - 4.0 * torch.rand((m, top), device="cuda", generator=gen).cumsum(1).sqrt()
        logits = logits + torch.randn((m, top), device="cuda", generator=gen) * 0.3
        # hidden states: unit noise, plus a part along the first tokens' rows that makes the
        # student lean to them, more or less
        lean = torch.rand((m, 1), device="cuda", generator=gen).mul_(10.0)
        x = torch.randn((m, k), device="cuda", generator=gen)
        for j in range(min(top, 3)):
            x += lean * (0.5 ** j) * _decode(s["w"][ids[:, j]]) * (2500.0 / k)
        s["x"] = x.to(t)
        ids = ids.to(torch.int32)
        if m > 8:
            # padding positions, and positions whose teacher kept fewer entries
            ids[torch.rand(m, device="cuda", generator=gen) < 0.05] = -1
            few = torch.rand((m, 1), device="cuda", generator=gen) < 0.1
            ids = torch.where(few & (torch.arange(top, device="cuda") >= (top + 1) // 2), -1, ids)
        s["ids"], s["logits"] = ids.contiguous(), logits.contiguous()
        s["dloss"] = torch.full((m,), 1.0 / m, device="cuda")
        if t == torch.float16:  # scaled against underflow, as such training does
            s["dloss"].mul_(4096.0)
    else:
        seqs, d = case["s"], case["d"]
        # sharp target distributions: noise, and some tokens that stand out
        l = torch.randn((seqs, d + 1, n), device="cuda", generator=gen).mul_(1.5)
        out = torch.randint(0, n, (seqs, d + 1, 12), device="cuda", generator=gen)
        l.scatter_add_(2, out, torch.rand((seqs, d + 1, 12), device="cuda", generator=gen).mul_(8.0).add_(7.0))
        # the draft's are near them
        q = torch.randn((seqs, d, n), device="cuda", generator=gen).mul_(0.7).add_(l[:, :d])
        q = torch.softmax(q, 2)
        draft = torch.zeros((seqs, d), dtype=torch.int32, device="cuda")
        if d:
            draft = torch.multinomial(q.view(seqs * d, n), 1, generator=gen).view(seqs, d).to(torch.int32)
        s["logits"], s["draft"] = l.to(t), draft
        s["probs"] = q.to(t) if case["probs"] and d else None
        s["u"] = torch.rand((seqs, d + 1), device="cuda", generator=gen)
        s["lens"] = None
        if case["ragged"]:
            s["lens"] = torch.randint(0, d + 1, (seqs,), device="cuda", generator=gen, dtype=torch.int32)
    return s


# ---------------------------------------------------------------- plain forms

def _decode(w):
    """float32 weights of Q4_0 rows: (code - 8) * scale."""
    b = w.view(w.shape[0], -1, 18)
    d = b[..., :2].contiguous().view(torch.float16).float()
    q = torch.cat([b[..., 2:] & 15, b[..., 2:] >> 4], dim=-1).float()
    return q.sub_(8.0).mul_(d).view(w.shape[0], -1)


GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(g, act):
    """The activation and its derivative (gelu: its tanh form)."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(GELU_A * (g + GELU_B * g * g * g))
    slope = GELU_A * (1.0 + 3.0 * GELU_B * g * g)
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * slope


def _plain_ffn(gate, up, x, r, act, keep):
    n = gate.shape[0]
    x32 = x.float()
    g, u = x32 @ _decode(gate).t(), x32 @ _decode(up).t()
    if r is not None:
        g, u = g + r[:, :n].float(), u + r[:, n:].float()
    h = (_act(g, act)[0] * u).to(x.dtype)
    return (h, torch.cat([g, u], 1).to(x.dtype)) if keep else h


def _plain_ffn_grad(gate, up, z, dh, act, keep):
    n = gate.shape[0]
    g, u, d = z[:, :n].float(), z[:, n:].float(), dh.float()
    a, da = _act(g, act)
    dg, du = d * u * da, d * a
    dx = (dg @ _decode(gate) + du @ _decode(up)).to(z.dtype)
    return (dx, torch.cat([dg, du], 1).to(z.dtype)) if keep else dx


def _plain_distill(w, x, ids, logits, temp, dloss, grad):
    t = _decode(w)
    l = (x.float() @ t.t()) / temp
    top = l.amax(dim=1, keepdim=True)
    e = (l - top).exp_()
    s = e.sum(dim=1, keepdim=True, dtype=torch.float64)
    lse = s.log() + top
    there = (ids >= 0) & (ids < w.shape[0])
    any_there = there.any(1)
    at = torch.where(there, ids, 0).long()
    b = torch.where(there, logits.double() / temp, -math.inf)
    b = b - torch.where(any_there, b.amax(1), 0.0).unsqueeze(1)
    q = b.exp()
    total = q.sum(1, keepdim=True)
    q = torch.where(any_there.unsqueeze(1), q / total, 0.0)
    logq = b - total.log()
    logp = l.gather(1, at).double() - lse
    loss = temp * temp * torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    if not grad:
        return loss.float(), lse.squeeze(1).float()
    p = e.div_(s.float()).scatter_add_(1, at, -q.float())
    p = p.mul_(torch.where(any_there, dloss * temp, 0.0).unsqueeze(1))
    return loss.float(), lse.squeeze(1).float(), (p @ t).to(x.dtype)


def _plain_verify(logits, draft, u, probs, lens, temp):
    seqs, rows, n = logits.shape
    d, dev = rows - 1, logits.device
    l = logits.double()
    top = l.amax(2, keepdim=True)
    if temp == 0:  # greedy: the lowest token of the largest logit
        place = torch.arange(n, device=dev)
        best = torch.where(l == top, place, n).amin(2, keepdim=True)
        p = (place == best).double()
    else:
        p = ((l - top) / temp).exp()
        p = p / p.sum(2, keepdim=True)
    if lens is None:
        lens = torch.full((seqs,), d, dtype=torch.int32, device=dev)
    pt = p[:, :d].gather(2, draft.long().unsqueeze(2)).squeeze(2)
    qt = 1.0 if probs is None else probs.gather(2, draft.long().unsqueeze(2)).squeeze(2).double()
    ok = (u[:, :d].double() * qt < pt) & (torch.arange(d, device=dev) < lens.unsqueeze(1))
    count = ok.int().cumprod(1).sum(1)
    each = torch.arange(seqs, device=dev)
    row = p[each, count]
    if d:
        at = count.clamp(max=d - 1)
        if probs is None:
            left = row.scatter(1, draft[each, at].long().unsqueeze(1), 0.0)
        else:
            left = (row - probs[each, at].double()).clamp(min=0.0)
        cut = (count < lens) & (left.sum(1) > 0)
        row = torch.where(cut.unsqueeze(1), left, row)
    c = row.cumsum(1)
    new = (c <= u[:, d:].double() * c[:, -1:]).sum(1).clamp(max=n - 1)
    place = torch.arange(d + 1, device=dev)
    tokens = torch.cat([draft.long(), new.unsqueeze(1)], 1)
    tokens = torch.where(place < count.unsqueeze(1), tokens, -1)
    tokens = torch.where(place == count.unsqueeze(1), new.unsqueeze(1), tokens)
    return tokens.to(torch.int32), count.to(torch.int32)


def run(s):
    c = s["case"]
    if own:
        import q4_quantized_speech_amd as q4
        if c["op"] == "ffn":
            h, z = q4.gated_ffn(s["gate"], s["up"], s["x"], act=c["act"], r=s.get("r"), keep=c["keep"])
            return (h, z) if c["keep"] else h
        if c["op"] == "ffn_grad":
            dx, dz = q4.gated_ffn_grad(s["gate"], s["up"], s["z"], s["dh"], act=c["act"], keep=c["keep"])
            return (dx, dz) if c["keep"] else dx
        if c["op"] == "distill":
            got = q4.lmhead_distill(s["w"], s["x"], s["ids"], s["logits"], temperature=c["temp"], dloss=s["dloss"],
                                    grad=c["grad"])
            return got if c["grad"] else got[:2]
        return q4.verify_draft(s["logits"], s["draft"], s["u"], probs=s["probs"], lens=s["lens"],
                               temperature=c["temp"])
    if c["op"] == "ffn":
        return _plain_ffn(s["gate"], s["up"], s["x"], s.get("r"), c["act"], c["keep"])
    if c["op"] == "ffn_grad":
        return _plain_ffn_grad(s["gate"], s["up"], s["z"], s["dh"], c["act"], c["keep"])
    if c["op"] == "distill":
        return _plain_distill(s["w"], s["x"], s["ids"], s["logits"], c["temp"], s["dloss"], c["grad"])
    return _plain_verify(s["logits"], s["draft"], s["u"], s["probs"], s["lens"], c["temp"])


def work(case):
    e, n = TYPES[case["type"]].itemsize, case["n"]
    if case["op"] == "verify":
        rows = case["s"] * (case["d"] + 1)
        # every row of the target, and the draft's row where a token is drawn from what is left
        drafts = case["s"] if case["probs"] and case["d"] else 0
        return {"bytes": (rows + drafts) * n * e + rows * 12 + case["s"] * 8, "flops": 2 * (rows + drafts) * n}
    m, k = case["m"], case["k"]
    if case["op"] == "distill":
        g = 1 if case["grad"] else 0
        return {"bytes": n * k * 18 // 32 + m * (k * e * (1 + g) + 8 + 4 * g + 8 * case["top"]),
                "flops": 2 * m * n * k * (1 + g)}
    width = {"ffn": 1 + (2 if case["keep"] else 0) + (2 if case.get("res") else 0),
             "ffn_grad": 3 + (2 if case["keep"] else 0)}[case["op"]]
    return {"bytes": 2 * n * k * 18 // 32 + m * (k + width * n) * e, "flops": 4 * m * n * k}


# ---------------------------------------------------------------- the definition in 64 bits

def _weights64(w):
    """float64 weights, a half block at a time through a table of the sixteen codes."""
    n = w.shape[0]
    blocks = w.reshape(n, -1, 18)
    codes = torch.arange(16, device=w.device, dtype=torch.float64) - 8
    scale = blocks[:, :, 0:2].contiguous().view(torch.float16).double()
    out = torch.empty((n, blocks.shape[1], 32), dtype=torch.float64, device=w.device)
    packed = blocks[:, :, 2:].int()
    out[:, :, :16] = codes[packed % 16] * scale
    out[:, :, 16:] = codes[packed // 16] * scale
    return out.reshape(n, -1)


def _gate64(g, act):
    """act(g) / g and act'(g), from the sigmoid that both activations are (gelu's tanh form is
    g * sigmoid(2 a))."""
    if act == "silu":
        s = torch.sigmoid(g)
        return s, s + g * s * torch.sigmoid(-g)
    a = 2 * (2 / math.pi) ** 0.5 * g * (1 + 0.044715 * g ** 2)
    s = torch.sigmoid(a)
    return s, s + g * s * torch.sigmoid(-a) * 2 * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    s, n = prepare(case, seed), case["n"]
    if case["op"] == "ffn":
        z = s["x"].double() @ torch.cat([_weights64(s["gate"]), _weights64(s["up"])]).t()
        if case["res"]:
            z += s["r"].double()
        g, u = z.split(n, 1)
        h = g * u * _gate64(g, case["act"])[0]
        return (h, z) if case["keep"] else h
    if case["op"] == "ffn_grad":
        g, u = s["z"].double().split(n, 1)
        share, slope = _gate64(g, case["act"])
        dz = torch.cat([u * slope, g * share], 1) * s["dh"].double().repeat(1, 2)
        dx = dz @ torch.cat([_weights64(s["gate"]), _weights64(s["up"])])
        return (dx, dz) if case["keep"] else dx
    if case["op"] == "distill":
        w, x, temp = _weights64(s["w"]), s["x"].double(), case["temp"]
        logp = torch.log_softmax(x @ w.t() / temp, 1)
        lse = torch.logsumexp(x @ w.t() / temp, 1)
        absent = (s["ids"] < 0) | (s["ids"] >= n)
        used = (~absent).any(1)
        idx = s["ids"].clamp(0, n - 1).long()
        b = (s["logits"].double() / temp).masked_fill(absent, -1e300)
        logq = torch.log_softmax(b, 1)
        q = logq.exp().masked_fill(absent | ~used[:, None], 0)
        loss = temp ** 2 * (q * (logq.masked_fill(absent, 0) - logp.gather(1, idx))).sum(1)
        if not case["grad"]:
            return loss, lse
        p = logp.exp_()
        for j in range(case["top"]):
            p[torch.arange(case["m"], device=x.device), idx[:, j]] -= q[:, j]
        return loss, lse, (p * (temp * s["dloss"].double() * used)[:, None]) @ w
    tokens = torch.full((case["s"], case["d"] + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(case["s"], dtype=torch.int32)
    draft, u = s["draft"].tolist(), s["u"].double().tolist()
    lens = s["lens"].tolist() if s["lens"] is not None else [case["d"]] * case["s"]
    for i in range(case["s"]):
        for j in range(case["d"] + 1):
            l = s["logits"][i, j].double()
            if case["temp"] == 0:
                p = torch.zeros_like(l)
                p[(l == l.max()).nonzero()[0]] = 1
            else:
                p = torch.softmax(l / case["temp"], 0)
            if j == lens[i]:
                break
            t = draft[i][j]
            q = torch.zeros_like(p)
            if s["probs"] is None:
                q[t] = 1
            else:
                q = s["probs"][i, j].double()
            if not u[i][j] * float(q[t]) < float(p[t]):
                rest = torch.where(p > q, p - q, 0)
                p = rest if float(rest.sum()) > 0 else p
                break
            tokens[i, j] = t
            accepted[i] += 1
        c = torch.cumsum(p, 0)
        new = torch.searchsorted(c, u[i][case["d"]] * float(c[-1]), right=True)
        tokens[i, int(accepted[i])] = min(int(new), n - 1)
    return tokens.to(s["logits"].device), accepted.to(s["logits"].device)
