"""Host-side refusals of a draft model's operators (gated_ffn, gated_ffn_grad,
lmhead_distill, verify_draft): every bad argument is rejected before any HIP call, so
these run without a GPU."""

import os

import pytest
import torch

import q4_quantized_speech_amd as q4

pytestmark = pytest.mark.skipif(not os.path.exists(q4.LIB_PATH), reason="libq4mi.so not built")

A = 0x10000  # fake, 16-byte aligned, never dereferenced: validation fails first
BIG = 1 << 40


def _call(fn, base, **change):
    return getattr(q4.lib(), fn)(*dict(base, **change).values())


def _need(fn, *args):
    return int(getattr(q4.lib(), fn + "_workspace_bytes")(*args))


FFN = dict(gate=A, up=A, x=A, r=A, h=A, z=A, act=0, type=0, M=80, N=64, K=64, ws=A, ws_bytes=BIG, stream=None)
GRAD = dict(gate=A, up=A, z=A, dh=A, dx=A, dz=A, act=0, type=0, M=4, N=64, K=64, ws=A, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("fn,base,required,optional", [
    ("q4_gated_ffn", FFN, ("gate", "up", "x", "h"), ("r", "z")),
    ("q4_gated_ffn_grad", GRAD, ("gate", "up", "z", "dh"), ("dx", "dz"))])
def test_gated_refusals(fn, base, required, optional):
    for name in required:
        assert _call(fn, base, **{name: None}) == q4.Q4_ERR_NULL, name
    for name in required + optional + ("ws",):
        assert _call(fn, base, **{name: A + 8}) == q4.Q4_ERR_ALIGN, name
    for t in (2, 8, -1, 31):
        assert _call(fn, base, type=t) == q4.Q4_ERR_FORMAT
        assert _need(fn, t, 80, 64, 64) == 0
    for act in (-1, 2):
        assert _call(fn, base, act=act) == q4.Q4_ERR_FORMAT
    for bad in (dict(M=0), dict(M=(1 << 20) + 1), dict(N=0), dict(N=(1 << 21) + 1), dict(K=0), dict(K=48),
                dict(K=1 << 23), dict(M=1 << 20, K=1 << 13), dict(M=1 << 20, N=1 << 13),
                dict(N=1 << 21, K=1 << 12)):
        assert _call(fn, base, **bad) == q4.Q4_ERR_SHAPE, bad
        m, n, k = (dict(base, **bad)[v] for v in "MNK")
        assert _need(fn, 0, m, n, k) == 0, bad
    for t in (0, 1, 30):
        need = _need(fn, t, base["M"], 64, 64)
        assert need > 0
        assert _call(fn, base, type=t, ws_bytes=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _call(fn, base, ws=None) == q4.Q4_ERR_WORKSPACE


def test_gated_grad_needs_an_output():
    assert _call("q4_gated_ffn_grad", GRAD, dx=None, dz=None) == q4.Q4_ERR_NULL


def test_gated_binding_refusals():
    w = torch.zeros((8, 36), dtype=torch.uint8)
    x, h, z = torch.zeros(4, 64), torch.zeros(4, 8), torch.zeros(4, 16)
    for bad in (dict(w_up=w[:4]), dict(w_up=w[:, :18].contiguous()), dict(w_gate=w[:, ::2]), dict(x=x[0]),
                dict(x=x[:, :32]), dict(x=x.double()), dict(r=h), dict(r=z.half()), dict(out=z), dict(z=h),
                dict(act="relu"), dict(act=0), dict(workspace=x), {}):
        with pytest.raises(ValueError):
            q4.gated_ffn(**{**dict(w_gate=w, w_up=w, x=x), **bad})   # the last: CPU tensors
    for bad in (dict(z=h), dict(z=z[0]), dict(z=z.double()), dict(dh=z), dict(dh=h.half()), dict(dx=h),
                dict(dz=h), dict(dz=z.bfloat16()), dict(act="gelu_new"), {}):
        with pytest.raises(ValueError):
            q4.gated_ffn_grad(**{**dict(w_gate=w, w_up=w, z=z, dh=h), **bad})


DISTILL = dict(w=A, x=A, ids=A, logits=A, temperature=1.0, dloss=A, loss=A, lse=A, dx=A, type=0, M=4, N=64, K=64,
               top=8, ws=A, ws_bytes=BIG, stream=None)


def test_distill_refusals():
    fn = "q4_lmhead_distill"
    for name in ("w", "x", "ids", "logits", "loss", "lse"):
        assert _call(fn, DISTILL, **{name: None}) == q4.Q4_ERR_NULL, name
    for name in ("w", "x", "ids", "logits", "dloss", "loss", "lse", "dx", "ws"):
        assert _call(fn, DISTILL, **{name: A + 4}) == q4.Q4_ERR_ALIGN, name
    for t in (2, 8, -1, 31):
        assert _call(fn, DISTILL, type=t) == q4.Q4_ERR_FORMAT
        assert _need(fn, t, 1, 4, 64, 64, 8) == 0
    for bad in (dict(M=0), dict(M=65537), dict(N=0), dict(N=1 << 31), dict(K=0), dict(K=40), dict(K=1 << 23),
                dict(N=1 << 30, K=32), dict(M=65536, K=1 << 18), dict(top=0), dict(top=257), dict(top=-1)):
        assert _call(fn, DISTILL, **bad) == q4.Q4_ERR_SHAPE, bad
        v = dict(DISTILL, **bad)
        assert _need(fn, 0, 1, v["M"], v["N"], v["K"], v["top"]) == 0, bad
    for t in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 61, 2.0 ** -61):
        assert _call(fn, DISTILL, temperature=t) == q4.Q4_ERR_SHAPE, t
    for grad in (0, 1):
        need = _need(fn, 0, grad, 4, 64, 64, 8)
        assert need > 0
        assert _call(fn, DISTILL, dx=A if grad else None, ws_bytes=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _call(fn, DISTILL, ws=None) == q4.Q4_ERR_WORKSPACE


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("m,n,k", [(1, 1 << 28, 32), (64, 1 << 26, 128), (65, 1 << 20, 4096), (32768, 131072, 1280)])
def test_distill_workspace_is_the_losses_and_the_teachers(m, n, k, grad):
    xent = _need("q4_lmhead_xent", 0, grad, m, n, k)
    need = _need("q4_lmhead_distill", 0, grad, m, n, k, 256)
    if grad or m > 16:  # without a gradient few rows of a loss against targets go another way
        assert xent < need <= xent + 4 * (4 * 256 + 1) * m + 5 * 256
    assert 0 < need


def test_distill_binding_refusals():
    w = torch.zeros((8, 36), dtype=torch.uint8)
    x, ids, l = torch.zeros(4, 64), torch.zeros((4, 3), dtype=torch.int32), torch.zeros(4, 3)
    for bad in (dict(x=x[0]), dict(x=x[:, :32]), dict(x=x.double()), dict(top_ids=ids.long()), dict(top_ids=ids[0]),
                dict(top_ids=ids[:3]), dict(top_ids=ids[:, ::2]), dict(top_logits=l[:, :2]), dict(top_logits=l.half()),
                dict(dloss=torch.zeros(3)), dict(loss=torch.zeros(4).half()), dict(dx=x.half()),
                dict(lse=torch.zeros(4, 1)), {}):
        with pytest.raises(ValueError):
            q4.lmhead_distill(**{**dict(w_q4=w, x=x, top_ids=ids, top_logits=l), **bad})


VERIFY = dict(logits=A, draft=A, probs=A, u=A, lens=A, temperature=1.0, tokens=A, accepted=A, type=0, S=3, D=2,
              N=100, ws=A, ws_bytes=BIG, stream=None)


def test_verify_refusals():
    fn = "q4_verify_draft"
    for name in ("logits", "draft", "u", "tokens", "accepted"):
        assert _call(fn, VERIFY, **{name: None}) == q4.Q4_ERR_NULL, name
    for name in ("logits", "draft", "probs", "u", "lens", "tokens", "accepted", "ws"):
        assert _call(fn, VERIFY, **{name: A + 4}) == q4.Q4_ERR_ALIGN, name
    for t in (2, 8, -1, 31):
        assert _call(fn, VERIFY, type=t) == q4.Q4_ERR_FORMAT
    for bad in (dict(S=0), dict(S=(1 << 20) + 1), dict(D=-1), dict(D=64), dict(N=0), dict(N=1 << 31),
                dict(S=1 << 20, N=1 << 20), dict(S=1 << 10, D=63, N=1 << 24)):
        assert _call(fn, VERIFY, **bad) == q4.Q4_ERR_SHAPE, bad
        v = dict(VERIFY, **bad)
        assert _need(fn, v["S"], v["D"], v["N"]) == 0, bad
    for t in (-1.0, float("nan"), float("inf"), 2.0 ** 61, 2.0 ** -61):
        assert _call(fn, VERIFY, temperature=t) == q4.Q4_ERR_SHAPE, t
    need = _need(fn, 3, 2, 100)
    assert need > 0
    assert _call(fn, VERIFY, ws_bytes=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _call(fn, VERIFY, ws=None) == q4.Q4_ERR_WORKSPACE


def test_verify_binding_refusals():
    l, t, u = torch.zeros(3, 3, 10), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, 3)
    for bad in (dict(logits=l[0]), dict(logits=l.double()), dict(logits=l[:, :, ::2]), dict(logits=l[:, :0]),
                dict(draft=t.long()), dict(draft=t[:, :1]), dict(u=u[:, :2]), dict(u=u.half()),
                dict(probs=torch.zeros(3, 2, 9)), dict(probs=torch.zeros(3, 3, 10)),
                dict(probs=torch.zeros(3, 2, 10).half()), dict(lens=torch.zeros(3, dtype=torch.int64)),
                dict(lens=torch.zeros(2, dtype=torch.int32)), dict(tokens=t), dict(accepted=u), {}):
        with pytest.raises(ValueError):
            q4.verify_draft(**{**dict(logits=l, draft=t, u=u), **bad})
