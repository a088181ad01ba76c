"""Host-side refusals of the operators that adapt a frozen Q4_0 model: every bad
argument is rejected before any HIP call, so these run without a GPU."""

import os

import pytest
import torch

import q4_quantized_speech_amd as q4

pytestmark = pytest.mark.skipif(not os.path.exists(q4.LIB_PATH), reason="libq4mi.so not built")

A = 0x10000  # fake, 16-byte aligned, never dereferenced: validation fails first
BIG = 1 << 40


def _call(fn, base, **change):
    args = dict(base, **change)
    return getattr(q4.lib(), fn)(*args.values())


LORA = dict(x=A, a=A, b=A, scale=A, ids=A, r=A, y=A, type=0, atype=0, M=4, N=64, K=64, R=8,
            adapters=2, ws=A, ws_bytes=BIG, stream=None)
GRAD = dict(x=A, dy=A, a=A, b=A, scale=A, ids=A, r=A, dx=A, da=A, db=A, type=0, atype=0, M=4, N=64,
            K=64, R=8, adapters=2, ws=A, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("fn,base,required,optional", [
    ("q4_lora", LORA, ("x", "a", "b", "ids", "y"), ("scale", "r")),
    ("q4_lora_grad", GRAD, ("x", "dy", "a", "b", "ids"), ("scale", "r", "dx", "da", "db"))])
def test_lora_refusals(fn, base, required, optional):
    for name in required:
        assert _call(fn, base, **{name: None}) == q4.Q4_ERR_NULL, name
    for name in required + optional + ("ws",):
        assert _call(fn, base, **{name: A + 4}) == q4.Q4_ERR_ALIGN, name
    for t in (2, 8, -1, 31):
        assert _call(fn, base, type=t) == q4.Q4_ERR_FORMAT
        assert _call(fn, base, atype=t) == q4.Q4_ERR_FORMAT
    assert _call(fn, base, type=1, atype=30) == q4.Q4_ERR_FORMAT
    assert _call(fn, base, type=30, atype=1) == q4.Q4_ERR_FORMAT
    for bad in (dict(M=0), dict(M=-1), dict(M=BIG), dict(N=0), dict(N=(1 << 22) + 1), dict(K=0),
                dict(K=48), dict(K=1 << 23), dict(R=0), dict(R=4), dict(R=12), dict(R=136),
                dict(adapters=0), dict(adapters=65536)):
        assert _call(fn, base, **bad) == q4.Q4_ERR_SHAPE, bad
    need = int(getattr(q4.lib(), fn + "_workspace_bytes")(4, 64, 64, 8))
    assert need > 0
    assert _call(fn, base, ws=None) == q4.Q4_ERR_WORKSPACE
    assert _call(fn, base, ws_bytes=need - 1) == q4.Q4_ERR_WORKSPACE
    assert int(getattr(q4.lib(), fn + "_workspace_bytes")(4, 64, 48, 8)) == 0


def test_lora_grad_needs_an_output():
    assert _call("q4_lora_grad", GRAD, dx=None, da=None, db=None) == q4.Q4_ERR_NULL
    # a workgroup per adapter and 64 columns
    assert _call("q4_lora_grad", GRAD, N=1 << 22, adapters=1000) == q4.Q4_ERR_SHAPE


def test_lora_binding_refusals():
    x, a, b = torch.zeros(4, 64), torch.zeros(2, 8, 64), torch.zeros(2, 32, 8)
    ids = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(x=x[:, ::2]), dict(x=x[0]), dict(x=x.double()), dict(a=a[:, :, :32]),
                dict(b=b.half()), dict(ids=ids.long()), dict(ids=ids[:3]),
                dict(scale=torch.zeros(3)), dict(scale=torch.zeros(2, dtype=torch.float16)),
                dict(r=torch.zeros(4, 33)), dict(out=torch.zeros(4, 32, dtype=torch.float16)),
                dict(workspace=torch.zeros(64)), {}):
        with pytest.raises(ValueError):
            q4.lora(**{**dict(x=x, a=a, b=b, ids=ids), **bad})   # the last: CPU tensors
    dy = torch.zeros(4, 32)
    for bad in (dict(dy=dy[:, :31]), dict(dy=dy.bfloat16()), dict(r=dy), dict(dx=dy),
                dict(da=torch.zeros(2, 8, 64).half()), dict(db=torch.zeros(2, 8, 32)), {}):
        with pytest.raises(ValueError):
            q4.lora_grad(**{**dict(x=x, dy=dy, a=a, b=b, ids=ids), **bad})


DX = dict(w=A, dy=A, dx=A, type=0, M=4, N=64, K=64, ws=A, ws_bytes=BIG, stream=None)
XENT = dict(w=A, x=A, targets=A, dloss=A, loss=A, lse=A, dx=A, type=0, M=4, N=64, K=64, ws=A,
            ws_bytes=BIG, stream=None)


def _need(fn, type=0, **change):
    a = dict(type=type, M=4, N=64, K=64, **({"grad": 1} if "xent" in fn else {}))
    a.update(change)
    order = (["type", "grad"] if "xent" in fn else ["type"]) + ["M", "N", "K"]
    return int(getattr(q4.lib(), fn + "_workspace_bytes")(*[a[k] for k in order]))


@pytest.mark.parametrize("fn,base,required,optional,shapes", [
    ("q4_matmul_dx", DX, ("w", "dy", "dx"), (),
     (dict(M=0), dict(M=(1 << 20) + 1), dict(N=0), dict(N=(1 << 22) + 1), dict(K=0), dict(K=40),
      dict(K=1 << 23), dict(M=1 << 20, K=1 << 14), dict(M=1 << 20, N=1 << 14), dict(N=1 << 22, K=1 << 12))),
    ("q4_lmhead_xent", XENT, ("w", "x", "targets", "loss", "lse"), ("dloss", "dx"),
     (dict(M=0), dict(M=65537), dict(N=0), dict(N=1 << 31), dict(K=0), dict(K=40), dict(K=1 << 23),
      dict(N=1 << 30, K=32), dict(M=65536, K=1 << 18)))])
def test_dx_and_xent_refusals(fn, base, required, optional, shapes):
    for name in required:
        assert _call(fn, base, **{name: None}) == q4.Q4_ERR_NULL, name
    for name in required + optional + ("ws",):
        assert _call(fn, base, **{name: A + 8}) == q4.Q4_ERR_ALIGN, name
    for t in (2, 8, -1, 31):
        assert _call(fn, base, type=t) == q4.Q4_ERR_FORMAT
        assert _need(fn, t) == 0
    for bad in shapes:
        assert _call(fn, base, **bad) == q4.Q4_ERR_SHAPE, bad
        assert _need(fn, **bad) == 0, bad
    for t in (0, 1, 30):
        need = _need(fn, t)
        assert need > 0
        assert _call(fn, base, type=t, ws_bytes=need - 1) == q4.Q4_ERR_WORKSPACE
    assert _call(fn, base, ws=None) == q4.Q4_ERR_WORKSPACE


def test_dx_and_xent_binding_refusals():
    w = torch.zeros((8, 36), dtype=torch.uint8)
    dy, x, t = torch.zeros(4, 8), torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(dy=dy[0]), dict(dy=dy[:, :7]), dict(dy=dy.double()), dict(out=torch.zeros(4, 63)),
                dict(out=x.half()), dict(w_q4=w[:, ::2]), {}):
        with pytest.raises(ValueError):
            q4.matmul_dx(**{**dict(w_q4=w, dy=dy), **bad})
    for bad in (dict(x=x[0]), dict(x=x[:, :32]), dict(x=x.double()), dict(targets=t.long()),
                dict(targets=t[:3]), dict(dloss=torch.zeros(3)), dict(loss=torch.zeros(4).half()),
                dict(dx=x.half()), dict(lse=torch.zeros(4, 1)), {}):
        with pytest.raises(ValueError):
            q4.lmhead_xent(**{**dict(w_q4=w, x=x, targets=t), **bad})


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("m,n,k", [(1, 1 << 28, 32), (1, 1 << 27, 64), (4, 1 << 27, 64), (3, 1 << 24, 512), (16, 1 << 24, 96),
                                   (64, 1 << 26, 128), (65, 1 << 20, 4096), (32768, 131072, 1280), (65536, 131072, 1280)])
def test_xent_workspace_holds_pieces(m, n, k, grad):
    """However large the table, the workspace holds pieces of at most 2^26 logits (2048 columns
    where a row's share is less) in float32 and as two parts, their maxima and sums per 64
    columns, a piece's unpacked weights (32768 rows) and x and dx a few times over."""
    logits = max(1 << 26, 2048 * m)
    most = logits * (8 if grad else 0) + logits // 4 * (0 if m <= 64 else 1) + 32768 * (k + 32) * 8 + 80 * m * k + (1 << 24)
    if not grad and m <= 64:
        most += logits * 4 + logits // 4  # a few rows may keep them all
    need = _need("q4_lmhead_xent", 0, grad=grad, M=m, N=n, K=k)
    assert 0 < need <= most, (need, most)
