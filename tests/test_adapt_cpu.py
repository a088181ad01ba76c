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
