"""gated_ffn_grad without dx: dz alone, with the bits it has beside dx, no workspace, on the
GPU; and its refusals, which come before any GPU call."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def test_refusals():
    w, z, h = torch.zeros((8, 36), dtype=torch.uint8), torch.zeros(4, 16), torch.zeros(4, 8)
    for bad in (dict(), dict(keep=True, dx=torch.zeros(4, 64)), dict(dz=z, dx=torch.zeros(4, 64))):
        with pytest.raises(ValueError, match="need_dx"):
            q4.gated_ffn_grad(w, w, z, h, need_dx=False, **bad)
    with pytest.raises(ValueError, match="GPU"):
        q4.gated_ffn_grad(w, w, z, h, need_dx=False, keep=True)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (7, 33, 64), (40, 300, 96), (130, 257, 128)])
def test_dz_alone(m, n, k, dtype, act):
    import test_gpu_gated as G
    qg, wg = G.weights(n, k, 51)
    qu, wu = G.weights(n, k, 52)
    gen = torch.Generator(device="cuda").manual_seed(m)
    z = (2 * torch.randn((m, 2 * n), device="cuda", generator=gen)).to(dtype)
    d = torch.randn((m, n), device="cuda", generator=gen).to(dtype)
    announce(f"gated_ffn_grad, dz alone {m}x{n}x{k} {dtype} {act}")
    none, dz = q4.gated_ffn_grad(qg, qu, z, d, act=act, keep=True, need_dx=False)
    torch.cuda.synchronize()
    assert none is None
    _, _, want, tol = G.gradient(wg, wu, z, d, act, dtype)
    G.assert_close(dz, want, tol, "dz")
    assert torch.equal(dz, q4.gated_ffn_grad(qg, qu, z, d, act=act, keep=True)[1])
    own = z.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _, same = q4.gated_ffn_grad(qg, qu, own, d, act=act, dz=own, need_dx=False, stream=st)
    st.synchronize()
    assert same is own and torch.equal(own, dz)
