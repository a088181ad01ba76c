"""The bits that gated_ffn_grad's products keep, which a result's own rounding hides.

Tolerances, derived before any run (u = 2^-24; B = sum |dz| |w|):
  cancelling sums  (2 N u + 2^-20) B and the slopes' errors, as test_gpu_gated derives
          them for operands of two binary16 parts, + half a step of the result, which is
          a few 2^-8 of its terms.  One part of dz is off by up to 2^-12 of each term.
  distance from the exact result rounded once, as a norm: an error of e relative to a
          value moves its rounding to a step of s = eps / 2 to eps with a chance of e / s,
          so its square is e s on average.  e is below 2^-20 (sums of float32 and
          two-part operands: some 2^-22) and s below eps: sqrt(2^-20 eps), and four
          times that as the bound; float32 itself: 2^-20 of the result."""

import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_gated as G
from gpu_util import announce, needs_gpu
from oracle import q4_oracle as O
from q4_quantized_speech_amd import synth

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def twin_rows(n, k, seed):
    """Weights whose rows 2 i and 2 i + 1 are alike: (bytes, float64)."""
    one = O.quantize_q4_0(synth.weights(n // 2, k, seed))
    w = torch.from_numpy(O.dequantize_q4_0(one, n // 2, k)).double()
    both = torch.from_numpy(one).view(n // 2, -1).repeat_interleave(2, 0).contiguous()
    return both.cuda(), w.repeat_interleave(2, 0).cuda()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(3, 8, 64), (20, 8, 96), (64, 8, 256), (130, 16, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gradient_of_sums_that_cancel(m, n, k, act, dtype):
    """Every unit has a twin with its weights, a gradient of the other sign and
    pre-activations a step away: what is left of dx is a few steps of its terms."""
    qg, wg = twin_rows(n, k, 1)
    qu, wu = twin_rows(n, k, 2)
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    step = torch.finfo(dtype).eps
    z = torch.randn((m, 2 * n), device="cuda", generator=gen)
    z[:, 1::2] = z[:, ::2] * (1 + step)
    d = torch.randn((m, n), device="cuda", generator=gen)
    d[:, 1::2] = -d[:, ::2]
    if dtype == F32:  # its own step would leave less than the tolerance
        z[:, 1::2] = z[:, ::2] * (1 + 2.0 ** -7)
    z, d = z.to(dtype), d.to(dtype)
    announce(f"gated_ffn_grad {m}x{n}x{k} {dtype} {act}")
    dx, _ = q4.gated_ffn_grad(qg, qu, z, d, act=act)
    torch.cuda.synchronize()
    want, tol, _, _ = G.gradient(wg, wu, z, d, act, F32)  # float32's: two parts
    tol = tol - G.half_step(F32, tol)
    G.assert_close(dx, want, tol + G.half_step(dtype, want.abs() + tol), "dx")


@pytest.mark.parametrize("m,n,k,act", [(16, 300, 512, "silu"), (64, 2000, 1024, "gelu"), (256, 1100, 1280, "silu")])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gradient_rounds_once(m, n, k, act, dtype):
    qg, wg = G.weights(n, k, 31)
    qu, wu = G.weights(n, k, 32)
    gen = torch.Generator(device="cuda").manual_seed(m)
    z = torch.randn((m, 2 * n), device="cuda", generator=gen).to(dtype)
    d = torch.randn((m, n), device="cuda", generator=gen).to(dtype)
    announce(f"gated_ffn_grad {m}x{n}x{k} {dtype} {act}")
    dx, _ = q4.gated_ffn_grad(qg, qu, z, d, act=act)
    torch.cuda.synchronize()
    want = G.gradient(wg, wu, z, d, act, dtype)[0]
    once = want.to(dtype).double()
    off = float((dx.double() - once).norm() / once.norm())
    bound = 2.0 ** -20 if dtype == F32 else 4 * (2.0 ** -20 * torch.finfo(dtype).eps) ** 0.5
    assert off <= bound, (off, bound)
