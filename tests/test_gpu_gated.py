"""The gated feed-forward block (gated_ffn) and its gradient (gated_ffn_grad)
against float64 forms on the oracle's decoded weights.

Tolerances, derived before any run (u = 2^-24, half a float32 step; B = the sum of
the terms' magnitudes):
  g, u    t = (K + 64) u B + 2^-20 B (float32 sums; operands as two binary16 parts)
          + 2^-38 max|x| sum|w| for values far below their row's largest.
  act     1.13 t (the slopes' largest) + (16 + 8 A) u |act|, A the magnitude of the
          sigmoid's argument: its relative rounding is an absolute one in the
          exponent.
  h       |u| e_act + (|act| + e_act) t_u + 4 u |h|, + half a step of the output.
  dg, du  the slope's error is (16 + 8 A) u (s + |g s (1 - s) a'|); 4 u of the products,
          + half a step for dz.
  dx      (2 N u + c) sum |dz| |w|, c = 2^-20 for float32, 2^-11 where dz is one
          binary16 part, + the sum of the errors of dz times |w|,
          + 2^-32 max|dh| max|z| sum|w|, + half a step."""

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


def weights(n, k, seed):
    """(bytes on the GPU, float64 weights on the GPU)."""
    qb = O.quantize_q4_0(synth.weights(n, k, seed))
    return torch.from_numpy(qb).cuda(), torch.from_numpy(O.dequantize_q4_0(qb, n, k)).double().cuda()


def half_step(dtype, want):
    f = torch.finfo(dtype)
    return f.eps / 2 * want.abs() * (1 + 2.0 ** -10) + f.tiny * f.eps


def assert_close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(0.0).max()))


def gate(g, act):
    """(A, s, act, act') of float64 g, from the definitions."""
    if act == "silu":
        a, da = g, torch.ones_like(g)
    else:
        c = (2 / np.pi) ** 0.5
        a, da = 2 * c * (g + 0.044715 * g ** 3), 2 * c * (1 + 3 * 0.044715 * g ** 2)
    s, rest = torch.sigmoid(a), torch.sigmoid(-a)
    turn = g * s * rest * da
    return a.abs(), s, g * s, s + turn, s.abs() + turn.abs()


def forward(wg, wu, x, r, act, dtype):
    x6, n, k = x.double(), wg.shape[0], wg.shape[1]
    out = []
    for j, w in enumerate((wg, wu)):
        v, b = x6 @ w.t(), x6.abs() @ w.abs().t()
        if r is not None:
            v, b = v + r[:, j * n:(j + 1) * n].double(), b + r[:, j * n:(j + 1) * n].double().abs()
        t = (k + 64) * U * b + 2.0 ** -20 * b + 2.0 ** -38 * x6.abs().amax(1, keepdim=True) * w.abs().sum(1)
        out += [v, t]
    g, tg, u, tu = out
    a, _, f, _, _ = gate(g, act)
    ef = 1.13 * tg + (16 + 8 * a) * U * f.abs()
    h = f * u
    th = u.abs() * ef + (f.abs() + ef) * tu + 4 * U * h.abs()
    z, tz = torch.cat([g, u], 1), torch.cat([tg, tu], 1)
    return h, th + half_step(dtype, h.abs() + th), z, tz + half_step(dtype, z.abs() + tz)


def inputs(m, n, k, dtype, seed, r):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, k), device="cuda", generator=gen)
    x *= 10.0 ** torch.empty((m, 1), device="cuda").uniform_(-2, 1, generator=gen)
    res = torch.randn((m, 2 * n), device="cuda", generator=gen).to(dtype) if r else None
    return x.to(dtype), res


SHAPES = [(1, 1, 32), (1, 40, 64), (2, 16, 96), (3, 33, 128), (4, 100, 160), (5, 17, 1280), (8, 47, 224),
          (9, 130, 3072), (16, 250, 1056), (17, 31, 64), (32, 97, 320), (33, 48, 1280), (48, 63, 32),
          (49, 200, 416), (64, 129, 1024), (65, 33, 32), (66, 300, 352), (130, 65, 1280), (257, 520, 96)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward_shapes(m, n, k, dtype):
    for act, r in (("silu", m % 2 == 0), ("gelu", m % 2 == 1)):
        qg, wg = weights(n, k, 10 * m + 1)
        qu, wu = weights(n, k, 10 * m + 2)
        x, res = inputs(m, n, k, dtype, m + n, r)
        announce(f"gated_ffn {m}x{n}x{k} {dtype} {act} r={r}")
        h, z = q4.gated_ffn(qg, qu, x, act=act, r=res, keep=True)
        torch.cuda.synchronize()
        want, tol, wz, tz = forward(wg, wu, x, res, act, dtype)
        assert_close(z, wz, tz, "z")
        assert_close(h, want, tol, "h")
        h2, none = q4.gated_ffn(qg, qu, x, act=act, r=res)
        assert none is None and torch.equal(h, h2)


@pytest.mark.parametrize("m,n,k,dtype", [(1, 9216, 3072, F32), (7, 9216, 3072, BF16), (38, 9216, 3072, F32),
                                         (76, 9216, 3072, F16), (375, 5120, 1280, F32), (1500, 5120, 1280, BF16)])
def test_forward_model_shapes(m, n, k, dtype):
    qg, wg = weights(n, k, 7)
    qu, wu = weights(n, k, 8)
    x, _ = inputs(m, n, k, dtype, m, False)
    announce(f"gated_ffn {m}x{n}x{k} {dtype}")
    h, z = q4.gated_ffn(qg, qu, x, keep=True)
    torch.cuda.synchronize()
    want, tol, wz, tz = forward(wg, wu, x, None, "silu", dtype)
    assert_close(z, wz, tz, "z")
    assert_close(h, want, tol, "h")


def gradient(wg, wu, z, dh, act, dtype):
    n = wg.shape[0]
    g, u, d = z[:, :n].double(), z[:, n:].double(), dh.double()
    a, s, f, slope, mag = gate(g, act)
    dg, du = d * u * slope, d * f
    eg = (d * u).abs() * (16 + 8 * a) * U * mag + 4 * U * dg.abs()
    eu = d.abs() * (16 + 8 * a) * U * f.abs() + 4 * U * du.abs()
    c = 2.0 ** -20 if dtype == F32 else 2.0 ** -11
    dx = dg @ wg + du @ wu
    far = 2.0 ** -32 * d.abs().amax(1, keepdim=True) * z.double().abs().amax(1, keepdim=True)
    tx = ((2 * n * U + c) * dg.abs() + eg + far) @ wg.abs() + ((2 * n * U + c) * du.abs() + eu + far) @ wu.abs()
    dz, tz = torch.cat([dg, du], 1), torch.cat([eg, eu], 1)
    return dx, tx + half_step(dtype, dx.abs() + tx), dz, tz + half_step(dtype, dz.abs() + tz)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradient_shapes(m, n, k, dtype):
    for act in ("silu", "gelu"):
        qg, wg = weights(n, k, 20 * m + 1)
        qu, wu = weights(n, k, 20 * m + 2)
        gen = torch.Generator(device="cuda").manual_seed(m + k)
        z = (2 * torch.randn((m, 2 * n), device="cuda", generator=gen)).to(dtype)
        dh = torch.randn((m, n), device="cuda", generator=gen)
        # float16 gradients stay inside its range
        dh *= 10.0 ** torch.empty((m, 1), device="cuda").uniform_(-1 if dtype == F16 else -4, 0, generator=gen)
        dh = dh.to(dtype)
        announce(f"gated_ffn_grad {m}x{n}x{k} {dtype} {act}")
        dx, dz = q4.gated_ffn_grad(qg, qu, z, dh, act=act, keep=True)
        torch.cuda.synchronize()
        want, tol, wz, tz = gradient(wg, wu, z, dh, act, dtype)
        assert_close(dz, wz, tz, "dz")
        assert_close(dx, want, tol, "dx")
        dx2, none = q4.gated_ffn_grad(qg, qu, z, dh, act=act)
        assert none is None and torch.equal(dx, dx2)


@pytest.mark.parametrize("m,n,k,dtype", [(76, 9216, 3072, F32), (1500, 5120, 1280, BF16), (38, 9216, 3072, F16)])
def test_gradient_model_shapes(m, n, k, dtype):
    qg, wg = weights(n, k, 9)
    qu, wu = weights(n, k, 10)
    gen = torch.Generator(device="cuda").manual_seed(m)
    z = torch.randn((m, 2 * n), device="cuda", generator=gen).to(dtype)
    dh = (0.01 * torch.randn((m, n), device="cuda", generator=gen)).to(dtype)
    announce(f"gated_ffn_grad {m}x{n}x{k} {dtype}")
    dx, dz = q4.gated_ffn_grad(qg, qu, z, dh, keep=True)
    torch.cuda.synchronize()
    want, tol, wz, tz = gradient(wg, wu, z, dh, "silu", dtype)
    assert_close(dz, wz, tz, "dz")
    assert_close(dx, want, tol, "dx")
