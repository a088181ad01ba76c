"""matmul_dx where neighbouring terms nearly cancel: the result is small beside its terms, so
its own rounding hides nothing of a weight's.

Rows of W come in pairs with the same codes and block scales one binary16 step apart, rows of
dy in pairs (g, -g).  Tolerance, derived before any run (u = 2^-24; B = the sum of the terms'
magnitudes): N u B for the float32 sum of N products, + 2^-20 B for the operands (two binary16
parts: exact weights, dy to 2^-22 or, in 16 bits, exact), + 2^-39 max|dy| sum|w| for values
far below their row's largest, + half a step of the result.  A weight rounded to 11 bits is
off by up to 2^-11 of a term, 2^9 times the second."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24


def paired(n, k, g):
    """2 n rows of Q4_0, pairs one step of the scale apart, and their float64 values."""
    codes = torch.randint(0, 256, (n, k // 32, 16), device="cuda", generator=g, dtype=torch.uint8)
    d = (torch.rand((n, k // 32, 1), device="cuda", generator=g) * 0.02 + 0.01).half()
    raw = torch.empty((n, 2, k // 32, 18), dtype=torch.uint8, device="cuda")
    raw[..., 2:] = codes.unsqueeze(1)
    q = torch.cat([codes & 15, codes >> 4], dim=2).double() - 8
    w = torch.empty((n, 2, k), device="cuda", dtype=torch.float64)
    for i in range(2):
        di = (d.view(torch.int16) + i).view(torch.float16)
        raw[:, i, :, :2] = di.view(torch.uint8).view(n, k // 32, 2)
        w[:, i] = (q * di.double()).reshape(n, k)
    return raw.view(2 * n, -1), w.view(2 * n, k)


def check(m, n, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    wq, w = paired(n, k, g)
    half = torch.randn((m, n, 1), device="cuda", generator=g).to(dtype)
    dy = torch.cat([half, -half], dim=2).view(m, 2 * n).contiguous()
    announce(f"dx {m}x{2 * n}x{k} {dtype}")
    got = q4.matmul_dx(wq, dy).double()
    d = dy.double()
    want, b = d @ w, d.abs() @ w.abs()
    f = torch.finfo(dtype)
    tol = (2 * n * U + 2.0 ** -20) * b + 2.0 ** -39 * d.abs().amax(1, keepdim=True) * w.abs().sum(0)
    tol += f.eps / 2 * want.abs() * (1 + 2.0 ** -10) + f.tiny * f.eps
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (5, 7, 96), (16, 40, 128), (31, 100, 160), (64, 33, 288), (300, 20, 416)])
def test_exact_weights(m, n, k, dtype):
    check(m, n, k, dtype)
