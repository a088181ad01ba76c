"""matmul_dx through unpacked weights, which few of its sizes take: very many rows of a small
matrix, or few rows of a very long one.  Tolerance as in the head's tests: N u B for the
float32 sum of N products, + 2^-20 B for the operands, + 2^-39 max|dy| sum|w|, + half a step
of the result (u = 2^-24, B the sum of the terms' magnitudes)."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: 0, F16: 1, BF16: 30}
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 43392), (3, 2, 131072), (60000, 70, 160), (61644, 76, 160), (60001, 64, 192),
                                   (65000, 109, 160)])
def test_unpacked(m, n, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + n)
    raw = torch.randint(0, 256, (n, k // 32, 18), device="cuda", generator=g, dtype=torch.uint8)
    d = (torch.rand((n, k // 32, 1), device="cuda", generator=g) * 0.01 + 0.001).half()
    raw[..., :2] = d.view(torch.uint8).view(n, k // 32, 2)
    q = torch.cat([raw[..., 2:] & 15, raw[..., 2:] >> 4], dim=2).double() - 8
    w = (q * d.double()).view(n, k)
    dy = (torch.randn((m, n), device="cuda", generator=g) * 0.1).to(dtype)
    need = int(q4.lib().q4_matmul_dx_workspace_bytes(CODE[dtype], m, n, k))
    # this route's: dy's operands, two parts of the weights and a float32 copy of the result
    assert need >= m * n * dy.element_size() + 4 * n * k + 4 * m * k
    announce(f"dx unpacked {m}x{n}x{k} {dtype}")
    got = q4.matmul_dx(raw.view(n, -1), dy)
    d6 = dy.double()
    want, b = d6 @ w, d6.abs() @ w.abs()
    f = torch.finfo(dtype)
    tol = (n * U + 2.0 ** -20) * b + 2.0 ** -39 * d6.abs().amax(1, keepdim=True) * w.abs().sum(0)
    tol += f.eps / 2 * want.abs() * (1 + 2.0 ** -10) + f.tiny * f.eps
    err = (got.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(q4.matmul_dx(raw.view(n, -1), dy), got)
