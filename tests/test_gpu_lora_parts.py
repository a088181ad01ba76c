"""The adapters' products are made of bfloat16 parts of their factors: values whose parts
are as large as truncation leaves them, one product at a time, so that a part product left
out shows.

v = 1 + 2^-7 - 2^-23 has the parts 1, 2^-7 - 2^-15, 2^-15 - 2^-23.  Bounds, derived before
any run (u = 2^-24, half a step of float32):
  float32 results  one product v v and sums with zeros: the rounding of the last sum (u), the
                   roundings of the small sums before it (2^-6 u each, at most eight), the
                   dropped product of the two smallest parts (2^-30), the residual's sum
                   (exact here: zeros): 2 u v v.
  16-bit results   the same, with a residual that leaves only the last bits of the result,
                   so that its own rounding is that of a small number: 2 u v and the
                   smallest step of the type."""

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24
V = 1 + 2.0 ** -7 - 2.0 ** -23


def one_hot(m, n, k, r, na, dtype, atype):
    """x, dy, a, b, ids with a single nonzero per row of x and dy and a single rank in use."""
    x, dy = torch.zeros((m, k), device="cuda", dtype=dtype), torch.zeros((m, n), device="cuda", dtype=dtype)
    a = torch.zeros((na, r, k), device="cuda", dtype=atype)
    b = torch.zeros((na, n, r), device="cuda", dtype=atype)
    return x, dy, a, b, torch.arange(m, device="cuda", dtype=torch.int32) % na


@pytest.mark.parametrize("m,na", [(3, 1), (40, 2), (300, 2)])
@pytest.mark.parametrize("atype", [F32, F16, BF16])
def test_float32(m, na, atype):
    n, k, r = 70, 64, 16
    va = float(torch.tensor(1 + 2.0 ** -7 - 2.0 ** -10).to(atype)) if atype != F32 else V
    for first in (True, False):  # the product with many bits is A x (B^T dy), or the one after it
        x, dy, a, b, ids = one_hot(m, n, k, r, na, F32, atype)
        x[:, 5], dy[:, 7] = (V, V)
        a[:, 3, 5] = va if first else 1.0
        b[:, 7, 3] = 1.0 if first else va
        announce(f"lora parts {m} adapters {na} {atype} first={first}")
        y = q4.lora(x, a, b, ids)[:, 7].double()
        # the exact product, or that of the rounded rank vector: A x is kept in float32
        want = V * va if first else float(torch.tensor(V)) * va
        assert ((y - want).abs() <= 2 * U * want).all(), float(((y - want) / want / U).abs().max())
        a[:, 3, 5] = 1.0 if first else va
        b[:, 7, 3] = va if first else 1.0
        dx = q4.lora_grad(x, dy, a, b, ids)[0][:, 5].double()
        assert ((dx - want).abs() <= 2 * U * want).all(), float(((dx - want) / want / U).abs().max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("m", [40, 300])
def test_rank_vectors_of_16_bit_results(m, dtype):
    """The residual takes all but the last bits of the result away, so its rounding is small."""
    n, k, r, na = 72, 64, 16, 2
    x, dy, a, b, ids = one_hot(m, n, k, r, na, dtype, F32)
    x[:, 5], dy[:, 7] = 1.0, 1.0
    a[:, 3, 5], b[:, 7, 3] = V, 1.0
    res = torch.zeros((m, n), device="cuda", dtype=dtype)
    res[:, 7] = -(1 + 2.0 ** -7)  # V - 1 - 2^-7 = -2^-23
    step = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    announce(f"rank vectors {m} {dtype}")
    y = q4.lora(x, a, b, ids, r=res)[:, 7].double()
    assert ((y + 2.0 ** -23).abs() <= 2 * U * V + step).all(), float(y.abs().max()) / U
    a[:, 3, 5], b[:, 7, 3] = 1.0, V
    res = torch.zeros((m, k), device="cuda", dtype=dtype)
    res[:, 5] = -(1 + 2.0 ** -7)
    dx = q4.lora_grad(x, dy, a, b, ids, r=res)[0][:, 5].double()
    assert ((dx + 2.0 ** -23).abs() <= 2 * U * V + step).all(), float(dx.abs().max()) / U
