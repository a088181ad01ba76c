"""gated_ffn_grad with rows that go through tiles of 48 (33 to 48, 65 to 96, 129 to 144 of
float32 and float16): whole tiles, and tiles whose last block of 16 rows is cut or empty.
References and tolerances are test_gpu_gated's."""

import pytest
import torch

import q4_quantized_speech_amd as q4
import test_gpu_gated as G
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16 = torch.float32, torch.float16


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("m", [33, 40, 47, 48, 65, 76, 81, 96, 130, 144])
def test_gradient_in_tiles_of_48_rows(m, dtype):
    for n, k in ((70, 160), (600, 96)):
        qg, wg = G.weights(n, k, 11)
        qu, wu = G.weights(n, k, 12)
        gen = torch.Generator(device="cuda").manual_seed(m)
        z = torch.randn((m, 2 * n), device="cuda", generator=gen).to(dtype)
        d = torch.randn((m, n), device="cuda", generator=gen).to(dtype)
        announce(f"gated_ffn_grad {m}x{n}x{k} {dtype}")
        dx, dz = q4.gated_ffn_grad(qg, qu, z, d, keep=True)
        torch.cuda.synchronize()
        want, tol, wz, tz = G.gradient(wg, wu, z, d, "silu", dtype)
        G.assert_close(dz, wz, tz, "dz")
        G.assert_close(dx, want, tol, "dx")
        # zero rows after them fill the last tile
        full = (m + 47) // 48 * 48
        if full > m:
            pad = torch.zeros((full - m, 1), device="cuda", dtype=dtype)
            more = q4.gated_ffn_grad(qg, qu, torch.cat([z, pad.expand(-1, 2 * n)]).contiguous(),
                                     torch.cat([d, pad.expand(-1, n)]).contiguous())[0]
            G.assert_close(more[:m], want, tol, "dx of the first rows")
            assert (more[m:] == 0).all()
