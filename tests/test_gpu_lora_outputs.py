"""q4_lora_grad leaves out what the caller does not ask for: each subset of (dx, da, db) through
the C entry point gives the full call's bits, from a workspace of NaN."""

import itertools

import pytest
import torch

import q4_quantized_speech_amd as q4
from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: 0, F16: 1, BF16: 30}


@pytest.mark.parametrize("dtype,atype", [(F32, F32), (F32, F16), (F16, F16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("m,n,k,r,na", [(5, 70, 64, 8, 2), (90, 203, 160, 24, 3), (300, 136, 96, 40, 2), (700, 65, 320, 72, 3)])
def test_subsets(m, n, k, r, na, dtype, atype):
    g = torch.Generator(device="cuda").manual_seed(m + n)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    x, dy, res = rand(m, k).to(dtype), rand(m, n).to(dtype), rand(m, k).to(dtype)
    a, b, scale = (rand(na, r, k) * 0.1).to(atype), (rand(na, n, r) * 0.1).to(atype), rand(na)
    ids = torch.randint(-1, na, (m,), device="cuda", generator=g, dtype=torch.int32)
    want = q4.lora_grad(x, dy, a, b, ids, scale=scale, r=res)
    need = int(q4.lib().q4_lora_grad_workspace_bytes(m, n, k, r))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for some in itertools.product((False, True), repeat=3):
        if not any(some):
            continue
        announce(f"lora_grad outputs {some} {m}x{n}x{k} r={r} {dtype} {atype}")
        ws.fill_(255)
        out = [torch.full_like(w, float("nan")) for w in want]
        at = [o.data_ptr() if s else None for o, s in zip(out, some)]
        status = q4.lib().q4_lora_grad(x.data_ptr(), dy.data_ptr(), a.data_ptr(), b.data_ptr(), scale.data_ptr(),
                                       ids.data_ptr(), res.data_ptr(), *at, CODE[dtype], CODE[atype], m, n, k, r, na,
                                       ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert status == q4.Q4_OK
        torch.cuda.synchronize()
        for o, w, s in zip(out, want, some):
            assert torch.equal(o, w) if s else o.isnan().all()
