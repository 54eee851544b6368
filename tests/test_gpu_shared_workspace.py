"""One workspace for quant_scaled_mm and scaled_mm calls of any shapes: the
arrival counters at its head stay zero, wherever a call keeps its codes."""
import numpy as np
import pytest
import torch

import int8_w8a8_scaled_gb300 as w8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shapes", [[(64, 512, 512)], [(5, 1024, 2048), (300, 768, 512), (64, 512, 512)]])
def test_quantising_matmuls_leave_the_counters_zero(shapes):
    gen = torch.Generator(device="cuda").manual_seed(1)
    ws = w8.Workspace()
    for M, N, K in shapes:
        x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
        wq = torch.randint(0, 120, (N, K), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
        one = torch.ones(1, device="cuda")
        w8.quant_scaled_mm(x, wq, one, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), workspace=ws, route="two_step")
    assert not ws.buf[:65536].any()
    # CTA pairs whose last round runs as K halves, which meet on the counters
    M, N, K = 1280, 4096, 1040
    cfg = {"swap_ab": 0, "block_n": 256, "split_k": 2, "cta_pair": 1}
    a, b = (torch.from_numpy(np.random.default_rng(i).integers(0, 120, (r, K)).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
            for i, r in ((0, M), (1, N)))
    outs = []
    for space in (ws, w8.Workspace()):
        out = torch.full((M, N), float("nan"), dtype=torch.float32, device="cuda")
        w8.scaled_mm(a, b, one, one, out, workspace=space, config=cfg)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
