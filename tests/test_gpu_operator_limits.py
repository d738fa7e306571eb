"""Calls at the ends of the ranges that the operators take."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("k,n", [(33, 7), (264, 136)], ids=["odd", "aligned"])
def test_accumulation_leaves_experts_without_rows_to_the_bit(k, n, out_dtype):
    g = torch.Generator().manual_seed(4)
    off = torch.tensor([0, 0, 20, 20], dtype=torch.int32, device="cuda")
    x, dy = torch.randn(20, k, generator=g).to(BF).cuda(), torch.randn(20, n, generator=g).to(BF).cuda()
    old = torch.randn(3, n, k, generator=g).to(out_dtype)
    old[:, 0, 0], old[:, 1, 1], old[:, 2, 2] = -0.0, INF, NAN
    whole = torch.int16 if out_dtype == BF else torch.int32
    old.view(whole)[:, 3, 3] = 0x7F81 if out_dtype == BF else 0x7F800001   # a signalling NaN
    out = old.cuda()
    moe.grouped_matmul_wgrad(dy, x, off, out=out, accumulate=True)
    got = out.cpu()
    for e in (0, 2):
        assert torch.equal(got[e].view(whole), old[e].view(whole))
    assert got[1, 0, 0] != 0
