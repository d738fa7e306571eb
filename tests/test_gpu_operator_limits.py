"""Calls at the ends of the ranges that the operators take."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
def test_combine_rows_of_more_tokens_than_a_launch_takes(k, out_dtype):
    N = (1 << 23) + 5
    rows = torch.randn(1000, 8, device="cuda").to(BF)
    at = (torch.arange(N * k, device="cuda") * 7919 % 1009).to(torch.int32)   # 1000 to 1008 are no rows
    at = torch.where(at < 1000, at, -1).to(torch.int32)
    padded = torch.cat([rows.float(), torch.zeros(1, 8, device="cuda")])
    want = padded[at.view(N, k).long()].sum(dim=1) if k == 1 else padded[at.view(N, k)[:, 0].long()] + padded[at.view(N, k)[:, 1].long()]
    for out in (None, torch.empty(N, 8, dtype=out_dtype, device="cuda")):
        got = moe.combine_rows(rows, at, k, out=out, out_dtype=out_dtype)
        assert got.shape == (N, 8) and torch.equal(got, want.to(out_dtype))   # one addition: exact in fp32 before its one rounding


def test_dispatch_rows_of_more_pairs_than_an_index_holds():
    # 2^27 tokens of 16 slots: pairs up to 2^31 - 1 can be named
    N, k = 1 << 27, 16
    x = torch.arange(N, dtype=torch.int32, device="cuda").to(torch.uint8).view(N, 1)
    pair = torch.tensor([0, 15, 16, 1 << 30, (1 << 31) - 1, -1], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    got = moe.dispatch_rows(x, pair, off, k)
    want = torch.tensor([0, 0, 1, (1 << 26) % 256, (N - 1) % 256, 0], dtype=torch.uint8, device="cuda").view(6, 1)
    assert torch.equal(got, want)


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
