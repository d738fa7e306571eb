"""The weighted combination and its gradients with more tokens than one launch
takes (2^23), on whole numbers, whose sums and products are exact."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from test_gpu_operators import BF, F32, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("over", [False, True], ids=["out", "over_the_rows"])
def test_more_tokens_than_one_launch(over):
    N, k, H, g = (1 << 23) + 77, 2, 8, torch.Generator(device="cuda").manual_seed(1)
    whole = lambda lo, hi, *s, dt=BF: torch.randint(lo, hi, s, generator=g, device="cuda").to(dt)   # noqa: E731
    at = torch.full((N * k,), -1, dtype=torch.int32, device="cuda")
    pairs = torch.arange(1, N * k, 3, device="cuda")   # every third slot is local, and rows lie in another order
    R = pairs.numel()
    at[pairs] = torch.arange(R, dtype=torch.int32, device="cuda").flip(0)
    rows, dy, w = whole(-4, 5, R, H), whole(-4, 5, N, H), whole(-4, 5, N, k, dt=F32)
    here, r = (at >= 0).view(N, k, 1), at.long().clamp(min=0)
    z = torch.where(here, rows[r].view(N, k, H), 0)
    say("combine of many tokens")
    y = moe.combine_rows(rows, at, k, weights=w)
    assert torch.equal(y.float(), (z.float() * w[..., None]).sum(dim=1))
    want = torch.empty_like(rows)
    want[r[pairs]] = (w.view(-1)[pairs, None] * dy[pairs // k].float()).to(BF)
    wantw = (z.float() * dy[:, None].float()).sum(dim=2)
    say("combine's gradients of many tokens")
    got, dw = moe.combine_rows_backward(dy, rows, at, w, out=rows if over else torch.empty_like(rows))
    assert torch.equal(got, want) and torch.equal(dw, wantw) and (got is rows) == over
