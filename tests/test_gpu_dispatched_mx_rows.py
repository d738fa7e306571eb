"""Codes and scale bytes in microscaled (MX) formats dispatched to the experts'
rows into buffers that dispatch_rows allocates, at hidden sizes whose rows are no
whole 16 (scales: four) bytes: the products' tile kernels take them, and results
are those of rows in buffers of the caller's, to the bit."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from test_gpu_operators import BF, F8, gen, normal, offsets, say, up

pytestmark = pytest.mark.gpu


def layout(N, k, L, seed):
    """row_pair and row_offset of pairs drawn for L experts, a third of them for none."""
    e = torch.randint(0, L + L // 2, (N * k,), generator=gen(seed))
    order = torch.argsort(e, stable=True)
    counts = torch.bincount(e, minlength=L + L // 2)[:L].tolist()
    return up(order.int()), up(offsets(counts)), sum(counts)


@pytest.mark.parametrize("H", [72, 1000, 2880, 7200])
@pytest.mark.parametrize("element", ["e4m3", "e2m1"])
def test_allocated_rows_go_to_the_tile_kernels(element, H):
    N, k, L, n = 50, 4, 6, 136
    g = gen(H)
    pair, off, R = layout(N, k, L, H)
    x, wn = up(normal(g, N, H)), up(normal(g, H))
    w, ws = moe.quantize_mx(up(normal(g, L, n, H)), "e2m1")
    say(f"dispatched rows {H} {element}")
    for q, s in (moe.quantize_mx(x, element), moe.rms_norm(x, wn, quantize="mx_" + element)):
        qr, sr = moe.dispatch_rows(q, pair, off, k), moe.dispatch_rows(s, pair, off, k)
        assert qr.stride(0) % 16 == 0 and sr.stride(0) % 4 == 0
        token = (pair[:R] // k).long()
        assert torch.equal(qr[:R].view(torch.uint8), q.view(torch.uint8)[token]) and torch.equal(sr[:R], s[token])
        got = moe.mx_matmul(qr, sr, w, ws, row_offset=off, tile=9)   # a tile kernel, or an error
        # the same rows in a buffer of the caller's, 32 bytes further apart
        qo = torch.zeros(N * k, q.stride(0) + 32, dtype=torch.uint8, device="cuda")[:, :q.shape[1]]
        so = torch.zeros(N * k, s.stride(0) + 32, dtype=torch.uint8, device="cuda")[:, :s.shape[1]]
        moe.dispatch_rows(q.view(torch.uint8), pair, off, k, out=qo)
        moe.dispatch_rows(s, pair, off, k, out=so)
        want = moe.mx_matmul(qo.view(F8) if element == "e4m3" else qo, so, w, ws, row_offset=off, tile=9)
        assert torch.equal(got[:R].view(torch.uint8), want[:R].view(torch.uint8))


def test_only_small_paddings_of_bytes_are_kept():
    pair, off, R = layout(20, 2, 3, 1)
    token = (pair[:R] // 2).long()
    for dtype, H, apart, want in ((torch.uint8, 90, 90, 90), (torch.uint8, 90, 92, 92), (torch.uint8, 90, 105, 105), (torch.uint8, 90, 106, 90),
                                  (F8, 1000, 1008, 1008), (BF, 90, 92, 90)):
        x = torch.randint(0, 100, (20, apart), generator=gen(apart)).to(dtype).cuda()[:, :H]
        out = moe.dispatch_rows(x, pair, off, 2)
        assert out.shape == (40, H) and out.stride() == (want, 1)
        assert torch.equal(out[:R].contiguous().view(torch.uint8), x.contiguous()[token].view(torch.uint8))
