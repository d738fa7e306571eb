"""Products whose sum is cut into ranges, added up side by side in a workspace and
joined: every tile and number of ranges against 64 bits (the bars of the whole
products hold for any order of the sums), what stays untouched, streams and
graphs."""
import ctypes

import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib, ops
from test_gpu_operators import BF, DGRAD, F32, FWD, WGRAD, gen, normal, offsets, run_fp8, run_grouped, up

pytestmark = pytest.mark.gpu
OPS = pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])


TILES = [(op, tile) for op in (FWD, DGRAD, WGRAD) for tile in ((1, 3, 4, 5) if op == WGRAD else range(1, 10))]


@pytest.mark.parametrize("splits", [2, 3, 64])
@pytest.mark.parametrize("op,tile", TILES)
def test_grouped_every_tile_in_ranges(op, tile, splits):
    # sums of 1032, 136 and up to 290: whole and ragged ranges, and empty ones
    run_grouped(op, [0, 33, 290, 1], 1032, 136, BF, seed=splits, first=2, behind=4, pad=8, tile=tile, splits=splits)
    run_grouped(op, [70, 257], 64, 264, F32, seed=splits, tile=tile, splits=splits)


@pytest.mark.parametrize("splits", [2, 5, 64])
@pytest.mark.parametrize("tile", range(1, 10))
def test_fp8_every_tile_in_ranges(tile, splits):
    run_fp8([0, 33, 290, 1], 324, 1040, 136, BF, behind=4, pad=16, tile=tile, splits=splits)
    run_fp8(None, 70, 272, 264, F32, tile=tile, splits=splits)


@OPS
def test_operands_of_any_alignment_are_not_cut(op):
    run_grouped(op, [33, 90], 131, 67, BF, seed=1, splits=4)


def needs(op, rows, L, n, k, **kw):
    x, w, y = torch.empty(rows, k, dtype=BF), torch.empty(L, n, k, dtype=BF), torch.empty(rows, n, dtype=BF)
    p = ops.check_grouped_inputs(op, x, w, y, torch.zeros(L + 1, dtype=torch.int32), **kw)
    return _lib.load().moe_grouped_workspace_bytes(ctypes.byref(p))


def test_automatic_choice():
    # few tiles and a long sum take a workspace of whole outputs, others none
    got = needs(WGRAD, 16000, 1, 128, 256)
    assert got >= 2 * 128 * 256 * 4 and got % (128 * 256 * 4) == 0
    assert needs(FWD, 16000, 1, 4096, 4096) == 0 and needs(FWD, 1, 1, 64, 64) == 0
    assert needs(WGRAD, 16000, 1, 128, 256, splits=1) == 0
    run_grouped(WGRAD, [9000, 0, 5000], 256, 128, BF, seed=4)
    run_grouped(WGRAD, [9000, 0, 5000], 256, 128, F32, seed=4)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
def test_accumulation_over_ranges(out_dtype):
    g = gen(3)
    counts, k, n = [700, 0, 300], 136, 72
    x, dy, off = up(normal(g, 1000, k)), up(normal(g, 1000, n)), up(offsets(counts))
    start = normal(g, 3, n, k).to(out_dtype)
    start[1, 0, :3] = torch.tensor([-0.0, float("nan"), float("inf")])
    out = up(start.clone())
    moe.grouped_matmul_wgrad(dy, x, off, out=out, accumulate=True, splits=5)
    new = moe.grouped_matmul_wgrad(dy, x, off, out_dtype=F32, splits=5)
    want = (start.cuda().float() + new).to(out_dtype)   # added in fp32, rounded once
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    bits = torch.int16 if out_dtype == BF else torch.int32
    assert torch.equal(out[1].cpu().view(bits), start[1].view(bits)), "an expert without rows was written"


def test_ranges_on_streams_and_repeats():
    # sums joined in their order: the same bits again, on a stream of the
    # caller's, and with two calls under way at once
    g = gen(5)
    x, dy, off = up(normal(g, 9000, 256)), up(normal(g, 9000, 128)), up(offsets([9000]))
    want = moe.grouped_matmul_wgrad(dy, x, off, splits=8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(want) for _ in range(6)] for _ in streams]
    for i in range(6):
        for s, o in zip(streams, outs):
            moe.grouped_matmul_wgrad(dy, x, off, out=o[i], splits=8, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for o in outs for t in o)


def test_ranges_in_two_graphs():
    g = gen(6)
    x, dy, off = up(normal(g, 9000, 256)), up(normal(g, 9000, 128)), up(offsets([9000]))
    w, xs = up(normal(g, 1, 128, 4096, std=0.02)), up(normal(g, 200, 4096))
    off2 = up(offsets([200]))
    dw, y = torch.empty(1, 128, 256, dtype=F32, device="cuda"), torch.empty(200, 128, dtype=BF, device="cuda")

    def one():
        moe.grouped_matmul_wgrad(dy, x, off, out=dw, splits=8)
        moe.grouped_matmul(xs, w, off2, out=y, splits=4)

    one()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            one()
        graphs.append(graph)
    for i in range(4):
        x.copy_(normal(gen(10 + i), 9000, 256))
        xs.copy_(normal(gen(20 + i), 200, 4096))
        one()   # eager
        want = dw.clone(), y.clone()
        for graph in graphs:
            dw.zero_()
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(dw, want[0]) and torch.equal(y, want[1])


def test_workspace_too_small():
    x, w, y = (torch.zeros(s, dtype=BF, device="cuda") for s in ((64, 1024), (1, 64, 1024), (64, 64)))
    off = up(offsets([64]))
    p = ops.check_grouped_inputs(FWD, x, w, y, off, splits=4)
    call = _lib.load().moe_grouped_matmul_split
    need = 4 * 64 * 64 * 4
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ptrs = [t.data_ptr() for t in (off, x, w, y, ws)]
    p.workspace_bytes = need - 1
    assert call(ctypes.byref(p), *ptrs, None) == -3   # MOE_ERR_WORKSPACE_TOO_SMALL
    p.workspace_bytes = need
    assert call(ctypes.byref(p), *ptrs[:4], None, None) == -3
    assert call(ctypes.byref(p), *ptrs, None) == _lib.MOE_OK
    torch.cuda.synchronize()
