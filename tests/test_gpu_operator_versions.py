"""What an operator writes gets a new version, so torch's check of tensors saved
for a backward pass sees an output that overwrites one."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def calls():
    """name: (call, tensors read, tensors written)"""
    off = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    idx = torch.arange(12, dtype=torch.int32, device="cuda")
    x, w, y = z(12, 32), z(2, 16, 32), z(12, 16)
    a, h, rw = z(12, 64), z(12, 32), z(12, dtype=F32)
    out = {k: z(*s, dtype=d) for k, s, d in [
        ("rows", (12, 32), BF), ("tokens", (6, 32), BF), ("y", (12, 16), BF), ("dx", (12, 32), BF), ("dw", (2, 16, 32), F32), ("h", (12, 32), BF),
        ("h8", (12, 32), F8), ("hs", (12, 1), F32), ("da", (12, 64), BF), ("drw", (12,), F32), ("q", (12, 32), F8), ("qs", (12, 1), F32),
        ("y8", (12, 16), BF)]}
    q, qs = moe.quantize_fp8(x)
    wq, wqs = moe.quantize_fp8(w, block_rows=128)
    o = out
    return {
        "dispatch_rows": (lambda: moe.dispatch_rows(x[:6], idx, off, 2, out=o["rows"]), (x, idx, off), (o["rows"],)),
        "combine_rows": (lambda: moe.combine_rows(x, idx, 2, out=o["tokens"]), (x, idx), (o["tokens"],)),
        "grouped_matmul": (lambda: moe.grouped_matmul(x, w, off, out=o["y"]), (x, w, off), (o["y"],)),
        "grouped_matmul_dgrad": (lambda: moe.grouped_matmul_dgrad(y, w, off, out=o["dx"]), (y, w, off), (o["dx"],)),
        "grouped_matmul_wgrad": (lambda: moe.grouped_matmul_wgrad(y, x, off, out=o["dw"]), (y, x, off), (o["dw"],)),
        "grouped_matmul_in_ranges": (lambda: moe.grouped_matmul(x, w, off, out=o["y"], splits=2), (x, w, off), (o["y"],)),
        "swiglu": (lambda: moe.swiglu(a, row_weight=rw, out=o["h"]), (a, rw), (o["h"],)),
        "swiglu_e4m3": (lambda: moe.swiglu(a, row_weight=rw, out=o["h8"], scales=o["hs"]), (a, rw), (o["h8"], o["hs"])),
        "swiglu_backward": (lambda: moe.swiglu_backward(a, h, row_weight=rw, out=o["da"], drow_weight=o["drw"]), (a, h, rw), (o["da"], o["drw"])),
        "quantize_fp8": (lambda: moe.quantize_fp8(x, out=o["q"], scales=o["qs"]), (x,), (o["q"], o["qs"])),
        "fp8_matmul": (lambda: moe.fp8_matmul(q, qs, wq, wqs, row_offset=off, out=o["y8"]), (q, qs, wq, wqs, off), (o["y8"],)),
    }


@pytest.mark.parametrize("stream", ["current", "other"])
@pytest.mark.parametrize("name", ["dispatch_rows", "combine_rows", "grouped_matmul", "grouped_matmul_dgrad", "grouped_matmul_wgrad",
                                  "grouped_matmul_in_ranges", "swiglu", "swiglu_e4m3", "swiglu_backward", "quantize_fp8", "fp8_matmul"])
def test_outputs_get_a_new_version_and_inputs_keep_theirs(name, stream):
    call, read, written = calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side if stream == "other" else torch.cuda.current_stream()):
        for _ in range(3):   # the first call of these sizes, and calls of sizes seen before
            before = [t._version for t in read], [t._version for t in written]
            call()
            assert [t._version for t in read] == before[0]
            assert all(t._version > v for t, v in zip(written, before[1]))
    torch.cuda.synchronize()


def test_a_saved_tensor_that_a_call_overwrites_is_noticed():
    class Swiglu(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            ctx.save_for_backward(a)
            return moe.swiglu(a)

        @staticmethod
        def backward(ctx, dh):
            a, = ctx.saved_tensors
            return moe.swiglu_backward(a, dh, out=a)[0]   # in place: this graph is walked once

    leaf = torch.randn(6, 64, device="cuda").to(BF).requires_grad_()
    for _ in range(2):   # sizes new and seen before
        leaf.grad = None
        a = leaf * 1
        loss = Swiglu.apply(a).float().sum()
        loss.backward(retain_graph=True)
        assert leaf.grad is not None
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_outputs_made_in_inference_mode_are_written():
    with torch.inference_mode():
        a, out = z(4, 32), z(4, 16)
        for _ in range(2):
            assert moe.swiglu(a, out=out) is out
    for _ in range(2):
        assert moe.swiglu(a, out=out) is out   # torch keeps no version of these
    torch.cuda.synchronize()
