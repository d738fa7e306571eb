"""Sizes at the ends of what the operators take (CPU only; meta tensors hold no
memory, and C pointers are never followed)."""
import ctypes
import os

import pytest
import torch

from moe_expert_ffn_persistent_amd import _lib, ops

BF, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


def meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _lib_or_skip():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmoe_ffn.so not built")
    return _lib.load()


@pytest.mark.parametrize("tokens,top_k,ok", [((1 << 30) + 1, 1, True), (1 << 31, 16, True), (1 << 40, 16, True), ((1 << 40) + 1, 1, False)])
def test_c_dispatch_takes_tokens_past_the_pairs_of_an_index(tokens, top_k, ok):
    # no rows: nothing is launched once the parameters are in order
    p = _lib.MoeRowsParams(tokens, 0, top_k, 8, 1, 2, 0, 8, 8)
    want = _lib.MOE_OK if ok else _lib.MOE_ERR_INVALID_ARG
    assert _lib_or_skip().moe_dispatch_rows(ctypes.byref(p), 16, 16, 16, 16, None) == want


def test_combine_rows_takes_more_tokens_in_pieces(monkeypatch):
    made = []
    monkeypatch.setattr(ops, "_first_call", lambda name, check, args, *rest: made.append((check(*args), args)))
    monkeypatch.setattr(ops, "_MAX_TOKENS", 100)
    rows, out, at = torch.zeros(8, 16, dtype=BF), torch.zeros(230, 16), torch.arange(230 * 3, dtype=I32).view(230, 3)
    assert ops.combine_rows(rows, at, 3, out=out) is out
    assert [p.tokens for p, _ in made] == [100, 100, 30]
    for n, (_, (r, pairs, k, o)) in zip((0, 100, 200), made):
        assert r is rows and k == 3 and pairs[0] == 3 * n and pairs.numel() == 3 * o.shape[0]
        assert o.data_ptr() == out[n:].data_ptr()
    with pytest.raises(ValueError):   # what is wrong with the whole call is said before any piece
        ops.combine_rows(rows, at, 3, out=torch.zeros(231, 16))
    assert len(made) == 3


def stretched(shape, strides, dtype=BF):
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta")


def off(n=1):
    return meta(n + 1, dtype=I32)


FWD = _lib.MOE_GROUPED_FORWARD
ROWS, COLS, STRIDE, MATRIX = 1 << 28, 1 << 20, 1 << 32, 1 << 52
# name: a check of a size (or stride, or number) that is the limit's with 0, past it with 1
LIMITS = {
    "dispatch_rows": lambda d: ops.check_dispatch_inputs(meta(4, 8), meta(ROWS + 1, dtype=I32), off(), 2, meta(ROWS + d, 8)),
    "dispatch_hidden": lambda d: ops.check_dispatch_inputs(meta(4, COLS + d), meta(8, dtype=I32), off(), 2, meta(8, COLS + d)),
    "dispatch_stride": lambda d: ops.check_dispatch_inputs(stretched((4, 8), (STRIDE + d, 1)), meta(8, dtype=I32), off(), 2, meta(8, 8)),
    "combine_rows": lambda d: ops.check_combine_rows_inputs(meta(ROWS + d, 8), meta(8, dtype=I32), 2, meta(4, 8)),
    "combine_out_stride": lambda d: ops.check_combine_rows_inputs(meta(8, 8), meta(8, dtype=I32), 2, stretched((4, 8), (STRIDE + d, 1))),
    "grouped_rows": lambda d: ops.check_grouped_inputs(FWD, meta(ROWS + d, 8), meta(1, 8, 8), meta(ROWS + d, 8), off()),
    "grouped_k": lambda d: ops.check_grouped_inputs(FWD, meta(4, COLS + d), meta(1, 8, COLS + d), meta(4, 8), off()),
    "grouped_n": lambda d: ops.check_grouped_inputs(FWD, meta(4, 8), meta(1, COLS + d, 8), meta(4, COLS + d), off()),
    "grouped_expert_stride": lambda d: ops.check_grouped_inputs(
        FWD, meta(4, 8), stretched((2, 8, 8), (MATRIX + d, 8, 1)), meta(4, 8), off(2)),
    "grouped_splits": lambda d: ops.check_grouped_inputs(FWD, meta(4, 8), meta(1, 8, 8), meta(4, 8), off(), splits=64 + d),
    "grouped_no_splits": lambda d: ops.check_grouped_inputs(FWD, meta(4, 8), meta(1, 8, 8), meta(4, 8), off(), splits=-d),
    "grouped_tile": lambda d: ops.check_grouped_inputs(FWD, meta(4, 8), meta(1, 8, 8), meta(4, 8), off(), tile=-d),
    "swiglu_rows": lambda d: ops.check_swiglu_inputs(meta(ROWS + d, 16), None, None, meta(ROWS + d, 8), None),
    "swiglu_inter": lambda d: ops.check_swiglu_inputs(meta(4, 2 * (COLS + d)), None, None, meta(4, COLS + d), None),
    "swiglu_scale_stride": lambda d: ops.check_swiglu_inputs(
        meta(4, 16), None, None, meta(4, 8, dtype=F8), stretched((4, 1), (STRIDE + d, 1), F32)),
    "swiglu_backward_rows": lambda d: ops.check_swiglu_backward_inputs(
        meta(ROWS + d, 16), meta(ROWS + d, 8), None, None, meta(ROWS + d, 16), None),
    "quantize_rows": lambda d: ops.check_quantize_inputs(
        meta(ROWS + d, 8), 1, None, meta(ROWS + d, 8, dtype=F8), meta(ROWS + d, 1, dtype=F32)),
    "quantize_batch": lambda d: ops.check_quantize_inputs(
        meta(65535 + d, 1, 8), 1, None, meta(65535 + d, 1, 8, dtype=F8), meta(65535 + d, 1, 1, dtype=F32)),
    "quantize_blocks": lambda d: ops.check_quantize_inputs(
        meta(1 << 17, (1 << 20) - 128 * (1 - d)), 128, None, meta(1 << 17, (1 << 20) - 128 * (1 - d), dtype=F8),
        meta(1 << 10, (1 << 13) - 1 + d, dtype=F32)),
    "fp8_rows": lambda d: ops.check_fp8_inputs(meta(ROWS + d, 16, dtype=F8), meta(ROWS + d, 1, dtype=F32), meta(8, 16, dtype=F8),
                                               meta(1, 1, dtype=F32), None, meta(ROWS + d, 8)),
    "fp8_n": lambda d: ops.check_fp8_inputs(meta(4, 16, dtype=F8), meta(4, 1, dtype=F32), meta(COLS + d, 16, dtype=F8),
                                            meta(-(-(COLS + d) // 128), 1, dtype=F32), None, meta(4, COLS + d)),
    "fp8_splits": lambda d: ops.check_fp8_inputs(meta(4, 16, dtype=F8), meta(4, 1, dtype=F32), meta(8, 16, dtype=F8),
                                                 meta(1, 1, dtype=F32), None, meta(4, 8), splits=64 + d),
}


@pytest.mark.parametrize("name", sorted(LIMITS))
def test_sizes_past_the_limits_are_refused(name):
    LIMITS[name](0)
    with pytest.raises(ValueError):
        LIMITS[name](1)


POINTERS = {   # parameters, and the alignment of each pointer
    "moe_dispatch_rows": (lambda: _lib.MoeRowsParams(4, 8, 2, 8, 4, 2, 0, 8, 8), (4, 4, 4, 4)),
    "moe_combine_rows": (lambda: _lib.MoeRowsParams(4, 8, 2, 8, 2, 0, 0, 8, 8), (2, 4, 4)),
    "moe_grouped_matmul": (lambda: _lib.MoeGroupedParams(0, 2, 4, 0, 8, 16, 16, 16, 8, 128, 0, 0, 0), (4, 2, 2, 4)),
    "moe_swiglu": (lambda: _lib.MoeSwigluParams(4, 8, 2, 1, 16, 8, 1, 0), (2, 4, 4, 1, 4)),
    "moe_swiglu_backward": (lambda: _lib.MoeSwigluParams(4, 8, 2, 0, 16, 8, 0, 16), (2, 2, 4, 4, 2, 4)),
    "moe_quantize_fp8": (lambda: _lib.MoeQuantizeParams(4, 1, 8, 1, 0, 2, 8, 8, 0, 0), (4, 4, 1, 4)),
    "moe_fp8_matmul": (lambda: _lib.MoeFp8Params(2, 4, 0, 8, 256, 256, 2, 256, 8, 2048, 0, 0), (4, 1, 4, 1, 4, 4)),
}


@pytest.mark.parametrize("name", sorted(POINTERS))
def test_c_entries_refuse_pointers_off_their_elements(name):
    params, need = POINTERS[name]
    for i, n in enumerate(need):
        for by in range(1, n):
            ptrs = [1 << 20] * len(need)
            ptrs[i] += by
            assert getattr(_lib_or_skip(), name)(ctypes.byref(params()), *ptrs, None) == _lib.MOE_ERR_INVALID_ARG, (i, by)
