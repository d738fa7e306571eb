"""Refusals of the operators around the expert FFN (CPU only): each mismatch
raises ValueError in the binding before any launch, and the C entry points
refuse bad parameters with MOE_ERR_INVALID_ARG before they touch the device."""
import ctypes
import os

import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib, ops

L, R, K, N = 3, 10, 40, 24
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def off(n=L):
    return torch.zeros(n + 1, dtype=torch.int32)


# ---- what is accepted --------------------------------------------------------

def test_grouped_accepts_strides_and_reports_them():
    x = z(R, 2 * K)[:, :K]
    w = z(L, N + 2, K + 8)[:, :N, :K]
    p = ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, x, w, z(R, N), off())
    assert (p.ld_x, p.ld_w, p.ld_y, p.expert_stride_w) == (2 * K, K + 8, N, (N + 2) * (K + 8))
    assert (p.n, p.k, p.rows, p.num_experts, p.expected_rows) == (N, K, R, L, 0)


def test_single_rows_and_experts_take_any_outer_stride():
    x = z(1, K).as_strided((1, K), (1, 1))
    w = z(1, 1, K).as_strided((1, 1, K), (1, 1, 1))
    p = ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, x, w, z(1, 1), off(1), expected_rows=5)
    assert p.ld_x >= K and p.ld_w >= K and p.expert_stride_w >= K and p.expected_rows == 5


def test_other_operators_accept_their_buffers():
    ops.check_dispatch_inputs(z(4, K), torch.zeros(8, dtype=torch.int32), off(), 2, z(8, K))
    ops.check_combine_rows_inputs(z(8, K), torch.zeros(8, dtype=torch.int32), 2, z(4, K, dtype=F32))
    ops.check_swiglu_inputs(z(R, 2 * K), z(R, dtype=F32), off(), z(R, K), None)
    ops.check_swiglu_inputs(z(R, 2 * K), None, None, z(R, K, dtype=F8), z(R, 1, dtype=F32))
    ops.check_swiglu_backward_inputs(z(R, 2 * K), z(R, K), None, None, z(R, 2 * K), None)
    ops.check_quantize_inputs(z(2, 130, 200), 128, None, z(2, 130, 200, dtype=F8), z(2, 2, 2, dtype=F32))
    ops.check_fp8_inputs(z(R, 200, dtype=F8), z(R, 2, dtype=F32), z(130, 200, dtype=F8), z(2, 2, dtype=F32), None, z(R, 130))


# ---- refusals ------------------------------------------------------------------

GROUPED = {
    "x_dtype": dict(x=z(R, K, dtype=F32)),
    "x_half": dict(x=z(R, K, dtype=torch.float16)),
    "x_dims": dict(x=z(1, R, K)),
    "x_transposed": dict(x=z(K, R).t()),
    "x_broadcast_rows": dict(x=z(1, K).expand(R, K)),
    "x_overlapping_rows": dict(x=z(R * K).as_strided((R, K), (K - 1, 1))),
    "x_not_a_tensor": dict(x=[[0.0] * K] * R),
    "w_dims": dict(w=z(N, K)),
    "w_features": dict(w=z(L, N, K + 1)),
    "w_broadcast_experts": dict(w=z(1, N, K).expand(L, N, K)),
    "w_out_features": dict(w=z(L, N + 1, K)),
    "y_rows": dict(y=z(R - 1, N)),
    "y_dtype": dict(y=z(R, N, dtype=torch.float16)),
    "offsets_dtype": dict(row_offset=torch.zeros(L + 1, dtype=torch.int64)),
    "offsets_experts": dict(row_offset=off(L + 1)),
    "offsets_strided": dict(row_offset=torch.zeros(2 * L + 2, dtype=torch.int32)[::2]),
    "offsets_none": dict(row_offset=torch.zeros(1, dtype=torch.int32)),
    "too_many_experts": dict(w=z(257, 1, K), y=z(R, 1), row_offset=off(257)),
    "no_features": dict(x=z(R, 0), w=z(L, N, 0)),
    "expected_rows": dict(expected_rows=0),
    "requires_grad": dict(x=z(R, K).requires_grad_()),
}


@pytest.mark.parametrize("case", sorted(GROUPED))
def test_grouped_refuses(case):
    kw = dict(x=z(R, K), w=z(L, N, K), y=z(R, N), row_offset=off())
    kw.update(GROUPED[case])
    with pytest.raises(ValueError):
        ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, **kw)


def test_grouped_gradients_take_the_types_of_what_they_write():
    ops.check_grouped_inputs(_lib.MOE_GROUPED_DGRAD, z(R, K, dtype=F32), z(L, N, K), z(R, N), off())
    ops.check_grouped_inputs(_lib.MOE_GROUPED_WGRAD, z(R, K), z(L, N, K, dtype=F32), z(R, N), off(), accumulate=True)
    with pytest.raises(ValueError):
        ops.check_grouped_inputs(_lib.MOE_GROUPED_DGRAD, z(R, K), z(L, N, K, dtype=F32), z(R, N), off())
    with pytest.raises(ValueError):
        ops.check_grouped_inputs(_lib.MOE_GROUPED_WGRAD, z(R, K, dtype=F32), z(L, N, K), z(R, N), off())
    with pytest.raises(ValueError):
        moe.grouped_matmul_wgrad(z(R, N), z(R, K), off(), accumulate=True)


def test_grad_mode_off_takes_tensors_that_require_grad():
    with torch.no_grad():
        ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, z(R, K), z(L, N, K).requires_grad_(), z(R, N), off())


ROWS = {
    "x_dtype": dict(x=z(4, K, dtype=torch.float64)),
    "row_pair_dtype": dict(row_pair=torch.zeros(8, dtype=torch.int64)),
    "row_pair_short": dict(row_pair=torch.zeros(7, dtype=torch.int32)),
    "top_k_zero": dict(top_k=0),
    "top_k_large": dict(top_k=17),
    "out_width": dict(out=z(8, K + 1)),
    "out_dtype": dict(out=z(8, K, dtype=F32)),
}


@pytest.mark.parametrize("case", sorted(ROWS))
def test_dispatch_refuses(case):
    kw = dict(x=z(4, K), row_pair=torch.zeros(8, dtype=torch.int32), row_offset=off(), top_k=2, out=z(8, K))
    kw.update(ROWS[case])
    with pytest.raises(ValueError):
        ops.check_dispatch_inputs(**kw)


COMBINE = {
    "rows_dtype": dict(rows=z(8, K, dtype=F32)),
    "pair_row_tokens": dict(pair_row=torch.zeros(9, dtype=torch.int32)),
    "pair_row_dtype": dict(pair_row=torch.zeros(8, dtype=torch.int64)),
    "out_tokens": dict(out=z(5, K)),
    "out_dtype": dict(out=z(4, K, dtype=torch.float16)),
    "top_k": dict(top_k=0),
}


@pytest.mark.parametrize("case", sorted(COMBINE))
def test_combine_rows_refuses(case):
    kw = dict(rows=z(8, K), pair_row=torch.zeros(8, dtype=torch.int32), top_k=2, out=z(4, K))
    kw.update(COMBINE[case])
    with pytest.raises(ValueError):
        ops.check_combine_rows_inputs(**kw)


SWIGLU = {
    "odd_columns": dict(a=z(R, 2 * K + 1)),
    "weight_dtype": dict(row_weight=z(R)),
    "weight_rows": dict(row_weight=z(R + 1, dtype=F32)),
    "out_shape": dict(h=z(R, 2 * K)),
    "out_fp32": dict(h=z(R, K, dtype=F32)),
    "scales_missing": dict(h=z(R, K, dtype=F8)),
    "scales_with_bf16": dict(scales=z(R, 1, dtype=F32)),
    "scales_shape": dict(h=z(R, K, dtype=F8), scales=z(R, 2, dtype=F32)),
    "requires_grad": dict(row_weight=z(R, dtype=F32).requires_grad_()),
}


@pytest.mark.parametrize("case", sorted(SWIGLU))
def test_swiglu_refuses(case):
    kw = dict(a=z(R, 2 * K), row_weight=None, row_offset=None, h=z(R, K), scales=None)
    kw.update(SWIGLU[case])
    with pytest.raises(ValueError):
        ops.check_swiglu_inputs(**kw)


@pytest.mark.parametrize("case", ["dh_shape", "da_shape", "drow_rows", "dh_dtype"])
def test_swiglu_backward_refuses(case):
    kw = dict(a=z(R, 2 * K), dh=z(R, K), row_weight=None, row_offset=None, da=z(R, 2 * K), drow_weight=None)
    kw.update({"dh_shape": dict(dh=z(R, K + 1)), "da_shape": dict(da=z(R, K)), "drow_rows": dict(drow_weight=z(R - 1, dtype=F32)),
               "dh_dtype": dict(dh=z(R, K, dtype=F32))}[case])
    with pytest.raises(ValueError):
        ops.check_swiglu_backward_inputs(**kw)


QUANT = {
    "block_rows": dict(block_rows=64),
    "dims": dict(x=z(4)),
    "x_dtype": dict(x=z(R, K, dtype=torch.float16)),
    "codes_shape": dict(codes=z(R, K + 1, dtype=F8)),
    "codes_dtype": dict(codes=z(R, K)),
    "scales_shape": dict(scales=z(R, 2, dtype=F32)),
    "scales_strided": dict(scales=z(2 * R, 1, dtype=F32)[::2]),
    "offsets_with_blocks": dict(block_rows=128, scales=z(1, 1, dtype=F32), row_offset=off()),
}


@pytest.mark.parametrize("case", sorted(QUANT))
def test_quantize_refuses(case):
    kw = dict(x=z(R, K), block_rows=1, row_offset=None, codes=z(R, K, dtype=F8), scales=z(R, 1, dtype=F32))
    kw.update(QUANT[case])
    with pytest.raises(ValueError):
        ops.check_quantize_inputs(**kw)


FP8 = {
    "x_bf16": dict(x=z(R, 200)),
    "w_dims": dict(row_offset=off()),
    "x_scales_shape": dict(x_scales=z(R, 1, dtype=F32)),
    "x_scales_dtype": dict(x_scales=z(R, 2)),
    "w_scales_shape": dict(w_scales=z(1, 2, dtype=F32)),
    "w_scales_strided": dict(w_scales=z(2, 4, dtype=F32)[:, ::2]),
    "out_shape": dict(y=z(R, 131)),
    "k": dict(w=z(130, 199, dtype=F8)),
    "grouped_experts": dict(w=z(L, 130, 200, dtype=F8), w_scales=z(L, 2, 2, dtype=F32), row_offset=off(L + 1)),
}


@pytest.mark.parametrize("case", sorted(FP8))
def test_fp8_refuses(case):
    kw = dict(x=z(R, 200, dtype=F8), x_scales=z(R, 2, dtype=F32), w=z(130, 200, dtype=F8), w_scales=z(2, 2, dtype=F32),
              row_offset=None, y=z(R, 130))
    kw.update(FP8[case])
    with pytest.raises(ValueError):
        ops.check_fp8_inputs(**kw)


def test_host_tensors_are_refused():
    with pytest.raises(ValueError):
        moe.grouped_matmul(z(R, K), z(L, N, K), off())
    with pytest.raises(ValueError):
        moe.grouped_matmul(z(R, K), z(L, N, K), off(), out=z(R, N))
    with pytest.raises(ValueError):
        moe.swiglu(z(R, 2 * K))
    with pytest.raises(ValueError):
        moe.quantize_fp8(z(R, K))
    with pytest.raises(ValueError):
        moe.dispatch_rows(z(4, K), torch.zeros(8, dtype=torch.int32), off(), 2)
    with pytest.raises(ValueError):
        moe.combine_rows(z(8, K), torch.zeros(8, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        moe.fp8_matmul(z(R, 200, dtype=F8), z(R, 2, dtype=F32), z(130, 200, dtype=F8), z(2, 2, dtype=F32))


def test_arguments_that_are_no_tensors_are_refused():
    # also where the output is given, and nothing has to be allocated first
    i32 = torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.dispatch_rows([1.0], i32, off(), 2, out=z(8, K)),
                 lambda: moe.dispatch_rows(z(4, K), [0] * 8, off(), 2),
                 lambda: moe.combine_rows(z(8, K), [0] * 8, 2),
                 lambda: moe.combine_rows([1.0], i32, 2, out=z(4, K)),
                 lambda: moe.grouped_matmul([1.0], z(L, N, K), off(), out=z(R, N)),
                 lambda: moe.grouped_matmul_wgrad(z(R, N), z(R, K), [0, 1]),
                 lambda: moe.swiglu([1.0], out=z(R, K)),
                 lambda: moe.swiglu_backward([1.0], z(R, K), out=z(R, 2 * K)),
                 lambda: moe.quantize_fp8([1.0], out=z(R, K, dtype=F8), scales=z(R, 1, dtype=F32)),
                 lambda: moe.fp8_matmul(z(R, 200, dtype=F8), z(R, 2, dtype=F32), [1.0], z(2, 2, dtype=F32)),
                 lambda: moe.fp8_matmul([1.0], z(R, 2, dtype=F32), z(N, 200, dtype=F8), z(1, 2, dtype=F32), out=z(R, N))):
        with pytest.raises(ValueError):
            call()


class _Stream:
    def __init__(self, device_index):
        self.device_index = device_index


def test_streams_of_another_device_are_refused():
    ops._check_stream(_Stream(1), 1)
    for stream in (_Stream(0), 7):
        with pytest.raises(ValueError, match="stream"):
            ops._check_stream(stream, 1)


def test_negated_views_are_refused():
    x = torch.zeros(R, 1, dtype=torch.complex64).conj().imag   # fp32, its sign not in memory
    assert x.is_neg()
    with pytest.raises(ValueError, match="negation"):
        ops.check_quantize_inputs(x.as_strided((R, 1), (2, 1)), 1, None, z(R, 1, dtype=F8), z(R, 1, dtype=F32))


def test_single_rows_with_huge_strides_count_as_their_length():
    x = torch.empty_strided((1, K), (1 << 40, 1), dtype=BF, device="meta")
    assert ops._matrix(x, "x", (BF,)) == K


# ---- the C entry points, with pointers that are never followed -------------------

def _lib_or_skip():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmoe_ffn.so not built")
    return _lib.load()


def _call(name, params, *ptrs):
    return getattr(_lib_or_skip(), name)(ctypes.byref(params), *ptrs, None)


def _grouped(**kw):
    base = dict(op=0, num_experts=2, rows=4, expected_rows=0, n=8, k=16, ld_x=16, ld_w=16, ld_y=8, expert_stride_w=128,
                out_dtype=_lib.MOE_Y_BF16, accumulate=0, tile=0)
    base.update(kw)
    return _lib.MoeGroupedParams(*base.values())


@pytest.mark.parametrize("kw", [dict(op=3), dict(op=-1), dict(num_experts=0), dict(num_experts=257), dict(rows=-1),
                                dict(rows=(1 << 28) + 1), dict(n=0), dict(k=0), dict(k=(1 << 20) + 1), dict(ld_x=15),
                                dict(ld_w=15), dict(ld_y=7), dict(expert_stride_w=127), dict(out_dtype=2),
                                dict(accumulate=1), dict(expected_rows=-1), dict(tile=-1)])
def test_c_grouped_refuses(kw):
    assert _call("moe_grouped_matmul", _grouped(**kw), 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


def test_c_grouped_refuses_missing_and_misaligned_pointers():
    for ptrs in ((None, 16, 16, 16), (16, None, 16, 16), (16, 16, None, 16), (16, 16, 16, None), (16, 17, 16, 16)):
        assert _call("moe_grouped_matmul", _grouped(), *ptrs) == _lib.MOE_ERR_INVALID_ARG
    assert _call("moe_grouped_matmul", _grouped(out_dtype=_lib.MOE_Y_FP32), 16, 16, 16, 18) == _lib.MOE_ERR_INVALID_ARG
    # a tile id that does not exist, or does not take these operands
    assert _call("moe_grouped_matmul", _grouped(tile=99), 16, 16, 16, 16) == _lib.MOE_ERR_UNSUPPORTED
    assert _call("moe_grouped_matmul", _grouped(tile=1), 16, 18, 16, 16) == _lib.MOE_ERR_UNSUPPORTED
    # nothing to do: no rows
    assert _call("moe_grouped_matmul", _grouped(rows=0), None, None, None, None) == _lib.MOE_OK
    assert _call("moe_grouped_matmul", _grouped(rows=0, op=2), None, None, None, None) == _lib.MOE_ERR_INVALID_ARG


def test_c_null_params_are_refused():
    lib = _lib_or_skip()
    for name, n in (("moe_dispatch_rows", 4), ("moe_combine_rows", 3), ("moe_grouped_matmul", 4), ("moe_swiglu", 5),
                    ("moe_swiglu_backward", 6), ("moe_quantize_fp8", 4), ("moe_fp8_matmul", 6)):
        assert getattr(lib, name)(None, *([16] * n), None) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(rows=-1), dict(top_k=0), dict(top_k=17), dict(hidden=0),
                                dict(elem_bytes=3), dict(num_experts=0), dict(ld_tokens=7), dict(ld_rows=7)])
def test_c_dispatch_refuses(kw):
    base = dict(tokens=4, rows=8, top_k=2, hidden=8, elem_bytes=2, num_experts=2, out_dtype=0, ld_tokens=8, ld_rows=8)
    base.update(kw)
    assert _call("moe_dispatch_rows", _lib.MoeRowsParams(*base.values()), 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(elem_bytes=4), dict(out_dtype=5), dict(tokens=(1 << 23) + 1), dict(ld_rows=7)])
def test_c_combine_refuses(kw):
    base = dict(tokens=4, rows=8, top_k=2, hidden=8, elem_bytes=2, num_experts=0, out_dtype=1, ld_tokens=8, ld_rows=8)
    base.update(kw)
    assert _call("moe_combine_rows", _lib.MoeRowsParams(*base.values()), 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(inter=0), dict(ld_a=15), dict(ld_h=7), dict(out_format=2),
                                dict(out_format=1, ld_scales=0), dict(num_experts=0)])
def test_c_swiglu_refuses(kw):
    base = dict(rows=4, inter=8, num_experts=2, out_format=0, ld_a=16, ld_h=8, ld_scales=1, ld_da=16)
    base.update(kw)
    assert _call("moe_swiglu", _lib.MoeSwigluParams(*base.values()), 16, 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(batch=0), dict(cols=0), dict(block_rows=2), dict(in_dtype=3), dict(ld_x=7),
                                dict(ld_codes=7), dict(batch=2, batch_stride_x=31), dict(block_rows=128)])
def test_c_quantize_refuses(kw):
    base = dict(rows=4, batch=1, cols=8, block_rows=1, in_dtype=1, num_experts=2, ld_x=8, ld_codes=8, batch_stride_x=32,
                batch_stride_codes=32)
    base.update(kw)
    assert _call("moe_quantize_fp8", _lib.MoeQuantizeParams(*base.values()), 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(num_experts=0), dict(rows=-1), dict(n=0), dict(k=0), dict(ld_x=255), dict(ld_xs=1),
                                dict(ld_w=255), dict(ld_y=7), dict(expert_stride_w=2047), dict(out_dtype=9), dict(tile=-1)])
def test_c_fp8_refuses(kw):
    base = dict(num_experts=2, rows=4, expected_rows=0, n=8, k=256, ld_x=256, ld_xs=2, ld_w=256, ld_y=8,
                expert_stride_w=2048, out_dtype=1, tile=0)
    base.update(kw)
    assert _call("moe_fp8_matmul", _lib.MoeFp8Params(*base.values()), 16, 16, 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


def test_c_fp8_dense_has_one_matrix():
    base = dict(num_experts=2, rows=4, expected_rows=0, n=8, k=256, ld_x=256, ld_xs=2, ld_w=256, ld_y=8,
                expert_stride_w=2048, out_dtype=1, tile=0)
    assert _call("moe_fp8_matmul", _lib.MoeFp8Params(*base.values()), None, 16, 16, 16, 16, 16) == _lib.MOE_ERR_INVALID_ARG


def test_c_fp8_refuses_tiles_it_does_not_have():
    base = dict(num_experts=1, rows=4, expected_rows=0, n=8, k=256, ld_x=256, ld_xs=2, ld_w=256, ld_y=8,
                expert_stride_w=2048, out_dtype=1, tile=99)
    assert _call("moe_fp8_matmul", _lib.MoeFp8Params(*base.values()), None, 16, 16, 16, 16, 16) == _lib.MOE_ERR_UNSUPPORTED
    base.update(tile=1)
    assert _call("moe_fp8_matmul", _lib.MoeFp8Params(*base.values()), None, 24, 16, 16, 16, 16) == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name, kw", [
    ("moe_dispatch_rows", dict(tokens=1 << 62)), ("moe_dispatch_rows", dict(ld_tokens=1 << 61)),
    ("moe_dispatch_rows", dict(ld_rows=(1 << 32) + 1)), ("moe_combine_rows", dict(ld_rows=1 << 62)),
    ("moe_grouped_matmul", dict(ld_w=1 << 62)), ("moe_grouped_matmul", dict(ld_x=1 << 33)),
    ("moe_grouped_matmul", dict(expert_stride_w=1 << 60)), ("moe_grouped_matmul", dict(rows=(1 << 28) + 1)),
    ("moe_swiglu", dict(ld_a=1 << 62)), ("moe_swiglu_backward", dict(ld_da=1 << 62)),
    ("moe_quantize_fp8", dict(ld_x=1 << 62)), ("moe_quantize_fp8", dict(batch_stride_codes=1 << 62)),
    ("moe_fp8_matmul", dict(ld_xs=1 << 62)), ("moe_fp8_matmul", dict(ld_w=1 << 62))])
def test_c_refuses_sizes_that_would_overflow(name, kw):
    rows = dict(tokens=4, rows=8, top_k=2, hidden=8, elem_bytes=2, num_experts=2, out_dtype=1, ld_tokens=8, ld_rows=8)
    swiglu = dict(rows=4, inter=8, num_experts=2, out_format=0, ld_a=16, ld_h=8, ld_scales=1, ld_da=16)
    struct, base, ptrs = {
        "moe_dispatch_rows": (_lib.MoeRowsParams, rows, 4), "moe_combine_rows": (_lib.MoeRowsParams, rows, 3),
        "moe_grouped_matmul": (_lib.MoeGroupedParams, dict(
            op=0, num_experts=2, rows=4, expected_rows=0, n=8, k=8, ld_x=8, ld_w=8, ld_y=8, expert_stride_w=64,
            out_dtype=1, accumulate=0, tile=0), 4),
        "moe_swiglu": (_lib.MoeSwigluParams, swiglu, 5), "moe_swiglu_backward": (_lib.MoeSwigluParams, swiglu, 6),
        "moe_quantize_fp8": (_lib.MoeQuantizeParams, dict(
            rows=4, batch=2, cols=8, block_rows=1, in_dtype=1, num_experts=0, ld_x=8, ld_codes=8, batch_stride_x=32,
            batch_stride_codes=32), 4),
        "moe_fp8_matmul": (_lib.MoeFp8Params, dict(
            num_experts=2, rows=4, expected_rows=0, n=8, k=256, ld_x=256, ld_xs=2, ld_w=256, ld_y=8,
            expert_stride_w=2048, out_dtype=1, tile=0), 6)}[name]
    params = struct(*dict(base, **kw).values())
    args = [16] * ptrs
    if name == "moe_quantize_fp8":
        args[1] = None
    assert _call(name, params, *args) == _lib.MOE_ERR_INVALID_ARG


def test_c_quantize_blocks_of_one_launch():
    # 2^23 blocks of 512 threads would be 2^32 threads
    base = dict(rows=1 << 23, batch=1, cols=1 << 14, block_rows=128, in_dtype=1, num_experts=0, ld_x=1 << 14,
                ld_codes=1 << 14, batch_stride_x=0, batch_stride_codes=0)
    assert _call("moe_quantize_fp8", _lib.MoeQuantizeParams(*base.values()), 16, None, 16, 16) == _lib.MOE_ERR_UNSUPPORTED
