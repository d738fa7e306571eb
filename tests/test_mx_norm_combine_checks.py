"""Refusals of the operators before and behind the expert FFN: RMS norm, MX
quantisation and products, weighted combination (CPU only). Each mismatch raises
ValueError in the binding before any launch, and the C entry points refuse bad
parameters with MOE_ERR_INVALID_ARG before they touch the device."""
import ctypes
import os

import pytest
import torch
from torch.autograd import forward_ad

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib, ops

BF, F32, F8, U8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8, torch.int32
R, H, N, K = 10, 72, 24, 70
EPS = ops._bits(1e-6)


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def off(n=3):
    return torch.zeros(n + 1, dtype=I32)


def meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def stretched(shape, strides, dtype=BF):
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta")


def _lib_or_skip():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmoe_ffn.so not built")
    return _lib.load()


def norm(**kw):
    a = dict(x=z(R, H), weight=z(H), residual=None, eps=EPS, quantize=_lib.MOE_NORM_BF16, out=z(R, H), scales=None, residual_out=None)
    return ops.check_rms_norm_inputs(**{**a, **kw})


def norm_backward(**kw):
    a = dict(dy=z(R, H), x=z(R, H), weight=z(H), eps=EPS, dresidual=None, dx=z(R, H), dweight=None)
    return ops.check_rms_norm_backward_inputs(**{**a, **kw})


def quantize(**kw):
    a = dict(x=z(R, K), element=_lib.MOE_MX_E2M1, row_offset=None, codes=z(R, 35, dtype=U8), scales=z(R, 3, dtype=U8))
    return ops.check_quantize_mx_inputs(**{**a, **kw})


def product(**kw):
    a = dict(x=z(R, K, dtype=F8), x_scales=z(R, 3, dtype=U8), w=z(N, 35, dtype=U8), w_scales=z(N, 3, dtype=U8), row_offset=None, y=z(R, N))
    return ops.check_mx_inputs(**{**a, **kw})


def combine(**kw):
    a = dict(rows=z(8, H), pair_row=z(8, dtype=I32), top_k=2, out=z(4, H), weights=z(4, 2, dtype=F32))
    return ops.check_combine_rows_inputs(**{**a, **kw})


def combine_backward(**kw):
    a = dict(dy=z(4, H), rows=z(9, H), pair_row=z(8, dtype=I32), weights=z(4, 2, dtype=F32), drows=z(9, H), dweights=z(4, 2, dtype=F32))
    return ops.check_combine_backward_inputs(**{**a, **kw})


def test_accepted_and_reported():
    p = norm(x=z(R, 2 * H)[:, :H], residual=z(R, H), residual_out=z(R, H + 8)[:, :H], weight=z(H, dtype=F32), out=z(R, H, dtype=F32))
    assert (p.rows, p.hidden, p.ld_x, p.ld_residual, p.ld_residual_out, p.ld_out) == (R, H, 2 * H, H, H + 8, H)
    assert (p.stream_dtype, p.weight_dtype, p.format) == (_lib.MOE_Y_BF16, _lib.MOE_Y_FP32, _lib.MOE_NORM_FP32)
    assert abs(p.eps - 1e-6) < 1e-12
    p = norm(x=z(R, H, dtype=F32), weight=None, quantize=_lib.MOE_NORM_MX_E2M1, out=z(R, 36, dtype=U8), scales=z(R, 4, dtype=U8)[:, :3])
    assert (p.format, p.ld_out, p.ld_scales) == (_lib.MOE_NORM_MX_E2M1, 36, 4)
    norm(quantize=_lib.MOE_NORM_FP8, out=z(R, H, dtype=F8), scales=z(R, 1, dtype=F32))
    p = norm_backward(dy=z(R, H, dtype=F32), dresidual=z(R, H), dweight=z(H, dtype=F32))
    assert (p.weight_gradient, p.format, p.ld_dy, p.ld_dresidual, p.ld_dx) == (1, _lib.MOE_NORM_FP32, H, H, H)
    p = quantize(x=z(2, R, K, dtype=F32), codes=z(2, R + 1, 48, dtype=U8)[:, :R, :35], scales=z(2, R, 4, dtype=U8)[:, :, :3])
    assert (p.batch, p.cols, p.ld_codes, p.batch_stride_codes, p.ld_scales, p.batch_stride_scales) == (2, K, 48, (R + 1) * 48, 4, 4 * R)
    p = product()
    assert (p.k, p.n, p.x_format, p.ld_w, p.num_experts) == (K, N, _lib.MOE_MX_E4M3, 35, 1)
    p = product(x=z(R, 35, dtype=U8), w=z(3, N, 35, dtype=U8), w_scales=z(3, N, 3, dtype=U8), row_offset=off())
    assert (p.k, p.x_format, p.num_experts, p.expert_stride_w, p.expert_stride_w_scales) == (K, _lib.MOE_MX_E2M1, 3, N * 35, N * 3)
    p = product(x=z(R, 69, dtype=F8))   # the last byte of a weight row holds one code
    assert p.k == 69
    combine()
    combine_backward(dy=z(4, H, dtype=F32))


@pytest.mark.skipif(not hasattr(torch, "float4_e2m1fn_x2"), reason="no 4-bit type")
def test_the_formats_own_types_are_taken():
    four, e8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    quantize(codes=z(R, 35, dtype=U8).view(four), scales=z(R, 3, dtype=U8).view(e8))
    product(x=z(R, 35, dtype=U8).view(four), w=z(N, 35, dtype=U8).view(four), x_scales=z(R, 3, dtype=U8).view(e8))


REFUSED = {
    "norm_dtype": lambda: norm(x=z(R, H, dtype=torch.float16)),
    "norm_dims": lambda: norm(x=z(1, R, H)),
    "norm_transposed": lambda: norm(x=z(H, R).t()),
    "norm_broadcast_rows": lambda: norm(x=z(1, H).expand(R, H)),
    "norm_out_shape": lambda: norm(out=z(R, H + 1)),
    "norm_out_dtype": lambda: norm(out=z(R, H, dtype=F8)),
    "norm_weight_size": lambda: norm(weight=z(H + 1)),
    "norm_weight_dtype": lambda: norm(weight=z(H, dtype=torch.float64)),
    "norm_weight_strided": lambda: norm(weight=z(2 * H)[::2]),
    "norm_weight_dims": lambda: norm(weight=z(1, H)),
    "norm_residual_alone": lambda: norm(residual=z(R, H)),
    "norm_residual_out_alone": lambda: norm(residual_out=z(R, H)),
    "norm_residual_dtype": lambda: norm(residual=z(R, H, dtype=F32), residual_out=z(R, H)),
    "norm_residual_rows": lambda: norm(residual=z(R - 1, H), residual_out=z(R, H)),
    "norm_residual_out_rows": lambda: norm(residual=z(R, H), residual_out=z(R + 1, H)),
    "norm_scales_without": lambda: norm(scales=z(R, 1, dtype=F32)),
    "norm_fp8_scales": lambda: norm(quantize=_lib.MOE_NORM_FP8, out=z(R, H, dtype=F8), scales=z(R, 2, dtype=F32)),
    "norm_fp8_scales_type": lambda: norm(quantize=_lib.MOE_NORM_FP8, out=z(R, H, dtype=F8), scales=z(R, 1, dtype=U8)),
    "norm_fp8_no_scales": lambda: norm(quantize=_lib.MOE_NORM_FP8, out=z(R, H, dtype=F8)),
    "norm_mx_scales": lambda: norm(quantize=_lib.MOE_NORM_MX_E4M3, out=z(R, H, dtype=F8), scales=z(R, 2, dtype=U8)),
    "norm_mx_scales_type": lambda: norm(quantize=_lib.MOE_NORM_MX_E4M3, out=z(R, H, dtype=F8), scales=z(R, 3, dtype=F32)),
    "norm_mx_out": lambda: norm(quantize=_lib.MOE_NORM_MX_E2M1, out=z(R, H, dtype=U8), scales=z(R, 3, dtype=U8)),
    "norm_requires_grad": lambda: norm(weight=z(H).requires_grad_()),
    "backward_dy": lambda: norm_backward(dy=z(R, H + 1)),
    "backward_dx_type": lambda: norm_backward(dx=z(R, H, dtype=F32)),
    "backward_dresidual_type": lambda: norm_backward(dresidual=z(R, H, dtype=F32)),
    "backward_dresidual_rows": lambda: norm_backward(dresidual=z(R + 1, H)),
    "backward_dweight": lambda: norm_backward(dweight=z(H)),
    "backward_dweight_size": lambda: norm_backward(dweight=z(H - 1, dtype=F32)),
    "quantize_dtype": lambda: quantize(x=z(R, K, dtype=torch.float16)),
    "quantize_codes_shape": lambda: quantize(codes=z(R, 36, dtype=U8)),
    "quantize_codes_type": lambda: quantize(codes=z(R, 35, dtype=F8)),
    "quantize_scales_shape": lambda: quantize(scales=z(R, 2, dtype=U8)),
    "quantize_scales_type": lambda: quantize(scales=z(R, 3, dtype=F32)),
    "quantize_codes_overlap": lambda: quantize(codes=z(1, 35, dtype=U8).expand(R, 35)),
    "quantize_offsets_of_a_batch": lambda: quantize(x=z(2, R, K), codes=z(2, R, 35, dtype=U8), scales=z(2, R, 3, dtype=U8), row_offset=off()),
    "quantize_dims": lambda: quantize(x=z(K)),
    "product_x_type": lambda: product(x=z(R, K)),
    "product_x_as_bytes": lambda: product(x=z(R, K, dtype=U8)),
    "product_w_type": lambda: product(w=z(N, 35, dtype=F8)),
    "product_w_width": lambda: product(w=z(N, 36, dtype=U8)),
    "product_w_dims": lambda: product(w=z(1, N, 35, dtype=U8)),
    "product_x_scales": lambda: product(x_scales=z(R, 2, dtype=U8)),
    "product_w_scales": lambda: product(w_scales=z(N + 1, 3, dtype=U8)),
    "product_scales_type": lambda: product(w_scales=z(N, 3, dtype=F32)),
    "product_out": lambda: product(y=z(R, N + 1)),
    "product_experts": lambda: product(w=z(2, N, 35, dtype=U8), w_scales=z(2, N, 3, dtype=U8), row_offset=off()),
    "product_experts_overlap": lambda: product(w=z(1, N, 35, dtype=U8).expand(3, N, 35), w_scales=z(3, N, 3, dtype=U8), row_offset=off()),
    "product_scales_overlap": lambda: product(w=z(3, N, 35, dtype=U8), w_scales=z(1, N, 3, dtype=U8).expand(3, N, 3), row_offset=off()),
    "product_expected_rows": lambda: product(expected_rows=0),
    "product_splits": lambda: product(splits=65),
    "combine_weights_type": lambda: combine(weights=z(4, 2)),
    "combine_weights_size": lambda: combine(weights=z(4, 3, dtype=F32)),
    "combine_weights_grad": lambda: combine(weights=z(4, 2, dtype=F32).requires_grad_()),
    "combine_backward_dy": lambda: combine_backward(dy=z(5, H)),
    "combine_backward_hidden": lambda: combine_backward(rows=z(9, H + 1)),
    "combine_backward_out": lambda: combine_backward(drows=z(8, H)),
    "combine_backward_out_type": lambda: combine_backward(drows=z(9, H, dtype=F32)),
    "combine_backward_weights": lambda: combine_backward(weights=z(8, dtype=F32)),
    "combine_backward_slots": lambda: combine_backward(weights=z(4, 17, dtype=F32), dweights=z(4, 17, dtype=F32), pair_row=z(68, dtype=I32)),
    "combine_backward_dweights": lambda: combine_backward(dweights=z(2, 4, dtype=F32)),
    "combine_backward_pairs": lambda: combine_backward(pair_row=z(7, dtype=I32)),
}


@pytest.mark.parametrize("case", sorted(REFUSED))
def test_refused(case):
    with pytest.raises(ValueError):
        REFUSED[case]()


@pytest.mark.parametrize("eps", [0, -1e-6, float("inf"), float("nan"), 1e-60, 1e60, "1", None])
def test_eps_is_a_positive_number(eps):
    with pytest.raises(ValueError, match="eps"):
        moe.rms_norm(z(2, 8), out=z(2, 8), eps=eps)


def test_names_of_formats():
    with pytest.raises(ValueError, match="quantize"):
        moe.rms_norm(z(2, 8), quantize="e4m3")
    with pytest.raises(ValueError, match="quantize"):
        moe.rms_norm(z(2, 8), quantize=["fp8"])
    with pytest.raises(ValueError, match="element"):
        moe.quantize_mx(z(2, 8), "fp8")


def test_host_tensors_are_refused():
    for call in (lambda: moe.rms_norm(z(2, 8)), lambda: moe.quantize_mx(z(2, 8)), lambda: moe.rms_norm_backward(z(2, 8), z(2, 8)),
                 lambda: moe.mx_matmul(z(2, 8, dtype=F8), z(2, 1, dtype=U8), z(3, 4, dtype=U8), z(3, 1, dtype=U8), out=z(2, 3)),
                 lambda: moe.combine_rows_backward(z(2, 8), z(4, 8), z(4, dtype=I32), z(2, 2, dtype=F32))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def dual(*shape, dtype=BF):
    return forward_ad.make_dual(torch.zeros(*shape, dtype=dtype), torch.ones(*shape, dtype=dtype))


@pytest.mark.parametrize("case", ["norm", "norm_weight", "backward", "quantize", "combine", "combine_backward"])
def test_tangents_are_refused(case):
    calls = {"norm": lambda: norm(x=dual(R, H)), "norm_weight": lambda: norm(weight=dual(H)), "backward": lambda: norm_backward(dy=dual(R, H)),
             "quantize": lambda: quantize(x=dual(R, K)), "combine": lambda: combine(weights=dual(4, 2, dtype=F32)),
             "combine_backward": lambda: combine_backward(rows=dual(9, H))}
    with forward_ad.dual_level(), torch.no_grad(), pytest.raises(ValueError, match="tangent"):
        calls[case]()


ROWS, COLS, STRIDE, MATRIX = 1 << 28, 1 << 20, 1 << 32, 1 << 52
LIMITS = {   # a size at its limit with 0, past it with 1
    "norm_rows": lambda d: norm(x=meta(ROWS + d, 8), weight=None, out=meta(ROWS + d, 8)),
    "norm_hidden": lambda d: norm(x=meta(2, COLS + d), weight=None, out=meta(2, COLS + d)),
    "norm_stride": lambda d: norm(x=stretched((2, 8), (STRIDE + d, 1)), weight=None, out=meta(2, 8)),
    "norm_backward_stride": lambda d: norm_backward(dy=meta(2, 8), x=meta(2, 8), weight=None, dx=stretched((2, 8), (STRIDE + d, 1))),
    "quantize_rows": lambda d: quantize(x=meta(ROWS + d, 8), codes=meta(ROWS + d, 4, dtype=U8), scales=meta(ROWS + d, 1, dtype=U8)),
    "quantize_batch": lambda d: quantize(x=meta(65535 + d, 1, 8), codes=meta(65535 + d, 1, 4, dtype=U8), scales=meta(65535 + d, 1, 1, dtype=U8)),
    "quantize_matrix_stride": lambda d: quantize(x=meta(2, 1, 8), codes=stretched((2, 1, 4), (MATRIX + d, 4, 1), U8), scales=meta(2, 1, 1, dtype=U8)),
    "product_rows": lambda d: product(x=meta(ROWS + d, 8, dtype=F8), x_scales=meta(ROWS + d, 1, dtype=U8), w=meta(8, 4, dtype=U8),
                                      w_scales=meta(8, 1, dtype=U8), y=meta(ROWS + d, 8)),
    "product_k": lambda d: product(x=meta(2, COLS // 2 + d, dtype=U8), x_scales=meta(2, COLS // 32 + d, dtype=U8), w=meta(8, COLS // 2 + d, dtype=U8),
                                   w_scales=meta(8, COLS // 32 + d, dtype=U8), y=meta(2, 8)),
    "product_n": lambda d: product(x=meta(2, 8, dtype=F8), x_scales=meta(2, 1, dtype=U8), w=meta(COLS + d, 4, dtype=U8),
                                   w_scales=meta(COLS + d, 1, dtype=U8), y=meta(2, COLS + d)),
    "combine_backward_tokens": lambda d: combine_backward(
        dy=meta((1 << 23) + d, 8), rows=meta(4, 8), pair_row=meta((1 << 23) + d, dtype=I32), weights=meta((1 << 23) + d, 1, dtype=F32),
        drows=meta(4, 8), dweights=meta((1 << 23) + d, 1, dtype=F32)),
}


@pytest.mark.parametrize("name", sorted(LIMITS))
def test_sizes_past_the_limits_are_refused(name):
    LIMITS[name](0)
    with pytest.raises(ValueError):
        LIMITS[name](1)


def test_weighted_combine_takes_more_tokens_in_pieces(monkeypatch):
    made = []
    monkeypatch.setattr(ops, "_first_call", lambda name, check, args, *rest: made.append((name, check(*args), args)))
    monkeypatch.setattr(ops, "_MAX_TOKENS", 100)
    rows, out, at, w = z(8, 16), z(230, 16), z(230, 3, dtype=I32), torch.rand(230, 3)
    assert ops.combine_rows(rows, at, 3, out=out, weights=w) is out
    assert [p.tokens for _, p, _ in made] == [100, 100, 30] and {n for n, _, _ in made} == {"moe_combine_weighted_rows"}
    for n, (_, _, args) in zip((0, 100, 200), made):
        assert args[4].data_ptr() == w[n:].data_ptr() and args[4].numel() == 3 * args[3].shape[0]


# ---- C entry points -------------------------------------------------------------------

NORM = dict(rows=4, hidden=16, stream_dtype=1, weight_dtype=1, format=0, weight_gradient=1, eps=1e-6, ld_x=16, ld_residual=16, ld_residual_out=16,
            ld_out=16, ld_scales=1, ld_dy=16, ld_dresidual=16, ld_dx=16, workspace_bytes=1 << 20)
MXQ = dict(rows=4, batch=2, cols=33, format=1, in_dtype=1, num_experts=2, ld_x=33, ld_codes=17, ld_scales=2, batch_stride_x=132,
           batch_stride_codes=68, batch_stride_scales=8)
MX = dict(num_experts=2, rows=4, expected_rows=0, n=8, k=64, ld_x=64, ld_x_scales=2, ld_w=32, ld_w_scales=2, ld_y=8, expert_stride_w=256,
          expert_stride_w_scales=16, x_format=0, out_dtype=1, tile=0, splits=0, workspace_bytes=0)
BACK = dict(tokens=4, rows=8, top_k=2, hidden=16, dy_dtype=1, ld_dy=16, ld_rows=16, ld_drows=16)
C = {   # parameters, values refused one by one, alignment of each pointer, pointers that may be NULL
    "moe_rms_norm": (_lib.MoeNormParams, NORM, [("rows", -1), ("rows", ROWS + 1), ("hidden", 0), ("hidden", COLS + 1), ("stream_dtype", 2),
                                                ("weight_dtype", -1), ("format", 5), ("format", -1), ("eps", 0.0), ("eps", float("nan")),
                                                ("eps", float("inf")), ("ld_x", 15), ("ld_residual", 15), ("ld_residual_out", 15), ("ld_out", 15),
                                                ("ld_x", STRIDE + 1)], (2, 2, 2, 2, 1, 2), (2, 4)),
    "moe_rms_norm_backward": (_lib.MoeNormParams, NORM, [("rows", -1), ("hidden", 0), ("format", 2), ("eps", -1.0), ("ld_x", 15), ("ld_dy", 15),
                                                         ("ld_dresidual", 15), ("ld_dx", 15), ("weight_gradient", 0), ("workspace_bytes", -1)],
                              (2, 2, 2, 2, 2, 4, 16), (2, 3)),
    "moe_quantize_mx": (_lib.MoeMxQuantizeParams, {**MXQ, "batch": 1}, [("rows", -1), ("batch", 0), ("batch", 65536), ("cols", 0), ("format", 2), ("in_dtype", 2),
                                                           ("ld_x", 32), ("ld_codes", 16), ("ld_scales", 1), ("num_experts", 0), ("num_experts", 257)],
                        (2, 4, 1, 1), (1,)),
    "moe_mx_matmul": (_lib.MoeMxParams, MX, [("num_experts", 0), ("num_experts", 257), ("rows", -1), ("expected_rows", -1), ("n", 0), ("k", 0),
                                             ("k", COLS + 1), ("ld_x", 63), ("ld_x_scales", 1), ("ld_w", 31), ("ld_w_scales", 1), ("ld_y", 7),
                                             ("expert_stride_w", 255), ("expert_stride_w_scales", 15), ("x_format", 2), ("out_dtype", 2),
                                             ("tile", -1), ("splits", -1), ("splits", 65), ("workspace_bytes", -1)], (4, 1, 1, 1, 1, 2, 16), (6,)),
    "moe_combine_weighted_rows": (_lib.MoeRowsParams, dict(tokens=4, rows=8, top_k=2, hidden=16, elem_bytes=2, num_experts=0, out_dtype=1, ld_tokens=16,
                                                           ld_rows=16), [("tokens", -1), ("top_k", 0), ("top_k", 17), ("elem_bytes", 4), ("ld_rows", 15)],
                                  (2, 4, 4, 2), ()),
    "moe_combine_rows_backward": (_lib.MoeCombineBackwardParams, BACK, [("tokens", -1), ("tokens", (1 << 23) + 1), ("rows", -1), ("top_k", 0), ("top_k", 17),
                                                                        ("hidden", 0), ("dy_dtype", 2), ("ld_dy", 15), ("ld_rows", 15), ("ld_drows", 15)],
                                  (2, 2, 4, 4, 2, 4), ()),
}


@pytest.mark.parametrize("name", sorted(C))
def test_c_entries_refuse(name):
    kind, good, bad, need, optional = C[name]
    fn = getattr(_lib_or_skip(), name)
    some = [1 << 20] * len(need)

    def call(values, ptrs):
        return fn(ctypes.byref(kind(**values)), *ptrs, None)

    assert fn(None, *some, None) == _lib.MOE_ERR_INVALID_ARG
    for field, value in bad:
        assert call({**good, field: value}, some) == _lib.MOE_ERR_INVALID_ARG, (field, value)
    for i, n in enumerate(need):
        for by in range(1, n):
            ptrs = list(some)
            ptrs[i] += by
            assert call(good, ptrs) == _lib.MOE_ERR_INVALID_ARG, (i, by)
        if i not in optional and not (name == "moe_rms_norm_backward" and i == 6):
            ptrs = list(some)
            ptrs[i] = None
            assert call(good, ptrs) == _lib.MOE_ERR_INVALID_ARG, i
    # no rows (tokens): in order, and nothing is launched
    none = {**good, ("tokens" if "tokens" in good else "rows"): 0}
    if name == "moe_rms_norm_backward":
        none["weight_gradient"] = 0
        some[5] = None
    assert call(none, some) == _lib.MOE_OK


def test_c_entries_refuse_more():
    lib = _lib_or_skip()
    p = 1 << 20
    fn = lib.moe_rms_norm
    for form, ld in ((_lib.MOE_NORM_FP8, 0), (_lib.MOE_NORM_MX_E4M3, 0)):
        q = _lib.MoeNormParams(**{**NORM, "format": form, "ld_scales": ld})
        assert fn(ctypes.byref(q), p, p, p, p, p, p, None) == _lib.MOE_ERR_INVALID_ARG
        q = _lib.MoeNormParams(**{**NORM, "format": form})
        assert fn(ctypes.byref(q), p, p, p, p, None, p, None) == _lib.MOE_ERR_INVALID_ARG   # no scales
    q = _lib.MoeNormParams(**{**NORM, "format": _lib.MOE_NORM_FP8})
    assert fn(ctypes.byref(q), p, p, p, p, p + 2, p, None) == _lib.MOE_ERR_INVALID_ARG
    # the weight gradient's workspace
    q = _lib.MoeNormParams(**NORM)
    need = lib.moe_rms_norm_workspace_bytes(ctypes.byref(_lib.MoeNormParams(**{**NORM, "rows": 5000, "hidden": 4096, "ld_x": 4096, "ld_dy": 4096, "ld_dx": 4096})))
    assert need > 0 and need % (4096 * 4) == 0
    small = _lib.MoeNormParams(**{**NORM, "rows": 5000, "hidden": 4096, **{f: 4096 for f in NORM if f.startswith("ld_")}, "workspace_bytes": need - 1})
    assert lib.moe_rms_norm_backward(ctypes.byref(small), p, p, p, p, p, p, p, None) == _lib.MOE_ERR_WORKSPACE_TOO_SMALL
    assert lib.moe_rms_norm_backward(ctypes.byref(small), p, p, p, p, p, p, None, None) == _lib.MOE_ERR_WORKSPACE_TOO_SMALL
    for change in (dict(weight_gradient=0), dict(rows=0), dict(hidden=0)):
        assert lib.moe_rms_norm_workspace_bytes(ctypes.byref(_lib.MoeNormParams(**{**NORM, **change}))) == 0
    # batches: matrices that overlap, offsets that go with one
    for change in (dict(batch_stride_x=131), dict(batch_stride_codes=67), dict(batch_stride_scales=7)):
        q = _lib.MoeMxQuantizeParams(**{**MXQ, **change})
        assert lib.moe_quantize_mx(ctypes.byref(q), p, None, p, p, None) == _lib.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_mx(ctypes.byref(_lib.MoeMxQuantizeParams(**MXQ)), p, p, p, p, None) == _lib.MOE_ERR_INVALID_ARG
    # an odd sum of packed rows, experts without offsets, a tile that is none
    assert lib.moe_mx_matmul(ctypes.byref(_lib.MoeMxParams(**{**MX, "x_format": 1, "k": 63})), p, p, p, p, p, p, None, None) == _lib.MOE_ERR_INVALID_ARG
    assert lib.moe_mx_matmul(ctypes.byref(_lib.MoeMxParams(**MX)), None, p, p, p, p, p, None, None) == _lib.MOE_ERR_INVALID_ARG
    assert lib.moe_mx_matmul(ctypes.byref(_lib.MoeMxParams(**{**MX, "tile": 99})), p, p, p, p, p, p, None, None) == _lib.MOE_ERR_UNSUPPORTED
    assert lib.moe_mx_workspace_bytes(None) == 0
