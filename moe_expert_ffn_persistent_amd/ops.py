"""Operators around the expert FFN (include/moe_ffn.h, "Operators around the
expert FFN"): rows dispatched to and combined from the local experts, matrix
products grouped by expert with their gradients, SwiGLU, quantisation to e4m3
with block scales and the block-scaled e4m3 product, RMS norm of the residual
stream with its gradients, quantisation to the OCP Microscaling (MX) formats and
their product.

Every call checks its tensors on the host (ValueError before anything is
enqueued), enqueues one or a few kernels on ``stream`` (a torch.cuda.Stream;
default: the current stream of the tensors' device) and returns without waiting. With
``out`` given nothing is allocated, but for the workspace of a product that cuts
its sum (see grouped_matmul) or of rms_norm_backward, and the call may be captured in a HIP graph. ``out`` must not overlap an input unless a function says it may. When a
call allocates its output, rows that no expert owns hold whatever the memory
held. Tensors used on a stream other than the one they were allocated on need
the caller's ``record_stream``, as everywhere in torch.

The functions record nothing for autograd; gradients are the operators named
so. Given a tensor that requires grad while grad mode is on, or one that carries
a forward-mode tangent, they raise rather than return a tensor that silently cuts
the graph: call them inside a torch.autograd.Function or, where no tangents are,
under torch.no_grad(). What a call writes gets a new version, so torch notices
when that was saved for a backward pass.
"""
from __future__ import annotations

import ctypes
import functools
import struct
import warnings

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import (MOE_GROUPED_DGRAD, MOE_GROUPED_FORWARD, MOE_GROUPED_WGRAD, MOE_MAX_LOCAL_EXPERTS,
                   MOE_MX_E2M1, MOE_MX_E4M3, MOE_NORM_BF16, MOE_NORM_FP32, MOE_NORM_FP8, MOE_NORM_MX_E2M1,
                   MOE_NORM_MX_E4M3, MOE_SWIGLU_BF16, MOE_SWIGLU_FP8, MOE_Y_BF16, MOE_Y_FP32,
                   MoeCombineBackwardParams, MoeFp8Params, MoeGroupedParams, MoeMxParams, MoeMxQuantizeParams,
                   MoeNormParams, MoeQuantizeParams, MoeRowsParams, MoeSwigluParams)

BLOCK = 128   # columns of one fp32 scale
MX_BLOCK = 32   # elements of one E8M0 scale
_OUT = {torch.bfloat16: MOE_Y_BF16, torch.float32: MOE_Y_FP32}
_CODES = (torch.float8_e4m3fn, torch.uint8)
_MX = {"e4m3": MOE_MX_E4M3, "e2m1": MOE_MX_E2M1}
_PAIRS = tuple(t for t in (torch.uint8, getattr(torch, "float4_e2m1fn_x2", None)) if t is not None)   # two e2m1 codes
_E8M0 = tuple(t for t in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if t is not None)
_NORM = {None: MOE_NORM_BF16, "fp8": MOE_NORM_FP8, "mx_e4m3": MOE_NORM_MX_E4M3, "mx_e2m1": MOE_NORM_MX_E2M1}
# the C entry points' limits
_MAX_ROWS, _MAX_COLS, _MAX_STRIDE, _MAX_MATRIX = 1 << 28, 1 << 20, 1 << 32, 1 << 52
_MAX_TOKENS = 1 << 23    # of one moe_combine_rows, weighted or not, or moe_combine_rows_backward
_MAX_BATCH, _MAX_BLOCKS = 65535, (1 << 23) - 1   # quantisation: matrices; 128 x 128 blocks of one
_MAX_SPLITS = 64


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _on(device, *named):
    """Every tensor given is on ``device``, and neither grad mode would be cut."""
    grad = torch.is_grad_enabled()
    for what, t in named:
        if t is None:
            continue
        if t.device != device:
            raise ValueError(f"{what}: on {t.device}, need {device}")
        if t.is_neg():
            raise ValueError(f"{what}: a view with a pending negation (resolve_neg() makes it a tensor)")
        if grad and t.requires_grad:
            raise ValueError(f"{what} requires grad, and this operator records nothing for autograd: "
                             "call it in a torch.autograd.Function or under torch.no_grad()")
        if t.is_floating_point() and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{what} carries a forward-mode tangent, and this operator records nothing for autograd: "
                             "call it in a torch.autograd.Function with a jvp")


def _matrix(t, what, dtypes, dims=2, most=_MAX_COLS):
    """A tensor of ``dims`` dimensions and one of ``dtypes`` whose rows are
    contiguous, of at most ``most`` elements, and do not overlap; returns the row
    stride."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: need a tensor, got {type(t).__name__}")
    if t.dim() != dims:
        raise ValueError(f"{what}: need {dims} dimensions, got shape {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: need dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    rows, cols = t.shape[-2:]
    if cols < 1:
        raise ValueError(f"{what}: rows of no elements")
    if cols > most:
        raise ValueError(f"{what}: rows of {cols} elements, at most {most} are taken")
    st = t.stride()
    if cols > 1 and st[-1] != 1:
        raise ValueError(f"{what}: rows must be contiguous (last stride 1, got {st[-1]})")
    ld = st[-2] if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}: rows overlap (row stride {ld} under {cols} columns)")
    if ld > _MAX_STRIDE:
        raise ValueError(f"{what}: row stride {ld}, at most {_MAX_STRIDE} is taken")
    return ld


def _at_most(n, what, most):
    if n > most:
        raise ValueError(f"{what}: {n}, at most {most} are taken")


def _batch_stride(t, what, ld):
    """Stride between the matrices of a 3-D tensor, which must not overlap."""
    need = (t.shape[1] - 1) * ld + t.shape[2]
    if t.shape[0] > 1 and t.stride(0) < need:
        raise ValueError(f"{what}: matrices overlap (stride {t.stride(0)} under {need} elements)")
    if t.shape[0] > 1 and t.stride(0) > _MAX_MATRIX:
        raise ValueError(f"{what}: stride {t.stride(0)} between matrices, at most {_MAX_MATRIX} is taken")
    return t.stride(0) if t.shape[0] > 1 else need


def _vector(t, what, n, dtype):
    """A contiguous tensor of ``n`` elements of ``dtype``, any shape."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what}: need a contiguous {dtype} tensor of {n} elements")


def _indices(t, what):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous int32 tensor")


def _offsets(t):
    """Experts of a row_offset tensor (int32 [L+1])."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("row_offset: need a contiguous int32 tensor [L+1]")
    L = t.numel() - 1
    if not 1 <= L <= MOE_MAX_LOCAL_EXPERTS:
        raise ValueError(f"row_offset: {L} experts, need 1 to {MOE_MAX_LOCAL_EXPERTS}")
    return L


def _expected(expected_rows):
    if expected_rows is None:
        return 0
    if expected_rows < 1:
        raise ValueError(f"expected_rows: need at least 1, got {expected_rows}")
    return int(expected_rows)


def _choice(tile, splits):
    """Numbers that name a kernel (an id that a call cannot take is MoeError)."""
    if tile < 0:
        raise ValueError(f"tile: need an id, or 0 for automatic, got {tile}")
    if not 0 <= splits <= _MAX_SPLITS:
        raise ValueError(f"splits: need 1 to {_MAX_SPLITS}, or 0 for automatic, got {splits}")


def _need_device(device):
    if device.type != "cuda":
        raise ValueError(f"need tensors on a GPU, got {device}")


def _sizes(t, what, dims):
    """Shape of an input that an output is allocated for (all else about it is
    checked with the call)."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{what}: need a tensor of {dims} dimensions")
    if not t.is_cuda:
        _need_device(t.device)
    return t.shape


def _type(t):
    return t.dtype if isinstance(t, torch.Tensor) else None


def _out_type(dtype):
    if dtype not in _OUT:
        raise ValueError(f"out_dtype: need bfloat16 or float32, got {dtype}")
    return dtype


def _empty(shape, dtype, device, stream):
    """An output for work on ``stream``, allocated for that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check_stream(stream, device.index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


_ENTRY: dict = {}   # entry point -> its address, once it has been called
_get_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_again = _remember = None   # the compiled call path, once it is loaded
_no_call_path = False       # it has not been built


def _check_stream(stream, device):
    """``stream`` is one of the tensors' device (an index)."""
    at = getattr(stream, "device_index", None)
    if at is None:
        raise ValueError(f"stream: need a torch.cuda.Stream, got {type(stream).__name__}")
    if at != device:
        raise ValueError(f"stream: of device {at}, the tensors are on device {device}")


# calls that may take a workspace, their last pointer, and what says its size
_WORKSPACE = {"moe_grouped_matmul_split": "moe_grouped_workspace_bytes", "moe_fp8_matmul_split": "moe_fp8_workspace_bytes",
              "moe_mx_matmul": "moe_mx_workspace_bytes", "moe_rms_norm_backward": "moe_rms_norm_workspace_bytes"}


def _call(name, check, args, plain, tensors, written, stream):
    """One C entry point, ``tensors`` its pointers in order, of which it writes
    those whose bit is set in ``written``. ``check(*args)`` makes its parameters
    from their sizes and the ``plain`` arguments; for sizes that it has seen the
    call is made again without it (csrc/opcall.cpp: a call costs the host 3.9 us,
    3.4 of them the launch)."""
    entry = _ENTRY.get(name)
    if entry is not None:
        device = _get_device()
        if stream is None:
            st = _again(entry, device, _raw_stream(device), True, plain, *tensors)
        elif getattr(stream, "device_index", None) == device:
            st = _again(entry, device, stream.cuda_stream, False, plain, *tensors)
            if st is False:   # a workspace, from the memory of that stream
                with torch.cuda.stream(stream):
                    st = _again(entry, device, stream.cuda_stream, True, plain, *tensors)
        else:
            st = None
        if st is not None:
            if st != _lib.MOE_OK:
                _lib.check(st, name)
            return
    _first_call(name, check, args, plain, tensors, written, stream)


def _load_call_path():
    global _again, _remember, _no_call_path
    try:
        call = _lib.load_opcall()
    except RuntimeError as e:
        _no_call_path = True
        warnings.warn(f"{e}; every call is checked and takes longer until then", RuntimeWarning)
    else:
        _again, _remember = call.again, call.remember


def _first_call(name, check, args, plain, tensors, written, stream):
    params = check(*args)
    device = next(t for t in tensors if t is not None).device
    _need_device(device)
    if stream is not None:
        _check_stream(stream, device.index)
    lib = _lib.load()
    fn = getattr(lib, name)
    if _again is None and not _no_call_path:
        _load_call_path()
    pointers = [_ptr(t) for t in tensors]
    for t, p in zip(tensors, pointers):
        if p == 0 and t.numel():   # it would count as absent
            raise ValueError(f"a {type(t).__name__} of shape {tuple(t.shape)} holds no memory of its own")
    need = 0
    if name in _WORKSPACE:
        need = params.workspace_bytes = getattr(lib, _WORKSPACE[name])(ctypes.byref(params))
        workspace = _empty((need,), torch.uint8, device, stream) if need else None
        pointers[-1] = _ptr(workspace)
    with torch.cuda.device(device):
        s = _raw_stream(device.index) if stream is None else stream.cuda_stream
        st = fn(ctypes.byref(params), *pointers, s)
    if st != _lib.MOE_OK:
        _lib.check(st, name)
    increment_version([t for i, t in enumerate(tensors) if written >> i & 1 and t is not None])
    if _remember is None:
        return
    entry = _ENTRY[name] = ctypes.cast(fn, ctypes.c_void_p).value
    _remember(bytes(params), entry, device.index, need, plain, *tensors, written=written)


# ---- rows to and from the experts -------------------------------------------

_ROW_TYPES = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4, torch.float8_e4m3fn: 1, torch.uint8: 1,
              torch.int16: 2}


def check_dispatch_inputs(x, row_pair, row_offset, top_k, out):
    ldx = _matrix(x, "x", tuple(_ROW_TYPES))
    N, H = x.shape
    L = _offsets(row_offset)
    if not 1 <= top_k <= 16:
        raise ValueError(f"top_k: need 1 to 16, got {top_k}")
    _indices(row_pair, "row_pair")
    ldo = _matrix(out, "out", (x.dtype,))
    if out.shape[1] != H:
        raise ValueError(f"out: rows of {out.shape[1]} elements, x has {H}")
    _at_most(out.shape[0], "rows of out", _MAX_ROWS)
    if row_pair.numel() < out.shape[0]:
        raise ValueError(f"row_pair: {row_pair.numel()} entries for {out.shape[0]} rows")
    _on(x.device, ("x", x), ("row_pair", row_pair), ("row_offset", row_offset), ("out", out))
    return MoeRowsParams(N, out.shape[0], top_k, H, _ROW_TYPES[x.dtype], L, 0, ldx, ldo)


def dispatch_rows(x, row_pair, row_offset, top_k, out=None, stream=None):
    """Rows of the local experts: ``out[r] = x[row_pair[r] // top_k]`` for r in
    row_offset[0] .. row_offset[L]-1 (a layout's arrays). x [N, H] of 1-, 2- or
    4-byte elements; out [rows, H], allocated with one row for every entry of
    row_pair when not given: back to back, or as far apart as those of x where
    these are bytes with less than 16 of padding (MX codes and scales, which
    mx_matmul's tile kernels take so). The gradient of combine_rows."""
    if out is None:
        _, H = _sizes(x, "x", 2)
        _indices(row_pair, "row_pair")
        apart = x.stride(0) if x.element_size() == 1 and 0 < x.stride(0) - H < 16 else H
        out = _empty((row_pair.numel(), apart), x.dtype, x.device, stream)[:, :H]
    _call("moe_dispatch_rows", check_dispatch_inputs, (x, row_pair, row_offset, top_k, out), (top_k,),
          (x, row_pair, row_offset, out), 0b1000, stream)
    return out


class _MoreTokens(ValueError):
    """Inputs that are in order but for more tokens than one call takes."""


def check_combine_rows_inputs(rows, pair_row, top_k, out, weights=None):
    ldr = _matrix(rows, "rows", (torch.bfloat16,))
    _at_most(rows.shape[0], "rows", _MAX_ROWS)
    if not 1 <= top_k <= 16:
        raise ValueError(f"top_k: need 1 to 16, got {top_k}")
    _indices(pair_row, "pair_row")
    if pair_row.numel() % top_k:
        raise ValueError(f"pair_row: {pair_row.numel()} entries, need top_k ({top_k}) a token")
    N = pair_row.numel() // top_k
    ldo = _matrix(out, "out", tuple(_OUT))
    if tuple(out.shape) != (N, rows.shape[1]):
        raise ValueError(f"out: need shape {(N, rows.shape[1])}, got {tuple(out.shape)}")
    if weights is not None:
        _vector(weights, "weights", N * top_k, torch.float32)
    _on(rows.device, ("rows", rows), ("pair_row", pair_row), ("weights", weights), ("out", out))
    if N > _MAX_TOKENS:
        raise _MoreTokens
    return MoeRowsParams(N, rows.shape[0], top_k, rows.shape[1], 2, 0, _OUT[out.dtype], ldo, ldr)


def combine_rows(rows, pair_row, top_k, out=None, out_dtype=torch.bfloat16, stream=None, weights=None):
    """Each token's rows summed in fp32, in ascending slot order: ``out[n] =
    sum of rows[pair_row[n * top_k + j]]`` over the slots whose pair_row is not
    negative, each times ``weights[n, j]`` (fp32 [N, top_k], a layout's topk_w)
    where they are given. rows bf16 [R, H]; out [N, H] bf16 (rounded once) or
    fp32. Without weights the gradient of dispatch_rows; with them
    combine_rows_backward is its gradient."""
    if out is None:
        _, H = _sizes(rows, "rows", 2)
        _indices(pair_row, "pair_row")
        out = _empty((pair_row.numel() // max(1, top_k), H), _out_type(out_dtype), rows.device, stream)
    try:
        if weights is None:
            _call("moe_combine_rows", check_combine_rows_inputs, (rows, pair_row, top_k, out), (top_k,), (rows, pair_row, out),
                  0b100, stream)
        else:
            _call("moe_combine_weighted_rows", check_combine_rows_inputs, (rows, pair_row, top_k, out, weights), (top_k,),
                  (rows, pair_row, weights, out), 0b1000, stream)
    except _MoreTokens:
        pairs = pair_row.view(-1)
        for n in range(0, out.shape[0], _MAX_TOKENS):
            some = slice(n * top_k, (n + _MAX_TOKENS) * top_k)
            combine_rows(rows, pairs[some], top_k, out=out[n:n + _MAX_TOKENS], stream=stream,
                         weights=None if weights is None else weights.view(-1)[some])
    return out


def check_combine_backward_inputs(dy, rows, pair_row, weights, drows, dweights):
    ldy = _matrix(dy, "dy", tuple(_OUT))
    ldr = _matrix(rows, "rows", (torch.bfloat16,))
    ldd = _matrix(drows, "out", (torch.bfloat16,))
    N, H = dy.shape
    if not isinstance(weights, torch.Tensor) or weights.dim() != 2 or weights.shape[0] != N:
        raise ValueError(f"weights: need a tensor [{N}, top_k]")
    k = weights.shape[1]
    if not 1 <= k <= 16:
        raise ValueError(f"weights: {k} slots a token, need 1 to 16")
    _vector(weights, "weights", N * k, torch.float32)
    _vector(dweights, "dweights", N * k, torch.float32)
    if tuple(dweights.shape) != (N, k):
        raise ValueError(f"dweights: need shape {(N, k)}, got {tuple(dweights.shape)}")
    _vector(pair_row, "pair_row", N * k, torch.int32)
    if rows.shape[1] != H or drows.shape != rows.shape:
        raise ValueError(f"shapes do not fit: dy {tuple(dy.shape)}, rows {tuple(rows.shape)}, out {tuple(drows.shape)}")
    _at_most(rows.shape[0], "rows", _MAX_ROWS)
    _on(dy.device, ("dy", dy), ("rows", rows), ("pair_row", pair_row), ("weights", weights), ("out", drows), ("dweights", dweights))
    if N > _MAX_TOKENS:
        raise _MoreTokens
    return MoeCombineBackwardParams(N, rows.shape[0], k, H, _OUT[dy.dtype], ldy, ldr, ldd)


def combine_rows_backward(dy, rows, pair_row, weights, out=None, dweights=None, stream=None):
    """Gradients of combine_rows with weights for dy [N, H] (bf16 or fp32):
    (drows bf16 [R, H], dweights fp32 [N, top_k]), ``drows[pair_row[n, j]] =
    weights[n, j] * dy[n]`` and ``dweights[n, j] = dy[n] . rows[pair_row[n, j]]``,
    0 for slots whose pair_row is negative (or no row). Rows that no slot names
    keep what ``out`` held. Each row belongs to one slot, as in a layout. ``out``
    may be rows itself."""
    if out is None:
        out = _empty(_sizes(rows, "rows", 2), torch.bfloat16, rows.device, stream)
    if dweights is None:
        dweights = _empty(_sizes(weights, "weights", 2), torch.float32, weights.device, stream)
    try:
        _call("moe_combine_rows_backward", check_combine_backward_inputs, (dy, rows, pair_row, weights, out, dweights), (),
              (dy, rows, pair_row, weights, out, dweights), 0b110000, stream)
    except _MoreTokens:   # a row has one slot, so it is read and written by one piece
        pairs, k = pair_row.view(-1), weights.shape[1]
        for n in range(0, dy.shape[0], _MAX_TOKENS):
            some = slice(n, n + _MAX_TOKENS)
            combine_rows_backward(dy[some], rows, pairs[n * k:(n + _MAX_TOKENS) * k], weights[some], out=out, dweights=dweights[some],
                                  stream=stream)
    return out, dweights


# ---- matrix products grouped by expert ---------------------------------------

def check_grouped_inputs(op, x, w, y, row_offset, expected_rows=None, accumulate=False, tile=0, splits=0):
    """x [rows, k], w [L, n, k], y [rows, n]; the operand that ``op`` writes is
    bf16 or fp32, the others bf16."""
    bf16, out = (torch.bfloat16,), tuple(_OUT)
    ldx = _matrix(x, "x" if op != MOE_GROUPED_DGRAD else "out", out if op == MOE_GROUPED_DGRAD else bf16)
    ldw = _matrix(w, "w" if op != MOE_GROUPED_WGRAD else "out", out if op == MOE_GROUPED_WGRAD else bf16, 3)
    ldy = _matrix(y, "dy" if op != MOE_GROUPED_FORWARD else "out", out if op == MOE_GROUPED_FORWARD else bf16)
    L, n, k = w.shape
    _at_most(x.shape[0], "rows", _MAX_ROWS)
    _at_most(n, "output features", _MAX_COLS)
    _choice(tile, splits)
    if _offsets(row_offset) != L:
        raise ValueError(f"row_offset: {row_offset.numel() - 1} experts, the weights have {L}")
    if x.shape[0] != y.shape[0] or x.shape[1] != k or y.shape[1] != n:
        raise ValueError(f"shapes do not fit: [rows, k] {tuple(x.shape)}, [L, n, k] {tuple(w.shape)}, "
                         f"[rows, n] {tuple(y.shape)}")
    _on(x.device, ("rows", x), ("weights", w), ("rows", y), ("row_offset", row_offset))
    written = x if op == MOE_GROUPED_DGRAD else w if op == MOE_GROUPED_WGRAD else y
    return MoeGroupedParams(op, L, x.shape[0], _expected(expected_rows), n, k, ldx, ldw, ldy,
                            _batch_stride(w, "weights", ldw), _OUT[written.dtype], int(accumulate), tile, splits)


_GROUPED_WRITES = {MOE_GROUPED_FORWARD: 0b1000, MOE_GROUPED_DGRAD: 0b10, MOE_GROUPED_WGRAD: 0b100}   # of row_offset, x, w, y


def _grouped(op, x, w, y, row_offset, expected_rows, accumulate, tile, splits, stream):
    _call("moe_grouped_matmul_split", check_grouped_inputs,
          (op, x, w, y, row_offset, expected_rows, accumulate, tile, splits),
          (op, expected_rows, accumulate, tile, splits), (row_offset, x, w, y, None), _GROUPED_WRITES[op], stream)


def grouped_matmul(x, w, row_offset, out=None, out_dtype=torch.bfloat16, expected_rows=None, tile=0, splits=0,
                   stream=None):
    """``out[r] = w[e] @ x[r]`` for the rows r of every expert e (row_offset
    [L+1]): x bf16 [rows, k], w bf16 [L, n, k], out [rows, n] bf16 or fp32.
    ``expected_rows`` (default: all rows of x) is how many rows the experts
    hold together, when the buffers have room for many more (a layout's have room
    for every pair, and tokens * top_k * L / E of them are used by even routing):
    it only chooses the kernel's tile and ranges, and with them the order of the
    fp32 additions.
    ``tile`` (0: automatic) names the tile outright. With few
    tiles and a long sum the sum is cut into ranges that are added up in a
    workspace (allocated for the call) and joined; ``splits`` names their number
    (0: automatic, 1: not cut and no workspace)."""
    if out is None:
        rows, _ = _sizes(x, "x", 2)
        _, n, _ = _sizes(w, "w", 3)
        out = _empty((rows, n), _out_type(out_dtype), x.device, stream)
    _grouped(MOE_GROUPED_FORWARD, x, w, out, row_offset, expected_rows, False, tile, splits, stream)
    return out


def grouped_matmul_dgrad(dy, w, row_offset, out=None, out_dtype=torch.bfloat16, expected_rows=None, tile=0,
                         splits=0, stream=None):
    """Input gradient of grouped_matmul: ``out[r] = w[e].T @ dy[r]``; dy bf16
    [rows, n], out [rows, k] bf16 or fp32."""
    if out is None:
        rows, _ = _sizes(dy, "dy", 2)
        _, _, k = _sizes(w, "w", 3)
        out = _empty((rows, k), _out_type(out_dtype), dy.device, stream)
    _grouped(MOE_GROUPED_DGRAD, out, w, dy, row_offset, expected_rows, False, tile, splits, stream)
    return out


def grouped_matmul_wgrad(dy, x, row_offset, out=None, out_dtype=torch.bfloat16, accumulate=False,
                         expected_rows=None, tile=0, splits=0, stream=None):
    """Weight gradient of grouped_matmul: ``out[e] = sum over its rows of the
    outer products dy[r] x[r]``, [L, n, k] bf16 or fp32; an expert without rows
    gets zeros. With ``accumulate`` the sums are added to ``out``."""
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        _, n = _sizes(dy, "dy", 2)
        _, k = _sizes(x, "x", 2)
        out = _empty((_offsets(row_offset), n, k), _out_type(out_dtype), x.device, stream)
    _grouped(MOE_GROUPED_WGRAD, x, out, dy, row_offset, expected_rows, accumulate, tile, splits, stream)
    return out


# ---- SwiGLU -------------------------------------------------------------------

def _check_gate_up(a, row_weight, row_offset):
    lda = _matrix(a, "gate_up", (torch.bfloat16,), most=2 * _MAX_COLS)
    rows, cols = a.shape
    _at_most(rows, "rows", _MAX_ROWS)
    if cols % 2:
        raise ValueError(f"gate_up: need gate and up columns, got {cols}")
    if row_weight is not None:
        _vector(row_weight, "row_weight", rows, torch.float32)
    return rows, cols // 2, lda, 1 if row_offset is None else _offsets(row_offset)


def _half(a):
    """Rows, and columns of gate or up."""
    rows, cols = _sizes(a, "gate_up", 2)
    if cols % 2:
        raise ValueError(f"gate_up: need gate and up columns, got {cols}")
    return rows, cols // 2


def check_swiglu_inputs(a, row_weight, row_offset, h, scales):
    rows, I, lda, L = _check_gate_up(a, row_weight, row_offset)
    ldh = _matrix(h, "out", (torch.bfloat16,) + _CODES)
    if tuple(h.shape) != (rows, I):
        raise ValueError(f"out: need shape {(rows, I)}, got {tuple(h.shape)}")
    fp8 = h.dtype in _CODES
    lds = 0
    if fp8:
        lds = _matrix(scales, "scales", (torch.float32,))
        if tuple(scales.shape) != (rows, _blocks(I)):
            raise ValueError(f"scales: need shape {(rows, _blocks(I))}, got {tuple(scales.shape)}")
    elif scales is not None:
        raise ValueError("scales belong to an e4m3 output")
    _on(a.device, ("gate_up", a), ("row_weight", row_weight), ("row_offset", row_offset), ("out", h), ("scales", scales))
    return MoeSwigluParams(rows, I, L, MOE_SWIGLU_FP8 if fp8 else MOE_SWIGLU_BF16, lda, ldh, lds, 0)


def swiglu(gate_up, row_weight=None, row_offset=None, out=None, scales=None, out_dtype=torch.bfloat16, stream=None):
    """``out[r] = row_weight[r] * silu(gate) * up`` with gate, up the halves of
    gate_up [rows, 2 I] (bf16, the rows of grouped_matmul with the fused
    kernel's w1). out bf16 [rows, I]; or e4m3 (out_dtype or out
    torch.float8_e4m3fn or uint8) with fp32 ``scales`` [rows, ceil(I/128)], the
    fp32 values quantised as quantize_fp8 does: then (out, scales) is returned.
    With ``row_offset`` only the experts' rows are computed."""
    if out is None:
        rows, I = _half(gate_up)
        if out_dtype != torch.bfloat16 and out_dtype not in _CODES:
            raise ValueError(f"out_dtype: need bfloat16, float8_e4m3fn or uint8, got {out_dtype}")
        out = _empty((rows, I), out_dtype, gate_up.device, stream)
    if scales is None and _type(out) in _CODES:
        rows, I = _half(gate_up)
        scales = _empty((rows, _blocks(I)), torch.float32, gate_up.device, stream)
    _call("moe_swiglu", check_swiglu_inputs, (gate_up, row_weight, row_offset, out, scales), (),
          (gate_up, row_weight, row_offset, out, scales), 0b11000, stream)
    return out if scales is None else (out, scales)


def check_swiglu_backward_inputs(a, dh, row_weight, row_offset, da, drow_weight):
    rows, I, lda, L = _check_gate_up(a, row_weight, row_offset)
    ldh = _matrix(dh, "dh", (torch.bfloat16,))
    ldda = _matrix(da, "out", (torch.bfloat16,), most=2 * _MAX_COLS)
    if tuple(dh.shape) != (rows, I):
        raise ValueError(f"dh: need shape {(rows, I)}, got {tuple(dh.shape)}")
    if tuple(da.shape) != (rows, 2 * I):
        raise ValueError(f"out: need shape {(rows, 2 * I)}, got {tuple(da.shape)}")
    if drow_weight is not None:
        _vector(drow_weight, "drow_weight", rows, torch.float32)
    _on(a.device, ("gate_up", a), ("dh", dh), ("row_weight", row_weight), ("row_offset", row_offset), ("out", da),
        ("drow_weight", drow_weight))
    return MoeSwigluParams(rows, I, L, MOE_SWIGLU_BF16, lda, ldh, 0, ldda)


def swiglu_backward(gate_up, dh, row_weight=None, row_offset=None, out=None, drow_weight=None, stream=None):
    """Gradients of swiglu for dh bf16 [rows, I]: (dgate_up [rows, 2 I] bf16,
    drow_weight fp32 [rows]); the second is None without row_weight and
    drow_weight. ``out`` may be gate_up itself."""
    if out is None:
        rows, I = _half(gate_up)
        out = _empty((rows, 2 * I), torch.bfloat16, gate_up.device, stream)
    if drow_weight is None and row_weight is not None:
        rows, _ = _sizes(gate_up, "gate_up", 2)
        drow_weight = _empty((rows,), torch.float32, gate_up.device, stream)
    _call("moe_swiglu_backward", check_swiglu_backward_inputs, (gate_up, dh, row_weight, row_offset, out, drow_weight), (),
          (gate_up, dh, row_weight, row_offset, out, drow_weight), 0b110000, stream)
    return out, drow_weight


# ---- e4m3 with block scales ----------------------------------------------------

def _scale_shape(x, block_rows):
    return tuple(x.shape[:-2]) + (-(-x.shape[-2] // block_rows), _blocks(x.shape[-1]))


def check_quantize_inputs(x, block_rows, row_offset, codes, scales):
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows: need 1 or {BLOCK}, got {block_rows}")
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x: need a matrix or a batch of matrices")
    ldx = _matrix(x, "x", tuple(_OUT), x.dim())
    ldc = _matrix(codes, "out", _CODES, x.dim())
    if codes.shape != x.shape:
        raise ValueError(f"out: need shape {tuple(x.shape)}, got {tuple(codes.shape)}")
    shape = _scale_shape(x, block_rows)
    _at_most(x.shape[-2], "rows", _MAX_ROWS)
    _at_most(x.shape[0] if x.dim() == 3 else 1, "matrices", _MAX_BATCH)
    if block_rows != 1:
        _at_most(shape[-2] * shape[-1], f"blocks of {BLOCK} x {BLOCK}", _MAX_BLOCKS)
    if not isinstance(scales, torch.Tensor) or tuple(scales.shape) != shape:
        raise ValueError(f"scales: need shape {shape}")
    _vector(scales, "scales", scales.numel(), torch.float32)
    L = 1
    if row_offset is not None:
        if x.dim() != 2 or block_rows != 1:
            raise ValueError("row_offset goes with a matrix in 1 x 128 blocks")
        L = _offsets(row_offset)
    _on(x.device, ("x", x), ("row_offset", row_offset), ("out", codes), ("scales", scales))
    batch = x.shape[0] if x.dim() == 3 else 1
    bsx = _batch_stride(x, "x", ldx) if x.dim() == 3 else 0
    bsc = _batch_stride(codes, "out", ldc) if x.dim() == 3 else 0
    return MoeQuantizeParams(x.shape[-2], batch, x.shape[-1], block_rows, _OUT[x.dtype], L, ldx, ldc, bsx, bsc)


def quantize_fp8(x, block_rows=1, row_offset=None, out=None, scales=None, stream=None):
    """x (bf16 or fp32, [rows, cols] or [batch, rows, cols]) in the e4m3 format
    with fp32 block scales of the fp8 kernels: (codes, scales). Blocks of
    ``block_rows`` (1: activations, 128: weights) x 128 elements, scale = amax /
    448 (1 for a block of zeros), codes the e4m3 values nearest to x / scale.
    With ``row_offset`` ([rows, cols], 1 x 128 blocks) only the experts' rows."""
    if out is None or scales is None:
        if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
            raise ValueError("x: need a matrix or a batch of matrices")
        if block_rows not in (1, BLOCK):
            raise ValueError(f"block_rows: need 1 or {BLOCK}, got {block_rows}")
        _need_device(x.device)
        if out is None:
            out = _empty(x.shape, torch.float8_e4m3fn, x.device, stream)
        if scales is None:
            scales = _empty(_scale_shape(x, block_rows), torch.float32, x.device, stream)
    args = x, block_rows, row_offset, out, scales
    if isinstance(x, torch.Tensor) and x.numel() == 0:
        check_quantize_inputs(*args)
    else:
        _call("moe_quantize_fp8", check_quantize_inputs, args, (block_rows,), (x, row_offset, out, scales), 0b1100, stream)
    return out, scales


def check_fp8_inputs(x, x_scales, w, w_scales, row_offset, y, expected_rows=None, tile=0, splits=0):
    ldx = _matrix(x, "x", _CODES)
    grouped = row_offset is not None
    ldw = _matrix(w, "w", _CODES, 3 if grouped else 2)
    ldxs = _matrix(x_scales, "x_scales", (torch.float32,))
    ldy = _matrix(y, "out", tuple(_OUT))
    rows, k = x.shape
    n = w.shape[-2]
    if n < 1:
        raise ValueError("w: no output features")
    _at_most(rows, "rows", _MAX_ROWS)
    _at_most(n, "output features", _MAX_COLS)
    _choice(tile, splits)
    if w.shape[-1] != k or tuple(y.shape) != (rows, n):
        raise ValueError(f"shapes do not fit: x {tuple(x.shape)}, w {tuple(w.shape)}, out {tuple(y.shape)}")
    if tuple(x_scales.shape) != (rows, _blocks(k)):
        raise ValueError(f"x_scales: need shape {(rows, _blocks(k))}, got {tuple(x_scales.shape)}")
    shape = tuple(w.shape[:-2]) + (_blocks(n), _blocks(k))
    if not isinstance(w_scales, torch.Tensor) or tuple(w_scales.shape) != shape:
        raise ValueError(f"w_scales: need shape {shape}")
    _vector(w_scales, "w_scales", w_scales.numel(), torch.float32)
    L, es = 1, 0
    if grouped:
        L = _offsets(row_offset)
        if w.shape[0] != L:
            raise ValueError(f"row_offset: {L} experts, the weights have {w.shape[0]}")
        es = _batch_stride(w, "w", ldw)
    _on(x.device, ("x", x), ("x_scales", x_scales), ("w", w), ("w_scales", w_scales), ("row_offset", row_offset), ("out", y))
    return MoeFp8Params(L, rows, _expected(expected_rows), n, k, ldx, ldxs, ldw, ldy, es, _OUT[y.dtype],
                        tile, splits)


def fp8_matmul(x, x_scales, w, w_scales, row_offset=None, out=None, out_dtype=torch.bfloat16, expected_rows=None,
               tile=0, splits=0, stream=None):
    """``out = (x * x_scales) @ (w * w_scales).T`` of e4m3 operands: x [rows, k]
    with scales [rows, ceil(k/128)], w [n, k] with scales [ceil(n/128),
    ceil(k/128)]; grouped by expert with ``row_offset``: w [L, n, k], w_scales
    [L, ...], every row times its expert's matrix. out [rows, n] bf16 or fp32.
    ``expected_rows``, ``tile`` and ``splits`` as for grouped_matmul.

    Sums are fp32 but for one step: the matrix cores add eight products after
    dropping what lies below 2^-13 of the largest one, which puts results about
    1.5e-5 (in the norm) from fp32 sums of the same codes; an fp32 ``out`` shows
    it. Operands that are no whole multiples of 16 bytes (k, or a row stride or
    pointer; n and out's of 8 elements) take a slower kernel that multiplies
    without that step."""
    if out is None:
        rows, _ = _sizes(x, "x", 2)
        n = _sizes(w, "w", 2 if row_offset is None else 3)[-2]
        out = _empty((rows, n), _out_type(out_dtype), x.device, stream)
    _call("moe_fp8_matmul_split", check_fp8_inputs,
          (x, x_scales, w, w_scales, row_offset, out, expected_rows, tile, splits), (expected_rows, tile, splits),
          (row_offset, x, x_scales, w, w_scales, out, None), 0b100000, stream)
    return out


# ---- microscaled (MX) formats ------------------------------------------------------

def _mx_blocks(n: int) -> int:
    return -(-n // MX_BLOCK)


def _element(element):
    if not isinstance(element, str) or element not in _MX:
        raise ValueError(f"element: need 'e4m3' or 'e2m1', got {element!r}")
    return _MX[element]


def _rows_apart(shape, dtype, step, device, stream):
    """An output whose rows start a multiple of ``step`` elements apart."""
    wide = -(-shape[-1] // step) * step
    return _empty((*shape[:-1], wide), dtype, device, stream)[..., :shape[-1]]


def _empty_mx(shape, element, device, stream):
    """(codes, scales) for elements of ``shape``, as the tile kernels take them."""
    if element == MOE_MX_E4M3:
        codes = _rows_apart(shape, torch.float8_e4m3fn, 16, device, stream)
    else:
        codes = _rows_apart((*shape[:-1], -(-shape[-1] // 2)), torch.uint8, 16, device, stream)
    return codes, _rows_apart((*shape[:-1], _mx_blocks(shape[-1])), torch.uint8, 4, device, stream)


def _mx_codes(t, what, element, shape):
    """Codes of elements of ``shape``; returns the row stride in bytes."""
    ld = _matrix(t, what, _CODES if element == MOE_MX_E4M3 else _PAIRS, len(shape))
    want = tuple(shape) if element == MOE_MX_E4M3 else tuple(shape[:-1]) + (-(-shape[-1] // 2),)
    if tuple(t.shape) != want:
        raise ValueError(f"{what}: need shape {want}, got {tuple(t.shape)}")
    return ld


def _mx_scales(t, what, shape):
    """Scale bytes of elements of ``shape``; returns the row stride."""
    ld = _matrix(t, what, _E8M0, len(shape))
    want = tuple(shape[:-1]) + (_mx_blocks(shape[-1]),)
    if tuple(t.shape) != want:
        raise ValueError(f"{what}: need shape {want}, got {tuple(t.shape)}")
    return ld


def check_quantize_mx_inputs(x, element, row_offset, codes, scales):
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x: need a matrix or a batch of matrices")
    ldx = _matrix(x, "x", tuple(_OUT), x.dim())
    _at_most(x.shape[-2], "rows", _MAX_ROWS)
    _at_most(x.shape[0] if x.dim() == 3 else 1, "matrices", _MAX_BATCH)
    ldc = _mx_codes(codes, "out", element, x.shape)
    lds = _mx_scales(scales, "scales", x.shape)
    L = 1
    if row_offset is not None:
        if x.dim() != 2:
            raise ValueError("row_offset goes with a matrix")
        L = _offsets(row_offset)
    _on(x.device, ("x", x), ("row_offset", row_offset), ("out", codes), ("scales", scales))
    batch, bs = 1, (0, 0, 0)
    if x.dim() == 3:
        batch, bs = x.shape[0], (_batch_stride(x, "x", ldx), _batch_stride(codes, "out", ldc), _batch_stride(scales, "scales", lds))
    return MoeMxQuantizeParams(x.shape[-2], batch, x.shape[-1], element, _OUT[x.dtype], L, ldx, ldc, lds, *bs)


def quantize_mx(x, element="e4m3", row_offset=None, out=None, scales=None, stream=None):
    """x (bf16 or fp32, [rows, cols] or [batch, rows, cols]) in an OCP Microscaling
    format, the W4A8 kernels' operands: (codes, scales). Blocks of 32 elements of a
    row share a power of two, floor(log2(amax)) less the element's largest
    exponent (8 for "e4m3", 2 for "e2m1"), and codes are the values nearest to x
    over it, ties to even, at most the largest. codes: "e4m3" float8_e4m3fn (or
    uint8) [..., cols]; "e2m1" uint8 (or float4_e2m1fn_x2) [..., ceil(cols/2)], two a
    byte, the first in the low bits. scales: E8M0 bytes, uint8 (or float8_e8m0fnu)
    [..., ceil(cols/32)]. Both have contiguous rows, allocated 16 (scales: 4) bytes
    or multiples of that apart. With ``row_offset`` only the experts' rows."""
    element = _element(element)
    if out is None or scales is None:
        if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
            raise ValueError("x: need a matrix or a batch of matrices")
        _need_device(x.device)
        c, s = _empty_mx(x.shape, element, x.device, stream)
        out, scales = c if out is None else out, s if scales is None else scales
    args = x, element, row_offset, out, scales
    if isinstance(x, torch.Tensor) and x.numel() == 0:
        check_quantize_mx_inputs(*args)
    else:
        _call("moe_quantize_mx", check_quantize_mx_inputs, args, (element,), (x, row_offset, out, scales), 0b1100, stream)
    return out, scales


def check_mx_inputs(x, x_scales, w, w_scales, row_offset, y, expected_rows=None, tile=0, splits=0):
    """The type of x says its format: float8_e4m3fn is e4m3, uint8 (or
    float4_e2m1fn_x2) two e2m1 codes a byte."""
    ldx = _matrix(x, "x", (torch.float8_e4m3fn,) + _PAIRS)
    grouped = row_offset is not None
    ldw = _matrix(w, "w", _PAIRS, 3 if grouped else 2)
    element = MOE_MX_E4M3 if x.dtype == torch.float8_e4m3fn else MOE_MX_E2M1
    ldy = _matrix(y, "out", tuple(_OUT))
    rows, n = x.shape[0], w.shape[-2]
    k = x.shape[1] if element == MOE_MX_E4M3 else 2 * x.shape[1]
    if n < 1:
        raise ValueError("w: no output features")
    _at_most(rows, "rows", _MAX_ROWS)
    _at_most(n, "output features", _MAX_COLS)
    _at_most(k, "elements of a row", _MAX_COLS)
    _choice(tile, splits)
    if w.shape[-1] != -(-k // 2) or tuple(y.shape) != (rows, n):
        raise ValueError(f"shapes do not fit: x {tuple(x.shape)} ({k} elements), w {tuple(w.shape)} (two elements a byte), "
                         f"out {tuple(y.shape)}")
    ldxs = _mx_scales(x_scales, "x_scales", (rows, k))
    ldws = _mx_scales(w_scales, "w_scales", tuple(w.shape[:-1]) + (k,))
    L, es, ess = 1, 0, 0
    if grouped:
        L = _offsets(row_offset)
        if w.shape[0] != L:
            raise ValueError(f"row_offset: {L} experts, the weights have {w.shape[0]}")
        es, ess = _batch_stride(w, "w", ldw), _batch_stride(w_scales, "w_scales", ldws)
    _on(x.device, ("x", x), ("x_scales", x_scales), ("w", w), ("w_scales", w_scales), ("row_offset", row_offset), ("out", y))
    return MoeMxParams(L, rows, _expected(expected_rows), n, k, ldx, ldxs, ldw, ldws, ldy, es, ess, element,
                       _OUT[y.dtype], tile, splits)


def mx_matmul(x, x_scales, w, w_scales, row_offset=None, out=None, out_dtype=torch.bfloat16, expected_rows=None,
              tile=0, splits=0, stream=None):
    """``out = (x * x_scales) @ (w * w_scales).T`` of MX operands (quantize_mx): x
    float8_e4m3fn [rows, k] or two e2m1 codes a byte, uint8 [rows, k/2], scales
    [rows, ceil(k/32)]; w e2m1, uint8 [n, ceil(k/2)], scales [n, ceil(k/32)]; grouped
    by expert with ``row_offset``: w [L, n, ...], w_scales [L, n, ...], every row
    times its expert's matrix. out [rows, n] bf16 or fp32. ``expected_rows``,
    ``tile`` and ``splits`` as for grouped_matmul.

    Scales are the matrix cores' own and exact; sums are fp32 but for the bits that
    the matrix cores drop (see fp8_matmul): a partial sum past fp32's largest value
    is infinite, also where the whole sum would not be. Operands off their 16 bytes (scales off
    four), or with such strides, take a slower kernel; what quantize_mx allocates
    is on them for any k."""
    if out is None:
        rows, _ = _sizes(x, "x", 2)
        n = _sizes(w, "w", 2 if row_offset is None else 3)[-2]
        out = _empty((rows, n), _out_type(out_dtype), x.device, stream)
    _call("moe_mx_matmul", check_mx_inputs,
          (x, x_scales, w, w_scales, row_offset, out, expected_rows, tile, splits), (expected_rows, tile, splits),
          (row_offset, x, x_scales, w, w_scales, out, None), 0b100000, stream)
    return out


# ---- RMS norm of the residual stream -------------------------------------------------

@functools.lru_cache(maxsize=64)
def _fp32_bits(v):
    return struct.unpack("<i", struct.pack("<f", float(v)))[0]


def _bits(eps):
    """The fp32 bits of eps, by which a call is remembered."""
    if isinstance(eps, (int, float)):
        try:
            bits = _fp32_bits(eps)
        except OverflowError:
            bits = 0
        if 0 < bits < 0x7f800000:   # above 0 and below infinity, no NaN
            return bits
    raise ValueError(f"eps: need a positive number, got {eps!r}")


def _eps(bits):
    return struct.unpack("<f", struct.pack("<i", bits))[0]


def _norm_weight(weight, hidden):
    if weight is None:
        return MOE_Y_FP32
    if not isinstance(weight, torch.Tensor) or weight.dtype not in _OUT or not weight.is_contiguous() or tuple(weight.shape) != (hidden,):
        raise ValueError(f"weight: need a contiguous bfloat16 or float32 tensor of {hidden} elements")
    return _OUT[weight.dtype]


def check_rms_norm_inputs(x, weight, residual, eps, quantize, out, scales, residual_out):
    ldx = _matrix(x, "x", tuple(_OUT))
    rows, H = x.shape
    _at_most(rows, "rows", _MAX_ROWS)
    wt = _norm_weight(weight, H)
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    ldr = ldo = lds = 0
    if residual is not None:
        ldr, ldo = _matrix(residual, "residual", (x.dtype,)), _matrix(residual_out, "residual_out", (x.dtype,))
        for t, what in ((residual, "residual"), (residual_out, "residual_out")):
            if t.shape != x.shape:
                raise ValueError(f"{what}: need shape {tuple(x.shape)}, got {tuple(t.shape)}")
    if quantize == MOE_NORM_BF16:
        ldy = _matrix(out, "out", tuple(_OUT))
        form = MOE_NORM_BF16 if out.dtype == torch.bfloat16 else MOE_NORM_FP32
        if out.shape != x.shape:
            raise ValueError(f"out: need shape {tuple(x.shape)}, got {tuple(out.shape)}")
        if scales is not None:
            raise ValueError("scales belong to a quantised output")
    elif quantize == MOE_NORM_FP8:
        form, ldy, lds = quantize, _matrix(out, "out", _CODES), _matrix(scales, "scales", (torch.float32,))
        if out.shape != x.shape or tuple(scales.shape) != (rows, _blocks(H)):
            raise ValueError(f"out, scales: need shapes {tuple(x.shape)} and {(rows, _blocks(H))}, got {tuple(out.shape)} and "
                             f"{tuple(scales.shape)}")
    else:
        form, element = quantize, MOE_MX_E4M3 if quantize == MOE_NORM_MX_E4M3 else MOE_MX_E2M1
        ldy, lds = _mx_codes(out, "out", element, x.shape), _mx_scales(scales, "scales", x.shape)
    _on(x.device, ("x", x), ("residual", residual), ("weight", weight), ("out", out), ("scales", scales),
        ("residual_out", residual_out))
    return MoeNormParams(rows, H, _OUT[x.dtype], wt, form, 0, _eps(eps), ldx, ldr, ldo, ldy, lds, 0, 0, 0, 0)


def rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, scales=None, residual_out=None, quantize=None,
             out_dtype=torch.bfloat16, stream=None):
    """RMS norm of the residual stream s = x + residual (x without one), rounded to
    the stream's type (x and residual both bf16 or both fp32, [rows, hidden]) and
    stored in ``residual_out``: ``out = s / sqrt(mean(s^2) + eps) * weight``, fp32
    throughout, weight bf16 or fp32 [hidden] or None (1).

    ``quantize`` None: out bf16 or fp32. "fp8": e4m3 codes with fp32 scales
    [rows, ceil(hidden/128)], as quantize_fp8 quantises the fp32 values, for
    fp8_matmul. "mx_e4m3" or "mx_e2m1": codes and E8M0 scale bytes as quantize_mx
    makes them, for mx_matmul.

    Returns out; (out, scales) when quantised; with residual, residual_out behind
    them: (out, residual_out) or (out, scales, residual_out). ``residual_out`` may be
    x or residual, and ``out`` x where the types agree. What ``out`` holds in
    quantised form is never rounded to bf16 before."""
    if not isinstance(quantize, (str, type(None))) or quantize not in _NORM:
        raise ValueError(f"quantize: need None, 'fp8', 'mx_e4m3' or 'mx_e2m1', got {quantize!r}")
    form = _NORM[quantize]
    if out is None or (scales is None and quantize is not None) or (residual is not None and residual_out is None):
        rows, H = _sizes(x, "x", 2)
        if quantize in ("mx_e4m3", "mx_e2m1"):
            if out is None or scales is None:
                c, s = _empty_mx((rows, H), _MX[quantize[3:]], x.device, stream)
                out, scales = c if out is None else out, s if scales is None else scales
        elif quantize == "fp8":
            out = _empty((rows, H), torch.float8_e4m3fn, x.device, stream) if out is None else out
            scales = _empty((rows, _blocks(H)), torch.float32, x.device, stream) if scales is None else scales
        elif out is None:
            out = _empty((rows, H), _out_type(out_dtype), x.device, stream)
        if residual is not None and residual_out is None:
            residual_out = _empty((rows, H), x.dtype, x.device, stream)
    eps = _bits(eps)
    _call("moe_rms_norm", check_rms_norm_inputs, (x, weight, residual, eps, form, out, scales, residual_out), (form, eps),
          (x, residual, weight, out, scales, residual_out), 0b111000, stream)
    got = [out] + ([scales] if scales is not None else []) + ([residual_out] if residual is not None else [])
    return got[0] if len(got) == 1 else tuple(got)


def check_rms_norm_backward_inputs(dy, x, weight, eps, dresidual, dx, dweight):
    ldy, ldx, ldd = _matrix(dy, "dy", tuple(_OUT)), _matrix(x, "x", tuple(_OUT)), 0
    rows, H = x.shape
    _at_most(rows, "rows", _MAX_ROWS)
    wt = _norm_weight(weight, H)
    ldo = _matrix(dx, "out", (x.dtype,))
    if dresidual is not None:
        ldd = _matrix(dresidual, "dresidual", (x.dtype,))
    for t, what in ((dy, "dy"), (dx, "out"), (dresidual, "dresidual")):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{what}: need shape {tuple(x.shape)}, got {tuple(t.shape)}")
    if dweight is not None:
        _vector(dweight, "dweight", H, torch.float32)
    _on(dy.device, ("dy", dy), ("x", x), ("weight", weight), ("dresidual", dresidual), ("out", dx), ("dweight", dweight))
    return MoeNormParams(rows, H, _OUT[x.dtype], wt, MOE_NORM_BF16 if dy.dtype == torch.bfloat16 else MOE_NORM_FP32,
                         int(dweight is not None), _eps(eps), ldx, 0, 0, 0, 0, ldy, ldd, ldo, 0)


def rms_norm_backward(dy, x, weight=None, eps=1e-6, dresidual=None, out=None, dweight=None, stream=None):
    """Gradients of rms_norm (without quantize) for dy [rows, hidden] bf16 or fp32:
    (dx, dweight). ``x`` is the stream that was normalised: rms_norm's residual_out,
    or its x where it had no residual. dx, of x's type and rounded once, is the
    gradient of x and of residual alike; ``dresidual`` (x's type) is the gradient
    that reaches residual_out from elsewhere and is added to it. dweight is fp32
    [hidden], summed in an order that sizes alone settle (partial sums in a
    workspace, allocated for the call); None without weight and dweight. ``out`` may
    be dresidual or x, or dy where the types agree."""
    if out is None:
        out = _empty(_sizes(x, "x", 2), x.dtype, x.device, stream)
    if dweight is None and weight is not None:
        _, H = _sizes(x, "x", 2)
        dweight = _empty((H,), torch.float32, x.device, stream)
    eps = _bits(eps)
    _call("moe_rms_norm_backward", check_rms_norm_backward_inputs, (dy, x, weight, eps, dresidual, out, dweight), (eps,),
          (dy, x, weight, dresidual, out, dweight, None), 0b110000, stream)
    return out, dweight
