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
