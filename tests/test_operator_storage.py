"""Tensors that wrap others and hold no memory of their own: their pointer is
null, which the C entry points take for an argument that is not there."""
import contextlib
import ctypes
import os
import types

import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib, build, ops

BF, F32 = torch.bfloat16, torch.float32


class Wrapper(torch.Tensor):
    @staticmethod
    def __new__(cls, t):
        r = torch.Tensor._make_wrapper_subclass(cls, t.shape, strides=t.stride(), dtype=t.dtype, device=t.device)
        r.inner = t
        return r

    @classmethod
    def __torch_dispatch__(cls, f, kinds, args=(), kw=None):
        return f(*[a.inner if isinstance(a, cls) else a for a in args], **(kw or {}))


def test_they_are_refused(monkeypatch):
    made = []
    monkeypatch.setattr(_lib, "load", lambda: types.SimpleNamespace(moe_swiglu=lambda p, *ptrs: made.append(ptrs) or _lib.MOE_OK))
    monkeypatch.setattr(ops, "_ENTRY", {})
    monkeypatch.setattr(ops, "_no_call_path", True)
    monkeypatch.setattr(ops, "_again", None)
    monkeypatch.setattr(ops, "_remember", None)
    monkeypatch.setattr(ops, "_need_device", lambda device: None)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    a, weight, out = torch.zeros(4, 16, dtype=BF), torch.ones(4), torch.zeros(4, 8, dtype=BF)
    moe.swiglu(a, row_weight=weight, out=out)
    assert len(made) == 1
    for kw in (dict(row_weight=Wrapper(weight)), dict(row_offset=Wrapper(torch.zeros(3, dtype=torch.int32)))):
        with pytest.raises(ValueError, match="no memory"):
            moe.swiglu(a, out=out, **kw)
    with pytest.raises(ValueError, match="no memory"):
        moe.swiglu(Wrapper(a), out=out)
    moe.swiglu(a[:0], row_weight=weight[:0], out=out[:0])   # null for tensors of no elements is in order
    assert len(made) == 2


@pytest.mark.skipif(not os.path.exists(build.OPCALL), reason="_opcall.so not built")
def test_they_are_left_to_the_checks():
    opcall = _lib.load_opcall()
    made = []
    fn = ctypes.CFUNCTYPE(ctypes.c_int32, *[ctypes.c_void_p] * 5)(lambda *p: made.append(p) or 0)
    entry = ctypes.cast(fn, ctypes.c_void_p).value
    a, b, c, none = torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4), torch.zeros(0, 4)
    assert opcall.remember(b"12345678", entry, -1, 0, (), a, b, c)
    assert not opcall.remember(b"12345678", entry, -1, 0, (), a, b, Wrapper(c))
    assert opcall.again(entry, -1, 0, True, (), a, b, Wrapper(c)) is None and not made
    assert opcall.again(entry, -1, 0, True, (), a, b, c) == 0 and len(made) == 1
    assert opcall.remember(b"12345678", entry, -1, 0, (), a, b, none) and opcall.again(entry, -1, 0, True, (), a, b, none) == 0
