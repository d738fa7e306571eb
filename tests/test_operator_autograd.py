"""The operators record nothing for autograd: what would silently lose a
gradient is refused (host tensors, no GPU needed)."""
import ctypes
import os

import pytest
import torch
from torch.autograd import forward_ad

from moe_expert_ffn_persistent_amd import _lib, build, ops

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HOST = -1   # device index of host tensors


def dual(*shape, dtype=BF):
    return forward_ad.make_dual(torch.zeros(*shape, dtype=dtype), torch.ones(*shape, dtype=dtype))


def checks():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)   # noqa: E731
    off, i32 = torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    return {
        "dispatch": lambda: ops.check_dispatch_inputs(dual(4, 8), i32, off, 2, z(8, 8)),
        "combine": lambda: ops.check_combine_rows_inputs(dual(8, 8), i32, 2, z(4, 8)),
        "grouped_x": lambda: ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, dual(4, 8), z(2, 8, 8), z(4, 8), off),
        "grouped_w": lambda: ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, z(4, 8), dual(2, 8, 8), z(4, 8), off),
        "grouped_out": lambda: ops.check_grouped_inputs(_lib.MOE_GROUPED_FORWARD, z(4, 8), z(2, 8, 8), dual(4, 8), off),
        "swiglu": lambda: ops.check_swiglu_inputs(dual(4, 16), None, None, z(4, 8), None),
        "swiglu_weight": lambda: ops.check_swiglu_inputs(z(4, 16), dual(4, dtype=F32), None, z(4, 8), None),
        "swiglu_backward": lambda: ops.check_swiglu_backward_inputs(z(4, 16), dual(4, 8), None, None, z(4, 16), None),
        "quantize": lambda: ops.check_quantize_inputs(dual(4, 8), 1, None, z(4, 8, dtype=F8), z(4, 1, dtype=F32)),
        "fp8_scales": lambda: ops.check_fp8_inputs(z(4, 16, dtype=F8), dual(4, 1, dtype=F32), z(8, 16, dtype=F8),
                                                   z(1, 1, dtype=F32), None, z(4, 8)),
    }


@pytest.mark.parametrize("case", sorted(checks()))
def test_tangents_are_refused(case):
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            checks()[case]()
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):   # forward mode stays on under no_grad
            checks()[case]()


def test_a_function_with_a_jvp_may_call_them():
    class F(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            ops.check_swiglu_inputs(a, None, None, torch.zeros(4, 8, dtype=BF), None)
            return a * 2

        @staticmethod
        def jvp(ctx, t):
            return t * 2

    with forward_ad.dual_level():
        out = F.apply(dual(4, 16))
        assert forward_ad.unpack_dual(out).tangent is not None


class Entry:
    def __init__(self, n, status=0):
        self.calls = 0
        kind = ctypes.CFUNCTYPE(ctypes.c_int32, ctypes.c_void_p, *[ctypes.c_void_p] * (n + 1))
        self.status = status
        self._fn = kind(self._called)
        self.address = ctypes.cast(self._fn, ctypes.c_void_p).value

    def _called(self, *a):
        self.calls += 1
        return self.status


@pytest.mark.skipif(not os.path.exists(build.OPCALL), reason="_opcall.so not built")
def test_tangents_are_refused_for_sizes_seen_before():
    opcall = _lib.load_opcall()
    entry, a, b, c = Entry(3), torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4, 8)
    assert opcall.remember(b"12345678", entry.address, HOST, 0, (), a, b, c)
    with forward_ad.dual_level():
        d = dual(4, 8, dtype=F32)
        assert opcall.again(entry.address, HOST, 0, True, (), d, b, c) is None
        assert opcall.again(entry.address, HOST, 0, True, (), a, b, d) is None
        assert not opcall.remember(b"12345678", entry.address, HOST, 0, (), d, b, c)
        assert entry.calls == 0
        assert opcall.again(entry.address, HOST, 0, True, (), a, b, c) == 0
        before = torch._C._is_fwd_grad_enabled()
        torch._C._set_fwd_grad_enabled(False)   # as inside a torch.autograd.Function
        try:
            assert opcall.again(entry.address, HOST, 0, True, (), d, b, c) == 0
        finally:
            torch._C._set_fwd_grad_enabled(before)
    assert opcall.again(entry.address, HOST, 0, True, (), a, b, c) == 0


@pytest.mark.skipif(not os.path.exists(build.OPCALL), reason="_opcall.so not built")
def test_what_a_call_of_known_sizes_writes_gets_a_new_version():
    opcall = _lib.load_opcall()
    entry, ts = Entry(4), [torch.zeros(4, 8) for _ in range(3)]
    opcall.remember(b"12345678", entry.address, HOST, 0, (), *ts, None, written=0b1110)
    for i in range(1, 4):
        assert opcall.again(entry.address, HOST, 0, True, (), *ts, None) == 0
        assert [t._version for t in ts] == [0, i, i]
    view = ts[2][1:3]
    assert view._version == 3   # a view shares its base's
    entry.status = -2           # a call that was refused wrote nothing
    assert opcall.again(entry.address, HOST, 0, True, (), *ts, None) == -2
    assert [t._version for t in ts] == [0, 3, 3]
    with torch.inference_mode():
        made = torch.zeros(4, 8)
    entry.status = 0
    assert opcall.again(entry.address, HOST, 0, True, (), ts[0], made, ts[2], None) == 0
    assert ts[2]._version == 4
    for call in (lambda: opcall.remember(b"1", entry.address, HOST, 0, (), *ts, writes=1),
                 lambda: opcall.remember(b"1", entry.address, HOST, 0, (), *ts, written="1")):
        with pytest.raises(TypeError):
            call()
