"""The operators' call path for sizes checked before (csrc/opcall.cpp), on host
tensors with an entry point written here: what it calls, and that everything a
check looks at tells two calls apart."""
import ctypes
import os
import threading

import pytest
import torch

from moe_expert_ffn_persistent_amd import _lib, build

if not os.path.exists(build.OPCALL):
    pytest.skip("_opcall.so not built", allow_module_level=True)
opcall = _lib.load_opcall()

HOST = -1   # device index of host tensors
BF, F32 = torch.bfloat16, torch.float32


class Entry:
    """A C entry point of n pointers that records its calls and returns `status`."""

    def __init__(self, n, status=0):
        self.calls, self.status = [], status
        kind = ctypes.CFUNCTYPE(ctypes.c_int32, ctypes.c_void_p, *[ctypes.c_void_p] * (n + 1))
        self._fn = kind(self._called)
        self.address = ctypes.cast(self._fn, ctypes.c_void_p).value

    def _called(self, params, *ptrs):
        self.calls.append((ctypes.string_at(params, 8), ptrs[:-1], ptrs[-1]))
        return self.status


def tensors(n, dtype=BF):
    return [torch.zeros(3 + i, 8, dtype=dtype) for i in range(n)]


@pytest.mark.parametrize("n", [3, 4, 5, 6, 7])
def test_calls_with_the_parameters_and_pointers_of_the_call(n):
    entry, ts = Entry(n, status=-2), tensors(n)
    assert opcall.again(entry.address, HOST, 77, True, (), *ts) is None and not entry.calls
    assert opcall.remember(b"params of", entry.address, HOST, 0, (), *ts)
    other = [t.clone() for t in ts]   # same sizes, other memory
    other[1][0, 0] = 5
    assert opcall.again(entry.address, HOST, 77, True, (), *other) == -2
    assert entry.calls == [(b"params o", tuple(t.data_ptr() for t in other), 77)]


def test_absent_tensors_are_null_and_not_interchangeable():
    entry, (a, b, c) = Entry(3), tensors(3)
    opcall.remember(b"12345678", entry.address, HOST, 0, (), a, None, c)
    assert opcall.again(entry.address, HOST, 0, True, (), a, None, c) == 0
    assert entry.calls[0][1] == (a.data_ptr(), None, c.data_ptr()) and entry.calls[0][2] is None
    assert opcall.again(entry.address, HOST, 0, True, (), a, b, c) is None
    assert opcall.again(entry.address, HOST, 0, True, (), a, c, None) is None


@pytest.mark.parametrize("change", [
    dict(shape=(4, 7)), dict(shape=(4, 8, 1)), dict(shape=(32,)), dict(dtype=torch.float16), dict(strides=(16, 1)),
    dict(strides=(1, 4)), dict(plain=(1, 3)), dict(plain=(2, None)), dict(plain=(1,)), dict(plain=(1, 2.0)),
    dict(grad=True), dict(device=0), dict(tensor=[1.0]), dict(plain=(1, 1 << 70)), dict(meta=True), dict(neg=True)],
    ids=str)
def test_whatever_a_check_looks_at_makes_another_call(change):
    entry = Entry(3)
    a, b = torch.zeros(4, 8, dtype=F32), torch.zeros(4, 8)
    x = torch.zeros(4, 8, dtype=F32)
    opcall.remember(b"12345678", entry.address, HOST, 0, (1, 2), x, a, b)
    assert opcall.again(entry.address, HOST, 0, True, (1, 2), x, a, b) == 0
    y = torch.zeros(change.get("shape", (4, 8)), dtype=change.get("dtype", F32))
    if "strides" in change:
        y = torch.zeros(64).as_strided((4, 8), change["strides"])
    if "grad" in change:
        y.requires_grad_()
    if "meta" in change:
        y = y.to("meta")
    if "neg" in change:
        y = torch._neg_view(y)
    if "tensor" in change:
        y = change["tensor"]
    got = opcall.again(entry.address, change.get("device", HOST), 0, True, change.get("plain", (1, 2)), y, a, b)
    assert got is None and len(entry.calls) == 1
    if "grad" in change:   # only while gradients would be recorded
        with torch.no_grad():
            assert opcall.again(entry.address, HOST, 0, True, (1, 2), y, a, b) == 0


def test_entry_points_are_told_apart():
    one, two, ts = Entry(3), Entry(3), tensors(3)
    opcall.remember(b"one.....", one.address, HOST, 0, (), *ts)
    assert opcall.again(two.address, HOST, 0, True, (), *ts) is None
    opcall.remember(b"two.....", two.address, HOST, 0, (), *ts)
    opcall.again(one.address, HOST, 0, True, (), *ts)
    opcall.again(two.address, HOST, 0, True, (), *ts)
    assert (one.calls[0][0], two.calls[0][0]) == (b"one.....", b"two.....")


def test_tensors_without_strides_are_left_to_the_checks():
    entry, (a, b, c) = Entry(3), tensors(3)
    sparse = torch.zeros(4, 8).to_sparse()
    assert not opcall.remember(b"12345678", entry.address, HOST, 0, (), sparse, b, c)
    assert opcall.again(entry.address, HOST, 0, True, (), sparse, b, c) is None


def test_arguments_of_the_wrong_kind_raise():
    entry, ts = Entry(3), tensors(3)
    for call in (lambda: opcall.again(entry.address, HOST, 0, True, ()), lambda: opcall.remember("text", entry.address, HOST, 0, (), *ts),
                 lambda: opcall.remember(b"x" * 129, entry.address, HOST, 0, (), *ts),
                 lambda: opcall.again(entry.address, "0", 0, True, (), *ts)):
        with pytest.raises(TypeError):
            call()


def test_the_store_of_calls_is_bounded():
    # more sizes than are kept: every call is either made or left to the checks
    entry, b, c = Entry(3), torch.zeros(2, 2), torch.zeros(2, 2)
    made = 0
    for rows in range(1, 3001):
        opcall.remember(rows.to_bytes(8, "little"), entry.address, HOST, 0, (), torch.zeros(rows, 1), b, c)
    for rows in range(1, 3001):
        if opcall.again(entry.address, HOST, 0, True, (), torch.zeros(rows, 1), b, c) is not None:
            assert int.from_bytes(entry.calls[-1][0], "little") == rows
            made += 1
    assert 0 < made <= 2048


def test_threads_call_side_by_side():
    # the lock is given up during a call: each call keeps its own parameters
    entries = [Entry(3) for _ in range(4)]
    ts = [[torch.zeros(2 + i, 4) for _ in range(3)] for i in range(4)]
    for i, e in enumerate(entries):
        opcall.remember(bytes([i]) * 8, e.address, HOST, 0, (), *ts[i])

    def run(i):
        for _ in range(300):
            opcall.again(entries[i].address, HOST, i, True, (), *ts[i])

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, e in enumerate(entries):
        want = (bytes([i]) * 8, tuple(t.data_ptr() for t in ts[i]), i or None)
        assert len(e.calls) == 300 and all(c == want for c in e.calls)


def test_a_workspace_is_allocated_for_the_call():
    entry, (a, b, c) = Entry(4), tensors(3)
    opcall.remember(b"12345678", entry.address, HOST, 4096, (), a, b, c, None)
    assert opcall.again(entry.address, HOST, 0, False, (), a, b, c, None) is False and not entry.calls
    assert opcall.again(entry.address, HOST, 0, True, (), a, b, c, None) == 0
    assert entry.calls[0][1][:3] == tuple(t.data_ptr() for t in (a, b, c)) and entry.calls[0][1][3] is not None
