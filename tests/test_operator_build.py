"""The compiled call path is a convenience: without a host compiler, or Python's
or torch's headers, the library is built and every operator works."""
import contextlib
import os
import subprocess
import types

import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib, build, ops


def missing():
    raise RuntimeError("the operators' call path is missing")


def test_the_library_is_built_without_the_call_path(monkeypatch, tmp_path, capsys):
    lib, opcall = tmp_path / "libmoe_ffn.so", tmp_path / "_opcall.so"
    opcall.write_text("of an earlier build")

    def run(cmd, **kw):
        if cmd[0] == "no-such-compiler":
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: no such file")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("linked")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "OPCALL", str(opcall))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert build.build(verbose=False) == str(lib)
    assert lib.read_text() == "linked"
    assert not opcall.exists()   # one of an earlier build may not fit this one
    assert "Python.h" in capsys.readouterr().err


def without_call_path(monkeypatch):
    monkeypatch.setattr(ops, "_ENTRY", {})
    monkeypatch.setattr(ops, "_again", None)
    monkeypatch.setattr(ops, "_remember", None)
    monkeypatch.setattr(ops, "_no_call_path", False)
    monkeypatch.setattr(_lib, "load_opcall", missing)


def test_operators_check_every_call_without_the_call_path(monkeypatch):
    made = []

    def entry(params, *ptrs):
        made.append(ptrs)
        return _lib.MOE_OK

    without_call_path(monkeypatch)
    monkeypatch.setattr(_lib, "load", lambda: types.SimpleNamespace(moe_swiglu=entry))
    monkeypatch.setattr(ops, "_need_device", lambda device: None)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 77)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    a, out = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="call path") as warned:
        for i in range(3):
            assert moe.swiglu(a, out=out) is out and out._version == i + 1
    assert len(warned) == 1
    assert made == [(a.data_ptr(), None, None, out.data_ptr(), None, 77)] * 3
    with pytest.raises(ValueError):
        moe.swiglu(a, out=out[:3])


@pytest.mark.gpu
def test_operators_give_the_same_without_the_call_path(monkeypatch):
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(40, 2048, generator=g).bfloat16().cuda(), torch.randn(2, 64, 2048, generator=g).bfloat16().cuda()
    off = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    run = lambda: [moe.grouped_matmul(x, w, off, splits=s) for s in (0, 2)] + list(moe.quantize_fp8(x))   # noqa: E731
    run()
    want = [t.cpu().view(torch.uint8) for t in run()]
    without_call_path(monkeypatch)
    with pytest.warns(RuntimeWarning, match="call path"):
        got = [t.cpu().view(torch.uint8) for t in run()]
    assert os.path.exists(_lib.LIB_PATH) and not ops._ENTRY
    assert all(torch.equal(a, b) for a, b in zip(got, want))
