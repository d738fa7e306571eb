"""The operators' call path when memory runs out (a child process with a limit on
its address space): a call is not kept, and the process goes on."""
import os
import subprocess
import sys

import pytest

from moe_expert_ffn_persistent_amd import build

CHILD = r"""
import ctypes, resource, sys
import torch
from moe_expert_ffn_persistent_amd import _lib
opcall = _lib.load_opcall()
fn = ctypes.CFUNCTYPE(ctypes.c_int32, *[ctypes.c_void_p] * 5)(lambda *a: 0)
entry = ctypes.cast(fn, ctypes.c_void_p).value
ts = [torch.zeros(2, 2) for _ in range(3)]
plain = (1,) * (8 << 20)                                       # a key of 128 MiB
assert opcall.again(entry, -1, 0, True, plain, *ts) is None    # its storage stays
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
limits = resource.getrlimit(resource.RLIMIT_AS)
resource.setrlimit(resource.RLIMIT_AS, (used + (64 << 20), limits[1]))
assert not opcall.remember(b"12345678", entry, -1, 0, plain, *ts)   # would keep a copy of the key
print("not kept", flush=True)
resource.setrlimit(resource.RLIMIT_AS, limits)
assert opcall.again(entry, -1, 0, True, plain, *ts) is None    # nothing was kept
assert opcall.remember(b"12345678", entry, -1, 0, (1,), *ts) and opcall.again(entry, -1, 0, True, (1,), *ts) == 0
print("works", flush=True)
"""


@pytest.mark.skipif(not os.path.exists(build.OPCALL), reason="_opcall.so not built")
def test_running_out_of_memory_ends_no_process():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=100, cwd=build.ROOT)
    assert r.returncode == 0 and r.stdout.split() == ["not", "kept", "works"], (r.returncode, r.stdout, r.stderr[-500:])
