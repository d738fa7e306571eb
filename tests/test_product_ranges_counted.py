"""Products whose sum is cut into ranges and whose tiles are more than the kernels
count are refused (CPU only: the C entry points, before they touch the device).
The kernel that takes over where the sum is whole knows no ranges."""
import ctypes
import os

import pytest

from moe_expert_ffn_persistent_amd import _lib

P = 1 << 20
ROWS, N, K = 1 << 24, 2048, 8192   # 2^20 x 2^6 tiles of 16 x 32, in 64 ranges 2^32


def _lib_or_skip():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmoe_ffn.so not built")
    return _lib.load()


def params(name):
    if name == "mx":
        return _lib.MoeMxParams(num_experts=1, rows=ROWS, n=N, k=K, ld_x=K, ld_x_scales=K // 32, ld_w=K // 2, ld_w_scales=K // 32, ld_y=N,
                                x_format=_lib.MOE_MX_E4M3, out_dtype=_lib.MOE_Y_BF16, tile=8, splits=64, workspace_bytes=1 << 62)
    if name == "fp8":
        return _lib.MoeFp8Params(num_experts=1, rows=ROWS, n=N, k=K, ld_x=K, ld_xs=K // 128, ld_w=K, ld_y=N, out_dtype=_lib.MOE_Y_BF16,
                                 tile=9, splits=64, workspace_bytes=1 << 62)
    return _lib.MoeGroupedParams(op=_lib.MOE_GROUPED_FORWARD, num_experts=1, rows=ROWS, n=N, k=K, ld_x=K, ld_w=K, ld_y=N, out_dtype=_lib.MOE_Y_BF16,
                                 tile=9, splits=64, workspace_bytes=1 << 62)


@pytest.mark.parametrize("name,entry,pointers", [("mx", "moe_mx_matmul", (None, P, P, P, P, P, P)), ("fp8", "moe_fp8_matmul_split", (None, P, P, P, P, P, P)),
                                                 ("grouped", "moe_grouped_matmul_split", (P, P, P, P, P))])
def test_ranges_of_uncounted_tiles_are_refused(name, entry, pointers):
    lib = _lib_or_skip()
    p = params(name)
    assert getattr(lib, entry)(ctypes.byref(p), *pointers, None) == _lib.MOE_ERR_UNSUPPORTED
