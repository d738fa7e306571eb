"""Products of MX operands whose scale bytes are at both ends of E8M0 (0 is 2^-127,
254 is 2^127), against 64 bits.

Values are whole numbers of -3 .. 3, so products are -9 .. 9 and sums of up to 1024
of them whole numbers below 2^14: where all blocks have the same product of scales,
2^d, every partial sum is a whole number times 2^d, exact in fp32 for d of -126 .. 113.
Below that a partial sum is rounded to a multiple of 2^-149 (by one of them at most,
rounded or cut off), one for each product at most: K 2^-149 in all. Above, a partial
sum past fp32's largest is infinite, and so not finite is the whole."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import moe_expert_ffn_persistent_amd as moe
from test_gpu_mx import FORMATS, NOT_OF
from test_gpu_operators import BF, F32, F8, gen, say

pytestmark = pytest.mark.gpu

ENDS = [0, 1, 2, 64, 126, 127, 128, 253, 254]
KERNELS = [(t, 0) for t in range(11)] + [(0, 1)]   # tile (0: chosen), bytes of padding (1: the kernel of any alignment)


def place(a, whole, pad):
    a = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    buf = torch.zeros(a.shape[0], -(-a.shape[1] // whole) * whole + pad, dtype=torch.uint8, device="cuda")
    buf[:, :a.shape[1]] = a.cuda()
    return buf[:, :a.shape[1]]


def codes(v, element, pad):
    if element == "e4m3":
        return place(mi.e4m3_encode(v.float().numpy()), 16, pad).view(F8)
    c = mi.e2m1_encode(v.numpy())
    return place((c[:, 0::2] | (c[:, 1::2] << np.uint8(4))).astype(np.uint8), 16, pad)


def product(xv, xs, wv, ws, element, tile, pad, out_dtype=F32):
    tile = 0 if tile in NOT_OF[element] else tile
    return moe.mx_matmul(codes(xv, element, pad), place(xs, 4, pad), codes(wv, "e2m1", pad), place(ws, 4, pad), out_dtype=out_dtype, tile=tile).cpu()


def whole(g, *shape):
    return torch.randint(-3, 4, shape, generator=g).double()


def bytes_of(rows, blocks, value):
    return torch.full((rows, blocks), value, dtype=torch.uint8)


@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("R,K,n", [(40, 1024, 72), (3, 416, 264), (300, 768, 520)])
@pytest.mark.parametrize("tile,pad", KERNELS)
def test_scales_that_cancel(R, K, n, element, tile, pad):
    g = gen(R)
    xv, wv, b = whole(g, R, K), whole(g, n, K), torch.tensor(ENDS)[torch.randint(0, len(ENDS), (K // 32,), generator=g)].to(torch.uint8)
    say(f"scales that cancel {R} {K} {n} {element} tile={tile} pad={pad}")
    got = product(xv, b.expand(R, -1), wv, (254 - b).expand(n, -1), element, tile, pad)
    assert torch.equal(got.double(), xv @ wv.t())


@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("tile,pad", [(0, 0), (1, 0), (9, 0), (0, 1)])
def test_one_product_of_scales(element, tile, pad):
    R, K, n, g = 33, 512, 72, gen(5)
    xv, wv = whole(g, R, K), whole(g, n, K)
    ref = xv @ wv.t()
    for a, b in ((0, 128), (128, 0), (1, 127), (127, 1), (0, 254), (254, 0), (254, 113), (113, 254), (183, 184), (0, 200), (254, 1), (1, 254)):
        say(f"scales {a} and {b}, {element} tile={tile} pad={pad}")
        got = product(xv, bytes_of(R, K // 32, a), wv, bytes_of(n, K // 32, b), element, tile, pad)
        assert torch.equal(got.double(), ref * 2.0 ** (a + b - 254)), (a, b)
    for a, b in ((0, 100), (100, 0), (40, 64), (60, 60)):
        got = product(xv, bytes_of(R, K // 32, a), wv, bytes_of(n, K // 32, b), element, tile, pad)
        assert ((got.double() - ref * 2.0 ** (a + b - 254)).abs() <= K * 2.0 ** -149).all(), (a, b)
    for a, b in ((0, 0), (0, 20), (20, 0), (1, 1)):   # nothing is left of them
        assert (product(xv, bytes_of(R, K // 32, a), wv, bytes_of(n, K // 32, b), element, tile, pad) == 0).all(), (a, b)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("tile,pad", [(0, 0), (1, 0), (9, 0), (0, 1)])
def test_sums_past_fp32(element, tile, pad, out_dtype):
    R, K, n, g = 33, 512, 72, gen(6)
    xv, wv = torch.randint(1, 4, (R, K), generator=g).double(), torch.randint(1, 4, (n, K), generator=g).double()
    xv[1::2] *= -1
    for a, b in ((254, 254), (254, 128), (200, 182)):
        got = product(xv, bytes_of(R, K // 32, a), wv, bytes_of(n, K // 32, b), element, tile, pad, out_dtype)
        assert torch.isposinf(got[0::2]).all() and torch.isneginf(got[1::2]).all(), (a, b)
    xv[:, K // 2:] = -xv[:, :K // 2]   # the whole sum is none, but not its parts
    wv[:, K // 2:] = wv[:, :K // 2]
    got = product(xv, bytes_of(R, K // 32, 254), wv, bytes_of(n, K // 32, 254), element, tile, pad, out_dtype)
    assert not torch.isfinite(got).any()
