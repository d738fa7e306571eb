"""Microscaled (MX) quantisation and products against plain 64-bit
implementations.

Quantisation is exact: scale bytes and codes are the recipe's
(moe_inputs.quantize_mx_*), but for the sign of zeros. Products, derived: sums as
in the other operators' tests ((C + 8) 2^-23 of the magnitudes, one rounding of
2^-8 or 2^-24), and the matrix cores' dropped bits: 7 2^-13 of the magnitudes at
most, as measured for e4m3 (the products here have fewer bits)."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib
from oracle import moe_oracle as mo
from test_gpu_operators import BF, DROP, F32, F8, assert_close, gen, normal, offsets, say, up

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "e2m1"]


def recipe(x, element):
    """(values, scale bytes) of fp32 x [R, C] by the input generator's recipe, padded with zeros to whole blocks"""
    a = x.float().numpy()
    R, C = a.shape
    a = np.pad(a, ((0, 0), (0, -C % 32)))
    q, s = (mi.quantize_mx_e4m3 if element == "e4m3" else mi.quantize_mx_e2m1)(a)
    v = mo.e4m3_to_f64(q) if element == "e4m3" else mo.e2m1_to_f64(mo.unpack_e2m1(q))
    return v[:, :C], s


def values(codes, element, cols):
    """The codes' values, in 64 bits"""
    c = codes.cpu().contiguous().view(torch.uint8).numpy()
    v = mo.e4m3_to_f64(c) if element == "e4m3" else mo.e2m1_to_f64(mo.unpack_e2m1(c))
    return v[..., :cols]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 7168), (3, 31), (5, 32), (4, 33), (7, 64), (33, 100), (130, 257), (17, 1000), (2, 20011), (3000, 40), (260, 2048)])
def test_quantize_mx_is_the_recipe(R, C, element, dtype):
    x = (torch.randn(R, C, generator=gen(R + C)) * torch.exp(2 * torch.randn(R, 1, generator=gen(C)))).to(dtype)
    x[0, : C // 2] = 0
    want, ws = recipe(x, element)
    say(f"quantize_mx {R} x {C} {element} {dtype}")
    q, s = moe.quantize_mx(up(x), element)
    assert (s.cpu().numpy() == ws).all()
    assert (values(q, element, C) == want).all()
    if element == "e2m1" and C % 2:
        assert (q.cpu()[:, -1] >> 4 == 0).all()


def test_every_border_between_codes():
    # every code's value, every border between two codes (ties) and their neighbours, in blocks whose largest value fixes the scale
    for element, most, grid in (("e2m1", 6.0, np.unique(np.abs(mo.e2m1_to_f64(np.arange(8, dtype=np.uint8))))),
                                ("e4m3", 448.0, np.unique(mo.e4m3_to_f64(np.arange(127, dtype=np.uint8))))):
        mid = (grid[1:] + grid[:-1]) / 2
        pts = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)), np.nextafter(mid.astype(np.float32), np.float32(0)),
                              [most * 1.1]])
        pts = np.concatenate([pts, -pts]).astype(np.float32)
        rows = []
        for e in (-126, -30, -1, 0, 5, 100):
            for i in range(0, len(pts), 31):
                block = np.zeros(32, np.float32)
                block[0] = most
                part = pts[i:i + 31]
                block[1:1 + len(part)] = part
                with np.errstate(over="ignore"):
                    rows.append(block * np.float32(2.0 ** min(e, 100)) if e > -126 else block * np.float32(2.0 ** -60) * np.float32(2.0 ** -60))
        x = torch.from_numpy(np.stack(rows).astype(np.float32))
        want, ws = recipe(x, element)
        q, s = moe.quantize_mx(up(x), element)
        assert (s.cpu().numpy() == ws).all()
        assert (values(q, element, 32) == want).all(), element


@pytest.mark.parametrize("element,emax", [("e4m3", 8), ("e2m1", 2)])
def test_scales_at_the_ends_of_fp32(element, emax):
    x = torch.zeros(8, 32)
    x[0, 3], x[1, 3], x[2, 3] = 2.0 ** -149, 2.0 ** -126, 2.0 ** (-127 + emax)
    x[3, 3], x[4, 3], x[5, 3] = 3.4028234663852886e38, float("inf"), float("nan")
    x[6] = -0.0
    x[7, 3], x[7, 4] = float("-inf"), 1.0
    q, s = moe.quantize_mx(up(x), element)
    assert s.view(-1).tolist() == [0, 0, 0, 254 - emax, 255, 255, 127, 255]
    v = values(q, element, 32)
    step = 2.0 ** -9 if element == "e4m3" else 0.5
    want = [np.round(2.0 ** (-149 + 127) / step) * step, np.round(2.0 / step) * step, 2.0 ** emax, 448.0 if element == "e4m3" else 6.0]
    assert [float(v[i, 3]) for i in range(4)] == want
    assert (np.isnan(v[4:6]).all() and np.isnan(v[7]).all()) if element == "e4m3" else (v[4:] == 0).all()
    assert (v[6] == 0).all()


@pytest.mark.parametrize("element", FORMATS)
def test_quantize_mx_strides_batches_and_experts(element):
    x = normal(gen(4), 3, 21, 104)
    want = [moe.quantize_mx(up(x[i]), element) for i in range(3)]
    q, s = moe.quantize_mx(up(x), element)
    for i in range(3):
        assert torch.equal(q[i].view(torch.uint8), want[i][0].view(torch.uint8)) and torch.equal(s[i], want[i][1])
    for lead, pad in ((1, 3), (4, 4), (8, 8), (2, 0)):
        buf = torch.zeros(21, 104 + pad + lead, dtype=BF, device="cuda")
        buf[:, lead:lead + 104] = up(x[0])
        bytes_ = want[0][0].shape[1]
        codes = torch.full((21, bytes_ + pad + lead), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.full((21, 4 + pad + lead), 0x55, dtype=torch.uint8, device="cuda")
        c, sc = codes[:, lead:lead + bytes_], scales[:, lead:lead + 4]
        moe.quantize_mx(buf[:, lead:lead + 104], element, out=c, scales=sc)
        assert torch.equal(c, want[0][0].view(torch.uint8)) and torch.equal(sc, want[0][1])
        assert (codes[:, :lead] == 0x55).all() and (codes[:, lead + bytes_:] == 0x55).all() and (scales[:, lead + 4:] == 0x55).all()
    off = offsets([4, 0, 7], first=3)
    codes, scales = torch.full_like(want[0][0].view(torch.uint8), 0x55), torch.full_like(want[0][1], 0x55)
    moe.quantize_mx(up(x[0]), element, row_offset=up(off), out=codes, scales=scales)
    assert torch.equal(codes[3:14], want[0][0].view(torch.uint8)[3:14]) and torch.equal(scales[3:14], want[0][1][3:14])
    for t in (codes, scales):
        assert (t[:3] == 0x55).all() and (t[14:] == 0x55).all()


def test_quantize_mx_takes_the_formats_own_types():
    x = up(normal(gen(6), 5, 64))
    q, s = moe.quantize_mx(x, "e2m1")
    if hasattr(torch, "float4_e2m1fn_x2"):
        q2 = torch.zeros(5, 32, dtype=torch.uint8, device="cuda").view(torch.float4_e2m1fn_x2)
        s2 = torch.zeros(5, 2, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        moe.quantize_mx(x, "e2m1", out=q2, scales=s2)
        assert torch.equal(q2.view(torch.uint8), q) and torch.equal(s2.view(torch.uint8), s)
        w, ws = moe.quantize_mx(up(normal(gen(7), 24, 64)), "e2m1")
        assert torch.equal(moe.mx_matmul(q2, s2, w.view(torch.float4_e2m1fn_x2), ws.view(torch.float8_e8m0fnu)), moe.mx_matmul(q, s, w, ws))


# ---- products -----------------------------------------------------------------------

def operand(g, element, *shape, pad=0, lead=0):
    """Codes and scale bytes of a bell over the formats' range on the device, rows `pad` + what a whole 16 (4) bytes takes apart,
    `lead` bytes into their buffers; and their values in 64 bits."""
    K = shape[-1]
    x = torch.randn(int(np.prod(shape[:-1])), K, generator=g) * torch.exp(torch.randn(int(np.prod(shape[:-1])), 1, generator=g))
    v, s = recipe(x, element)
    q = (mi.e4m3_encode(v.astype(np.float32)) if element == "e4m3" else None)
    if q is None:
        c = mi.e2m1_encode(np.pad(v, ((0, 0), (0, K % 2))))
        q = (c[:, 0::2] | (c[:, 1::2] << np.uint8(4))).astype(np.uint8)
    full = torch.from_numpy(mo.e8m0_to_f64(s)).repeat_interleave(32, dim=1)[:, :K] * torch.from_numpy(np.ascontiguousarray(v))

    def place(a, whole):
        wide = -(-a.shape[-1] // whole) * whole + pad
        rows = [*shape[:-1]]
        if len(rows) == 2:
            rows[1] += 1 if pad else 0
        buf = torch.full((int(np.prod(rows)) * wide + lead,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN scales and codes behind the rows
        t = buf[lead:].view(*rows, wide)[..., :a.shape[-1]]
        t = t[:, :shape[1]] if len(rows) == 2 else t
        t.copy_(torch.from_numpy(np.ascontiguousarray(a)).view(*shape[:-1], -1))
        return t

    codes = place(q, 16)
    return codes.view(F8) if element == "e4m3" else codes, place(s, 4), full.view(shape)


def reference(x, w, off):
    out = torch.zeros(x.shape[0], w.shape[-2], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(len(off) - 1):
        r, we = slice(int(off[e]), int(off[e + 1])), w[e] if w.dim() == 3 else w
        out[r], mag[r] = x[r] @ we.t(), x[r].abs() @ we.abs().t()
    return out, mag


def run_mx(counts, R, K, n, element, out_dtype, pad=0, lead=0, behind=0, expected_rows=None, tile=0, splits=0, first=0):
    g = gen(R + K + n)
    rows, L = first + R + behind, 0 if counts is None else len(counts)
    off = offsets([rows] if counts is None else counts, first)
    x, xs, xv = operand(g, element, rows, K, pad=pad, lead=lead)
    w, ws, wv = operand(g, "e2m1", *((L,) if L else ()), n, K, pad=pad, lead=lead)
    ref, mag = reference(xv, wv, off)
    if counts is not None:   # rows that no expert owns
        xs[:first], xs[first + R:] = 255, 255
    wide = -(-n // 8) * 8 + pad
    buf = torch.full((rows * wide + lead,), 7.0, dtype=out_dtype, device="cuda")
    y = buf[lead:].view(rows, wide)[:, :n]
    say(f"mx counts={counts} R={R} K={K} n={n} {element} {out_dtype} pad={pad} lead={lead} tile={tile} splits={splits}")
    moe.mx_matmul(x, xs, w, ws, row_offset=None if counts is None else up(off), out=y, expected_rows=expected_rows, tile=tile, splits=splits)
    got = buf.cpu()[lead:].view(rows, wide)
    own = slice(first, first + R) if counts is not None else slice(None)
    assert_close(got[own, :n], ref[own], out_dtype, mag[own], K, f"mx {counts} {K} {n}", DROP)
    if counts is not None:
        assert (got[:first] == 7).all() and (got[first + R:] == 7).all(), "a row that no expert owns was written"
    assert (got[:, n:] == 7).all() and (buf[:lead] == 7).all(), "written outside the rows"


NOT_OF = {"e4m3": (4,), "e2m1": (6, 10)}   # tiles of the other type of rows

SHAPES = [
    (None, 1, 128, 8), (None, 1, 7168, 264), (None, 5, 2, 1), (None, 17, 32, 16), (None, 130, 1000, 72), (None, 300, 512, 264), (None, 33, 96, 19),
    (None, 64, 34, 136), (None, 257, 290, 520), (None, 3, 62, 37), (None, 12, 4100, 40),
    ([0, 1, 0, 5], 6, 64, 64), ([33, 0, 64, 129, 1], 227, 136, 72), ([7, 250, 0, 0, 260], 517, 1000, 200), ([0, 0, 0], 0, 128, 128),
    ([16, 17, 15, 31, 32, 33], 144, 256, 128), ([5, 70, 2], 77, 38, 19),
]


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("counts,R,K,n", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_mx_matches_64_bits(counts, R, K, n, element, out_dtype):
    run_mx(counts, R, K, n, element, out_dtype, behind=3 if counts else 0, first=2 if counts else 0)


@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("pad,lead", [(16, 0), (16, 16), (3, 0), (0, 1), (4, 4), (5, 3), (48, 16)])
@pytest.mark.parametrize("counts,R,K,n", [([40, 0, 9, 130], 179, 204, 136), (None, 70, 330, 40)], ids=["grouped", "dense"])
def test_mx_strides_and_alignment(counts, R, K, n, pad, lead, element):
    run_mx(counts, R, K, n, element, BF, pad=pad, lead=lead, behind=9 if counts else 0)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("pad,lead", [(3, 0), (5, 3)])
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("counts,R,K,n", [([300, 0, 249, 150, 1], 700, 206, 2601), (None, 700, 384, 2600), (None, 513, 34, 3001)], ids=["grouped", "dense", "short"])
def test_many_rows_of_any_alignment(counts, R, K, n, pad, lead, element, out_dtype):
    run_mx(counts, R, K, n, element, out_dtype, pad=pad, lead=lead, behind=3 if counts else 0)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", range(1, 11))
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("counts,R,K,n", [([0, 33, 290, 1], 324, 272, 328), (None, 300, 64, 8), ([3, 0, 200], 203, 34, 65),
                                          ([64, 128], 192, 512, 256), (None, 1, 8338, 136), (None, 257, 1056, 523), ([191, 129], 320, 2112, 136)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_mx_every_tile(counts, R, K, n, element, tile, out_dtype):
    if tile in NOT_OF[element]:
        with pytest.raises(_lib.MoeError) as err:
            run_mx(counts, R, K, n, element, out_dtype, tile=tile)
        assert err.value.status == _lib.MOE_ERR_UNSUPPORTED
        return
    run_mx(counts, R, K, n, element, out_dtype, pad=16, tile=tile, behind=3 if counts else 0)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", range(1, 11))
@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("splits", [2, 3, 64])
def test_mx_sums_in_ranges(splits, element, tile, out_dtype):
    if tile not in NOT_OF[element]:
        run_mx([0, 40, 3, 70], 113, 1380, 136, element, out_dtype, tile=tile, splits=splits, behind=5, first=1)


@pytest.mark.parametrize("element", FORMATS)
def test_mx_automatic_ranges_and_refusals(element):
    # few tiles and a long sum, whole and in ranges; ranges need whole 16 bytes of out
    for n in (64, 61):
        run_mx(None, 3, 16384, n, element, BF)
        run_mx([2, 0, 1], 3, 8224, n, element, F32)
    with pytest.raises(_lib.MoeError) as err:
        run_mx(None, 3, 512, 61, element, BF, splits=2)
    assert err.value.status == _lib.MOE_ERR_UNSUPPORTED
    for kw in (dict(tile=11), dict(tile=1, pad=1)):
        with pytest.raises(_lib.MoeError) as err:
            run_mx(None, 3, 512, 64, element, BF, **kw)
        assert err.value.status == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("element", FORMATS)
def test_mx_result_does_not_depend_on_timing(element):
    g = gen(9)
    x, xs, _ = operand(g, element, 40, 8192)
    w, ws, _ = operand(g, "e2m1", 136, 8192)
    want = moe.mx_matmul(x, xs, w, ws, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(moe.mx_matmul(x, xs, w, ws, out_dtype=F32), want)


@pytest.mark.parametrize("pad", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("K", [1, 3, 33, 127, 129, 1001])
def test_odd_sums_of_e4m3_rows(K, pad):
    # the last byte of a weight row holds one code; what stands beside it is not looked at
    g = gen(K)
    x, xs, xv = operand(g, "e4m3", 20, K, pad=pad)
    w, ws, wv = operand(g, "e2m1", 24, K, pad=pad)
    w[:, -1] |= 0x70
    ref, mag = reference(xv, wv, [0, 20])
    got = moe.mx_matmul(x, xs, w, ws, out_dtype=F32)
    assert_close(got, ref, F32, mag, K, f"odd {K}", DROP)


@pytest.mark.parametrize("element", FORMATS)
@pytest.mark.parametrize("R,K,n", [(40, 1024, 72), (3, 416, 264), (300, 768, 520)])
@pytest.mark.parametrize("tile,pad", [(t, 0) for t in range(11)] + [(0, 1)])
def test_exact_products(R, K, n, element, pad, tile):
    tile = 0 if tile in NOT_OF[element] else tile
    # small whole numbers times powers of two: every sum is exact in fp32 and nothing lies 2^13 below another product,
    # so a wrong element, scale or block shows as a wrong bit
    g = gen(3)
    table = np.array([0, 1, 2, 4], dtype=np.float64)
    xi, wi = torch.randint(-3, 4, (R, K), generator=g), torch.randint(-3, 4, (n, K), generator=g)
    xv = torch.from_numpy(table)[xi.abs()] * torch.sign(xi)
    wv = torch.from_numpy(table)[wi.abs()] * torch.sign(wi)
    xs, ws = (torch.randint(126, 129, (r, K // 32), generator=g).to(torch.uint8) for r in (R, n))

    def place(a, whole):
        buf = torch.zeros(a.shape[0], -(-a.shape[1] // whole) * whole + pad, dtype=torch.uint8, device="cuda")
        buf[:, :a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return buf[:, :a.shape[1]]

    def pairs(v):
        c = mi.e2m1_encode(v.numpy())
        return (c[:, 0::2] | (c[:, 1::2] << np.uint8(4))).astype(np.uint8)

    x = place(mi.e4m3_encode(xv.float().numpy()), 16).view(F8) if element == "e4m3" else place(pairs(xv), 16)
    spread = lambda s: torch.pow(2.0, s.double() - 127).repeat_interleave(32, dim=1)   # noqa: E731
    ref = (xv * spread(xs)) @ (wv * spread(ws)).t()
    got = moe.mx_matmul(x, place(xs.numpy(), 4), place(pairs(wv), 16), place(ws.numpy(), 4), out_dtype=F32, tile=tile)
    assert torch.equal(got.cpu().double(), ref)


@pytest.mark.parametrize("pad", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("element", FORMATS)
def test_scales_of_both_ends_and_nan(element, pad):
    g = gen(12)
    R, K, n = 20, 256, 40
    x, xs, xv = operand(g, element, R, K, pad=pad)
    w, ws, wv = operand(g, "e2m1", n, K, pad=pad)
    # scales far from 1 that cancel: each side's factor is exact
    xs += 100 - 80
    ws -= 100 - 80
    ref, mag = reference(xv, wv, [0, R])
    got = moe.mx_matmul(x, xs, w, ws, out_dtype=F32)
    assert_close(got, ref, F32, mag, K, "shifted scales", DROP)
    xs[3, 5] = 255   # NaN: one row; one feature
    ws[7, 0] = 255
    bad = moe.mx_matmul(x, xs, w, ws, out_dtype=F32)
    assert torch.isnan(bad[3]).all() and torch.isnan(bad[:, 7]).all()
    keep = [i for i in range(R) if i != 3]
    cols = [i for i in range(n) if i != 7]
    assert torch.equal(bad[keep][:, cols], got[keep][:, cols])


def test_offsets_past_the_rows_are_clamped():
    g = gen(11)
    x, xs, xv = operand(g, "e4m3", 50, 128)
    w, ws, wv = operand(g, "e2m1", 4, 64, 128)
    bad = torch.tensor([-7, 20, 44, 1000, 2 ** 31 - 1], dtype=torch.int32)
    ref, mag = reference(xv, wv, [0, 20, 44, 50, 50])
    got = moe.mx_matmul(x, xs, w, ws, row_offset=up(bad))
    assert_close(got, ref, BF, mag, 128, "clamped", DROP)


def test_no_rows():
    g = gen(1)
    w, ws, _ = operand(g, "e2m1", 16, 64)
    x, xs = torch.zeros(0, 64, device="cuda").to(F8), torch.zeros(0, 2, dtype=torch.uint8, device="cuda")
    assert moe.mx_matmul(x, xs, w, ws).shape == (0, 16)


def test_most_experts():
    counts = torch.randint(0, 5, (256,), generator=gen(5)).tolist()
    run_mx(counts, sum(counts), 64, 72, "e4m3", BF)
