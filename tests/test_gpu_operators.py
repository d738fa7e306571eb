"""The operators around the expert FFN against plain 64-bit implementations.

Bars, derived: a result rounded to bf16 is off by at most 2^-8 of its value
(half a step). Behind that stands the fp32 arithmetic: a sum of C products of
exact operands, each addition off by at most one unit in the last place of the
running sum (2^-23 of it, which covers rounding and truncation), is off by at
most (C + 8) 2^-23 of the sum of the products' magnitudes, in any order; the 8
covers the joining of partial sums. Row copies and quantisation are exact."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ULP = 2.0 ** -23
DROP = 7 * 2.0 ** -13
FWD, DGRAD, WGRAD = _lib.MOE_GROUPED_FORWARD, _lib.MOE_GROUPED_DGRAD, _lib.MOE_GROUPED_WGRAD


def say(*a):
    print("[ops]", *a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def up(t):
    return None if t is None else t.cuda()


def offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32)


def strided(t, pad, lead=0, fill=float("nan")):
    """t on the device inside a larger buffer: rows `pad` elements apart more,
    the first element `lead` elements into it; the padding holds `fill`."""
    shape = list(t.shape)
    shape[-1] += pad
    if t.dim() == 3:
        shape[1] += 1 if pad else 0
    n = int(np.prod(shape))
    buf = torch.full((n + lead,), fill, dtype=torch.float32).to(t.dtype).cuda()
    v = buf[lead:].view(shape)[tuple(slice(0, s) for s in t.shape)]
    v.copy_(t)
    return v


def assert_close(got, ref, dtype, mag, terms, what, drop=0.0):
    got = got.double().cpu()
    tol = HALF[dtype] * (1 + 2.0 ** -8) * (ref.abs() + drop * mag) + ((terms + 8) * ULP + drop) * mag + 1e-37
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / tol).max():.3g} of the bar"


def reference(op, x, w, y, off):
    """(result, sum of magnitudes, terms) in 64 bits; rows outside: untouched."""
    x, w, y = (None if t is None else t.double() for t in (x, w, y))
    if op == FWD:
        out = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    elif op == DGRAD:
        out = torch.zeros(y.shape[0], w.shape[2], dtype=torch.float64)
    else:
        out = torch.zeros(len(off) - 1, y.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    terms = 0
    for e in range(len(off) - 1):
        r = slice(int(off[e]), int(off[e + 1]))
        if op == FWD:
            out[r], mag[r], terms = x[r] @ w[e].t(), x[r].abs() @ w[e].abs().t(), x.shape[1]
        elif op == DGRAD:
            out[r], mag[r], terms = y[r] @ w[e], y[r].abs() @ w[e].abs(), y.shape[1]
        else:
            out[e], mag[e] = y[r].t() @ x[r], y[r].abs().t() @ x[r].abs()
            terms = max(terms, r.stop - r.start)
    return out, mag, terms


def call(op, x, w, y, off, **kw):
    if op == FWD:
        return moe.grouped_matmul(x, w, off, out=y, **kw)
    if op == DGRAD:
        return moe.grouped_matmul_dgrad(y, w, off, out=x, **kw)
    return moe.grouped_matmul_wgrad(y, x, off, out=w, **kw)


def run_grouped(op, counts, k, n, out_dtype, seed, first=0, behind=0, pad=0, lead=0, expected_rows=None, tile=0, splits=0):
    """One grouped product with NaN in every row that no expert owns and a
    sentinel in the output, checked against 64 bits."""
    g = gen(seed)
    L, R = len(counts), first + sum(counts) + behind
    off = offsets(counts, first)
    lo, hi = first, first + sum(counts)
    x, w, y = normal(g, R, k), normal(g, L, n, k, std=0.05), normal(g, R, n, std=0.5)
    ref, mag, terms = reference(op, x, w, y, off)
    for t in (x, y):
        t[:lo], t[hi:] = float("nan"), float("nan")
    if op == FWD:
        y = torch.full((R, n), 7.0, dtype=out_dtype)
    elif op == DGRAD:
        x = torch.full((R, k), 7.0, dtype=out_dtype)
    else:
        w = torch.full((L, n, k), 7.0, dtype=out_dtype)
    dx, dw, dy = strided(x, pad, lead), strided(w, pad, lead), strided(y, pad, lead)
    say(f"op={op} counts={counts if L < 9 else L} k={k} n={n} out={out_dtype} first={first} behind={behind} pad={pad} lead={lead}")
    got = call(op, dx, dw, dy, up(off), expected_rows=expected_rows, tile=tile, splits=splits)
    torch.cuda.synchronize()
    if op == WGRAD:
        assert_close(got, ref, out_dtype, mag, terms, f"wgrad {counts}")
    else:
        rows = slice(lo, hi)
        assert_close(got[rows], ref[rows], out_dtype, mag[rows], terms, f"op {op} {counts}")
        assert (got[:lo] == 7.0).all() and (got[hi:] == 7.0).all(), "a row that no expert owns was written"
    if pad:   # nothing was written between the rows
        whole = torch.as_strided(got, got.shape[:-1] + (got.shape[-1] + pad,), got.stride())[..., got.shape[-1]:]
        inner = whole if got.dim() == 2 else whole[:, :-1]
        assert torch.isnan(inner[:-1].float()).all(), "written behind a row's end"
    return got


SHAPES = [
    ([0, 1, 0, 5], 64, 64),
    ([33, 0, 64, 129, 1], 136, 72),
    ([7, 250, 0, 0, 260], 1000, 520),
    ([300], 384, 640),
    ([1, 1, 1, 1], 2048, 256),
    ([700, 513], 512, 768),
    ([16, 17, 15, 31, 32, 33], 256, 128),
    ([0, 0, 0], 128, 128),
    ([5, 70, 2], 37, 19),
    ([3, 0, 66], 1, 1),
    ([129, 2], 130, 257),
]


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[1]}x{s[2]}")
def test_grouped_matches_64_bits(shape, op, out_dtype):
    counts, k, n = shape
    run_grouped(op, counts, k, n, out_dtype, seed=k + n + op, behind=3)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("pad,lead", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3), (24, 16)])
def test_grouped_strides_and_alignment(op, pad, lead):
    run_grouped(op, [40, 0, 9, 130], 200, 136, BF, seed=pad * 31 + lead, first=5, behind=70, pad=pad, lead=lead)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("expected", [1, 40, 100, 400, 5000])
def test_grouped_tile_choice_changes_no_result(op, expected):
    # expected_rows chooses the kernel; any choice is right for any counts
    run_grouped(op, [0, 33, 290, 5], 264, 328, BF, seed=17, expected_rows=expected, behind=1)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", range(1, 10))
@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts,k,n", [([0, 33, 290, 1], 264, 328), ([70, 257], 64, 8), ([3, 0, 200], 8, 64), ([64, 128], 512, 256),
                                        ([191, 129], 1032, 136), ([1, 700], 2056, 72)])
def test_grouped_every_tile(counts, k, n, op, tile, out_dtype):
    if op == WGRAD and tile in (2, 6, 7, 8, 9):   # not tiles of this product
        with pytest.raises(_lib.MoeError) as err:
            run_grouped(op, counts, k, n, out_dtype, seed=1, tile=tile)
        assert err.value.status == _lib.MOE_ERR_UNSUPPORTED
        return
    run_grouped(op, counts, k, n, out_dtype, seed=k + n, first=2, behind=4, pad=8, tile=tile)


@pytest.mark.parametrize("pad", [0, 1], ids=["aligned", "odd"])
@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
def test_grouped_without_any_rows(op, pad):
    # no expert has rows in buffers that hold some: rows stay, weight gradients are zeros
    run_grouped(op, [0, 0, 0], 264 + pad, 328, BF, seed=7, first=3, behind=40)
    run_grouped(op, [0], 264 + pad, 328, F32, seed=8)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
def test_grouped_most_experts(op):
    counts = torch.randint(0, 5, (256,), generator=gen(5)).tolist()
    run_grouped(op, counts, 64, 72, BF, seed=3)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
def test_grouped_offsets_past_the_rows_are_clamped(op):
    # never a read or write outside the buffers: offsets past the rows count as the rows
    g = gen(11)
    L, R, k, n = 4, 50, 128, 64
    x, w, y = normal(g, R, k), normal(g, L, n, k, std=0.05), normal(g, R, n)
    bad = torch.tensor([-7, 20, 44, 1000, 2 ** 31 - 1], dtype=torch.int32)
    good = torch.tensor([0, 20, 44, 50, 50], dtype=torch.int32)
    ref, mag, terms = reference(op, x, w, y, good)
    got = call(op, *(up(t) for t in (x, w, y)), up(bad))
    torch.cuda.synchronize()
    assert_close(got, ref, BF, mag, terms, "clamped")


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("k,n", [(264, 136), (33, 7)])
def test_wgrad_accumulates(out_dtype, k, n):
    g = gen(23)
    counts = [0, 70, 3]
    off = offsets(counts)
    x, y = normal(g, 73, k), normal(g, 73, n)
    old = normal(g, 3, n, k, dtype=out_dtype)
    ref, mag, terms = reference(WGRAD, x, None, y, off)
    got = moe.grouped_matmul_wgrad(up(y), up(x), up(off), out=up(old), accumulate=True)
    torch.cuda.synchronize()
    ref = ref + old.double()
    assert_close(got, ref, out_dtype, mag + old.double().abs(), terms, "accumulate")
    assert torch.equal(got[0].cpu(), old[0])   # an expert without rows keeps its sum
    # no rows at all: zeros, or the old sum
    none = torch.zeros(4, dtype=torch.int32).cuda()
    z = moe.grouped_matmul_wgrad(up(y[:0]), up(x[:0]), none, out_dtype=out_dtype)
    assert (z == 0).all()
    assert torch.equal(moe.grouped_matmul_wgrad(up(y[:0]), up(x[:0]), none, out=up(old), accumulate=True).cpu(), old)


@pytest.mark.parametrize("op", [FWD, DGRAD, WGRAD], ids=["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_grouped_keeps_other_experts_clean(op, value):
    # an infinity or NaN in one expert's rows reaches that expert's results only
    g = gen(31)
    counts, k, n = [3, 40, 5], 72, 80
    off = offsets(counts)
    x, w, y = normal(g, 48, k), normal(g, 3, n, k, std=0.05), normal(g, 48, n)
    x[3:43], y[3:43] = value, value
    got = call(op, *(up(t) for t in (x, w, y)), up(off)).cpu()
    keep = [0, 2] if op == WGRAD else list(range(3)) + list(range(43, 48))
    ref, mag, terms = reference(op, x, w, y, off)
    assert_close(got[keep], ref[keep], BF, mag[keep], terms, "clean")


@pytest.mark.parametrize("tile", [0, 1, 6])
def test_grouped_subnormals_and_overflow(tile):
    # subnormal bf16 operands count in full, and a sum past bf16's largest value
    # is an infinity of its sign
    x = torch.full((4, 64), 2.0 ** -130, dtype=BF)
    w = torch.full((1, 8, 64), 2.0 ** 100, dtype=BF)
    x[1], x[2] = 2.0 ** 60, -(2.0 ** 60)
    got = moe.grouped_matmul(up(x), up(w), up(offsets([4])), tile=tile).cpu()
    assert (got[0] == 2.0 ** -24).all() and (got[1] == float("inf")).all() and (got[2] == -float("inf")).all()


def test_grouped_allocates_its_output_and_takes_a_stream():
    g = gen(2)
    x, w, off = normal(g, 60, 128), normal(g, 2, 64, 128), offsets([20, 40])
    want = moe.grouped_matmul(up(x), up(w), up(off))
    side = torch.cuda.Stream()
    dx, dw, doff = up(x), up(w), up(off)
    torch.cuda.synchronize()
    got = moe.grouped_matmul(dx, dw, doff, out_dtype=BF, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


# ---- rows -------------------------------------------------------------------------

def routing(N, k, E, L, seed):
    g = gen(seed)
    expert = torch.rand(N, E, generator=g).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(expert, stable=True).indices
    local = order[expert[order] < L]
    row_pair = torch.full((N * k,), -5, dtype=torch.int32)
    row_pair[:len(local)] = local.to(torch.int32)
    pair_row = torch.full((N * k,), -1, dtype=torch.int32)
    pair_row[local] = torch.arange(len(local), dtype=torch.int32)
    return row_pair, pair_row, offsets(torch.bincount(expert, minlength=E)[:L].numpy()), len(local)


@pytest.mark.parametrize("dtype", [BF, F32, torch.uint8], ids=["bf16", "fp32", "bytes"])
@pytest.mark.parametrize("N,k,E,L,H", [(1, 1, 1, 1, 8), (40, 3, 8, 2, 264), (7, 8, 16, 16, 1000), (33, 2, 4, 1, 37), (5, 4, 64, 1, 4096),
                                       (300, 16, 32, 8, 136)])
def test_dispatch_rows(N, k, E, L, H, dtype):
    row_pair, _, off, R = routing(N, k, E, L, N + H)
    x = torch.randint(0, 255, (N, H), generator=gen(1)).to(dtype)
    out = torch.full((N * k + 3, H), 9, dtype=dtype).cuda()
    pair = torch.cat([row_pair, torch.zeros(3, dtype=torch.int32)])
    say(f"dispatch N={N} k={k} H={H} {dtype} R={R}")
    got = moe.dispatch_rows(up(x), up(pair), up(off), k, out=out).cpu()
    assert torch.equal(got[:R], x[row_pair[:R].long() // k])
    assert (got[R:] == 9).all()


def test_dispatch_rows_strides_and_pairs_out_of_range():
    x = normal(gen(3), 20, 48)
    pair = torch.tensor([0, 39, 40, -1, 7, 2 ** 31 - 1], dtype=torch.int32)
    for lead, pad in ((0, 8), (1, 3), (0, 0)):
        got = moe.dispatch_rows(strided(x, pad, lead), up(pair), up(offsets([6])), 2, out=strided(torch.zeros(6, 48, dtype=BF), pad, lead)).cpu()
        want = x[[0, 19, 0, 0, 3, 0]]
        want[[2, 3, 5]] = 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,k,E,L,H", [(1, 1, 1, 1, 8), (40, 3, 8, 2, 264), (7, 8, 16, 16, 1000), (33, 2, 4, 1, 37), (300, 16, 32, 8, 136)])
def test_combine_rows(N, k, E, L, H, out_dtype):
    _, pair_row, _, R = routing(N, k, E, L, N + H)
    rows = normal(gen(4), R + 2, H)
    pair_row[0] = R + 2 if pair_row[0] < 0 else pair_row[0]   # past the rows: adds nothing
    at = pair_row.long().view(N, k)
    use = (at >= 0) & (at < R + 2)
    ref = torch.zeros(N, H, dtype=torch.float64)
    seq = torch.zeros(N, H, dtype=F32)
    for j in range(k):
        v = torch.where(use[:, j:j + 1], rows[at[:, j].clamp(0, R + 1)].float(), torch.zeros(()))
        ref += v.double()
        seq = seq + v
    got = moe.combine_rows(up(rows), up(pair_row), k, out_dtype=out_dtype).cpu()
    mag = ref.abs()
    assert torch.equal(got, seq.to(out_dtype)), "the fp32 sum in ascending slots, rounded once"
    assert_close(got, ref, out_dtype, mag + 16, k, "combine")
    lead = moe.combine_rows(strided(rows, 3, 1), up(pair_row), k, out=strided(torch.zeros(N, H, dtype=out_dtype), 3, 1)).cpu()
    assert torch.equal(lead, got)


@pytest.mark.parametrize("H", [37, 512, 520, 1016, 1030, 2056, 4104])
def test_combine_rows_of_many_tokens(H):
    # more than 1024 tokens: threads a token by the row's length; an odd number of them
    test_combine_rows(1101, 3, 4, 2, H, BF)


# ---- SwiGLU ------------------------------------------------------------------------

def swiglu_ref(a, weight, dh=None):
    I = a.shape[1] // 2
    g, u = a[:, :I].double(), a[:, I:].double()
    w = torch.ones(a.shape[0], 1, dtype=torch.float64) if weight is None else weight.double()[:, None]
    s = 1 / (1 + torch.exp(-g))
    h = g * s * u * w
    if dh is None:
        return h
    d = dh.double()
    return h, torch.cat([d * w * u * s * (1 + g * (1 - s)), d * w * g * s], 1), (d * g * s * u).sum(1), (d * g * s * u).abs().sum(1)


def swiglu_tol(a, ref):
    # e^-g through 2^(-g log2 e): the product is off by half a unit, 2^-24 |g|
    # relative in the result; exp2, 1 + e, the reciprocal and three products a
    # unit each. silu and its derivative carry that, the derivative's two terms
    # each: (|g| + 8) 2^-22.
    I = a.shape[1] // 2
    g = a[:, :I].double().abs()
    return (g + 8) * 2.0 ** -22


@pytest.mark.parametrize("R,I", [(1, 8), (3, 64), (17, 128), (40, 520), (5, 2048), (300, 136), (4, 37), (2, 5000)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_forward_and_backward(R, I, weighted):
    g = gen(R * I)
    a = normal(g, R + 2, 2 * I, std=3.0)
    a[0, :min(4, I)] = torch.tensor([100.0, -100.0, 0.0, -0.0], dtype=BF)[:min(4, I)]
    weight = torch.rand(R + 2, generator=g) if weighted else None
    dh = normal(g, R + 2, I)
    off = offsets([R // 2, R - R // 2])
    h, da, dw, dwmag = swiglu_ref(a, weight, dh)
    rel = swiglu_tol(a, h)
    a[R:] = float("nan")
    for lead, pad in ((0, 0), (1, 3)):
        say(f"swiglu R={R} I={I} weighted={weighted} lead={lead}")
        da_in = strided(a, pad, lead)
        got = moe.swiglu(da_in, row_weight=up(weight), row_offset=up(off), out=strided(torch.full((R + 2, I), 7.0, dtype=BF), pad, lead)).cpu()
        assert (got[R:] == 7).all()
        err = (got[:R].double() - h[:R]).abs()
        assert (err <= h[:R].abs() * (HALF[BF] * (1 + 2.0 ** -8) + rel[:R]) + 2.0 ** -120).all()
        out = strided(torch.full((R + 2, 2 * I), 7.0, dtype=BF), pad, lead)
        dweight = torch.full((R + 2,), 7.0).cuda()
        moe.swiglu_backward(da_in, strided(dh, pad, lead), row_weight=up(weight), row_offset=up(off), out=out, drow_weight=dweight)
        got, gw = out.cpu(), dweight.cpu()
        assert (got[R:] == 7).all() and (gw[R:] == 7).all()
        # dg = dh w u (s + g s (1 - s)): the two terms may cancel, so its bar
        # goes by their magnitudes
        gd, s = a[:R, :I].double(), 1 / (1 + torch.exp(-a[:R, :I].double()))
        w = torch.ones(R, 1, dtype=torch.float64) if weight is None else weight[:R].double()[:, None]
        terms = dh[:R].double().abs() * w * a[:R, I:].double().abs() * (s + (gd * s * (1 - s)).abs() + (gd * s).abs() * 2.0 ** -10)
        mag = torch.cat([terms, da[:R, I:].abs()], 1)
        err = (got[:R].double() - da[:R]).abs()
        assert (err <= da[:R].abs() * HALF[BF] * (1 + 2.0 ** -8) + mag * torch.cat([rel[:R], rel[:R]], 1) + 2.0 ** -120).all()
        err = (gw[:R].double() - dw[:R]).abs()
        assert (err <= dwmag[:R] * ((I + 8) * ULP + rel[:R].max())).all()


def test_swiglu_backward_in_place_and_without_weights():
    g = gen(9)
    a, dh = normal(g, 20, 256), normal(g, 20, 128)
    want, dw = moe.swiglu_backward(up(a), up(dh))
    assert dw is None
    buf = up(a)
    got, _ = moe.swiglu_backward(buf, up(dh), out=buf)
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)


def test_swiglu_gradient_against_differences():
    # the formula the kernel implements, differentiated numerically in 64 bits
    g = gen(12)
    a, dh, weight = normal(g, 6, 48), normal(g, 6, 24), torch.rand(6, generator=g)
    da, dw = moe.swiglu_backward(up(a), up(dh), row_weight=up(weight))
    da, dw = da.double().cpu(), dw.double().cpu()
    f = lambda a_, w_: (swiglu_ref(a_, w_) * dh.double()).sum()   # noqa: E731
    for trial in range(6):
        va = torch.randn(6, 48, generator=g, dtype=torch.float64)
        vw = torch.randn(6, generator=g, dtype=torch.float64)
        h = 1e-6
        num = (f(a.double() + h * va, weight.double() + h * vw) - f(a.double() - h * va, weight.double() - h * vw)) / (2 * h)
        got = (da * va).sum() + (dw * vw).sum()
        # each of the 288 entries of da is rounded to bf16 (2^-8 of it)
        assert abs(got - num) <= (da * va).abs().sum() * 2.0 ** -8 + (dw * vw).abs().sum() * 1e-5 + 1e-6


# ---- quantisation ---------------------------------------------------------------------

def codes_of(t):
    return t.cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("R,C", [(1, 8), (5, 128), (130, 200), (257, 1000), (128, 4096), (3, 37), (300, 129)])
def test_quantize_is_the_formats_recipe_bit_for_bit(R, C, block_rows, dtype):
    g = gen(R * C + block_rows)
    x = torch.randn(R, C, generator=g) * torch.exp(3 * torch.randn(R, 1, generator=g))
    if R > 2:
        x[1] = 0
        x[2] *= 1e-30
    x = x.to(dtype)
    want_q, want_s = mi.quantize_e4m3_blocks(x.float().numpy(), block_rows, 128) if C % 128 == 0 and R % block_rows == 0 else padded_recipe(x, block_rows)
    say(f"quantize R={R} C={C} block_rows={block_rows} {dtype}")
    for lead, pad in ((0, 0), (1, 3)):
        q, s = moe.quantize_fp8(strided(x, pad, lead), block_rows=block_rows, out=strided(torch.zeros(R, C, dtype=F8), pad, lead))
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(codes_of(q.contiguous()), want_q)


def padded_recipe(x, block_rows):
    R, C = x.shape
    p = np.zeros((-(-R // block_rows) * block_rows, -(-C // 128) * 128), np.float32)
    p[:R, :C] = x.float().numpy()
    q, s = mi.quantize_e4m3_blocks(p, block_rows, 128)
    return q[:R, :C], s


def test_quantize_near_ties_and_extremes():
    # every quotient lands on or next to a border between two codes, in the
    # normal and the subnormal range: amax 448 makes the scale 1
    base = np.array([float(torch.tensor(c, dtype=torch.uint8).view(F8).float()) for c in range(127)], np.float32)
    mid = (base[1:] + base[:-1]) / 2
    v = np.concatenate([mid, np.nextafter(mid, np.float32(1e9)), np.nextafter(mid, np.float32(0)), base[1:], [448.0]]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
    x = np.concatenate([np.full((len(v), 1), 448, np.float32), v], 1)
    for scale in (1.0, 1.0 / 3.0, 3.1e-5, 7.7e20):
        xs = (x * np.float32(scale)).astype(np.float32)
        want_q, want_s = mi.quantize_e4m3_blocks(xs, 1, 128)
        q, s = moe.quantize_fp8(torch.from_numpy(xs).cuda())
        assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(codes_of(q), want_q)


def test_quantize_tiny_and_non_finite_blocks():
    x = torch.zeros(4, 256)
    x[0, 3], x[1, 5], x[2, 7] = float("inf"), float("nan"), 1e-44
    x[0, 128:], x[3] = 1.0, 1e-38
    q, s = moe.quantize_fp8(x.cuda())
    q, s = codes_of(q), s.cpu()
    assert torch.isinf(s[0, 0]) and torch.isnan(s[1, 0]) and s[2, 0] == 1 and s[0, 1] == torch.tensor(1.0) / 448
    assert (q[0, :128] == 0x7f).all() and (q[1, :128] == 0x7f).all() and (q[2] == 0).all()
    assert (q[0, 128:] == 0x7e).all()
    want_q, want_s = mi.quantize_e4m3_blocks(x[3:].numpy(), 1, 128)
    assert np.array_equal(q[3:], want_q) and np.array_equal(s[3:].numpy(), want_s)


def test_quantize_batches_and_row_offset():
    x = normal(gen(6), 3, 130, 264)
    q, s = moe.quantize_fp8(up(x), block_rows=128)
    for e in range(3):
        qe, se = moe.quantize_fp8(up(x[e]), block_rows=128)
        assert torch.equal(q[e].view(torch.uint8), qe.view(torch.uint8)) and torch.equal(s[e], se)
    out, scales = torch.full((130, 264), 1.0).to(F8).cuda(), torch.full((130, 3), 9.0).cuda()
    moe.quantize_fp8(up(x[0]), row_offset=up(offsets([4, 100], 2)), out=out, scales=scales)
    want, ws = moe.quantize_fp8(up(x[0]))
    assert torch.equal(out[2:106].view(torch.uint8), want[2:106].view(torch.uint8)) and torch.equal(scales[2:106], ws[2:106])
    assert (out.float()[:2] == 1).all() and (out.float()[106:] == 1).all() and (scales[106:] == 9).all()


@pytest.mark.parametrize("R,I", [(1, 128), (9, 2048), (40, 200), (3, 37)])
def test_swiglu_to_e4m3(R, I):
    g = gen(I)
    a, weight = normal(g, R, 2 * I), torch.rand(R, generator=g)
    h = swiglu_ref(a, weight)
    q, s = moe.swiglu(up(a), row_weight=up(weight), out_dtype=F8)
    q, s = q.float().cpu().double(), s.cpu().double()
    pad = torch.zeros(R, -(-I // 128) * 128, dtype=torch.float64)
    pad[:, :I] = h
    amax = pad.view(R, -1, 128).abs().amax(2)
    rel = float(swiglu_tol(a, h).max())
    assert ((s - amax / 448).abs() <= amax / 448 * (rel + 2.0 ** -23)).all()
    spread = s.repeat_interleave(128, 1)[:, :I]
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6
    assert ((q * spread - h).abs() <= torch.maximum(h.abs() * 2.0 ** -4, spread * 2.0 ** -10) * (1 + 1e-5) + h.abs() * 2 * rel).all()


# ---- e4m3 products -----------------------------------------------------------------------

def e4m3(g, *shape):
    return (torch.randn(*shape, generator=g) * 100).clamp(-448, 448).to(F8)


def fp8_reference(x, xs, w, ws, off):
    K, n = x.shape[1], w.shape[-2]
    kb, nb = torch.arange(K) // 128, torch.arange(n) // 128
    xd = x.double() * xs.double()[:, kb]
    w, ws = (w, ws) if w.dim() == 3 else (w[None], ws[None])
    out = torch.zeros(x.shape[0], n, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(w.shape[0]):
        r = slice(int(off[e]), int(off[e + 1]))
        wd = w[e].double() * ws[e].double()[nb][:, kb]
        out[r], mag[r] = xd[r] @ wd.t(), xd[r].abs() @ wd.abs().t()
    return out, mag


FP8_SHAPES = [
    (None, 1, 128, 64), (None, 1, 2048, 512), (None, 5, 7168, 136), (None, 33, 272, 200), (None, 300, 1024, 640), (None, 260, 16, 8),
    (None, 129, 37, 19), (None, 1, 1, 1),
    ([0, 1, 0, 9], 10, 256, 128), ([33, 0, 64, 129, 1], 227, 400, 264), ([300, 4, 500], 804, 512, 768), ([2, 3], 5, 130, 257),
    ([16, 17, 15, 31, 32, 33], 144, 256, 128),
]


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("counts,R,K,n", FP8_SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_fp8_matches_64_bits(counts, R, K, n, out_dtype):
    run_fp8(counts, R, K, n, out_dtype)


@pytest.mark.parametrize("pad,lead", [(16, 0), (16, 16), (3, 1), (8, 8)])
@pytest.mark.parametrize("counts,R", [(None, 70), ([40, 0, 25], 65)])
def test_fp8_strides_and_alignment(counts, R, pad, lead):
    run_fp8(counts, R, 272, 136, BF, pad=pad, lead=lead, behind=6 if counts else 0)


@pytest.mark.parametrize("expected", [1, 40, 200, 5000])
def test_fp8_tile_choice_changes_no_result(expected):
    run_fp8([0, 33, 290, 5], 328, 384, 320, BF, expected_rows=expected, behind=1)


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", range(1, 10))
@pytest.mark.parametrize("counts,R,K,n", [([0, 33, 290, 1], 324, 272, 328), (None, 300, 64, 8), ([3, 0, 200], 203, 16, 64),
                                          ([64, 128], 192, 512, 256), (None, 1, 8336, 136), (None, 257, 1040, 520)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_fp8_every_tile(counts, R, K, n, tile, out_dtype):
    run_fp8(counts, R, K, n, out_dtype, behind=3 if counts else 0, pad=16, tile=tile)


def run_fp8(counts, R, K, n, out_dtype, pad=0, lead=0, behind=0, expected_rows=None, tile=0, splits=0):
    g = gen(R + K + n)
    rows = R + behind
    L = 0 if counts is None else len(counts)
    off = offsets([rows] if counts is None else counts)
    x, w = e4m3(g, rows, K), e4m3(g, *((L,) if L else ()), n, K)
    xs = torch.rand(rows, -(-K // 128), generator=g) * 0.02 + 1e-3
    ws = torch.rand(*((L,) if L else ()), -(-n // 128), -(-K // 128), generator=g) * 0.01 + 1e-3
    ref, mag = fp8_reference(x, xs, w, ws, off)
    if behind:
        xs[R:] = float("nan")
    y = torch.full((rows, n), 7.0, dtype=out_dtype)
    say(f"fp8 counts={counts} R={R} K={K} n={n} {out_dtype} pad={pad} lead={lead}")
    got = moe.fp8_matmul(strided(x, pad, lead), strided(xs, 1 if pad else 0), strided(w, pad, lead), up(ws), row_offset=None if counts is None else up(off),
                         out=strided(y, pad, lead), expected_rows=expected_rows, tile=tile, splits=splits).cpu()
    assert_close(got[:R], ref[:R], out_dtype, mag[:R], K, f"fp8 {counts} {K} {n}", DROP)
    assert (got[R:] == 7).all()


# ---- together -------------------------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True])
def test_training_step_of_the_experts(graph):
    """Routing layout, rows to the experts, both products with SwiGLU between,
    rows back, and every gradient, against autograd in 64 bits; once as eager
    calls and once captured in a HIP graph and replayed three times with eager
    work between."""
    S, T, E, k, L, H, I = 2, 30, 8, 3, 4, 256, 128
    N = S * T
    g = gen(77)
    x, dy = normal(g, N, H), normal(g, N, H)
    w1, w2 = normal(g, L, 2 * I, H, std=0.06), normal(g, L, H, I, std=0.06)
    logits = torch.randn(N, E, generator=g)
    ffn = moe.MoeExpertFFN(S, T, E, k, 0, L, H, I)
    lb = ffn.layout(logits=up(logits))
    cap = N * k
    d = {n: up(t) for n, t in dict(x=x, dy=dy, w1=w1, w2=w2).items()}
    e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    b = dict(xr=e(cap, H), a=e(cap, 2 * I), h=e(cap, I), yr=e(cap, H), y=e(N, H, dt=F32), dyr=e(cap, H), dh=e(cap, I), da=e(cap, 2 * I),
             dw=e(cap, dt=F32), dxr=e(cap, H), dx=e(N, H, dt=F32), dw1=e(L, 2 * I, H, dt=F32), dw2=e(L, H, I, dt=F32))

    def step():
        off = lb.row_offset
        moe.dispatch_rows(d["x"], lb.row_pair, off, k, out=b["xr"])
        moe.grouped_matmul(b["xr"], d["w1"], off, out=b["a"])
        moe.swiglu(b["a"], row_weight=lb.row_weight, row_offset=off, out=b["h"])
        moe.grouped_matmul(b["h"], d["w2"], off, out=b["yr"])
        moe.combine_rows(b["yr"], lb.pair_row, k, out=b["y"])
        moe.dispatch_rows(d["dy"], lb.row_pair, off, k, out=b["dyr"])
        moe.grouped_matmul_dgrad(b["dyr"], d["w2"], off, out=b["dh"])
        moe.grouped_matmul_wgrad(b["dyr"], b["h"], off, out=b["dw2"])
        moe.swiglu_backward(b["a"], b["dh"], row_weight=lb.row_weight, row_offset=off, out=b["da"], drow_weight=b["dw"])
        moe.grouped_matmul_dgrad(b["da"], d["w1"], off, out=b["dxr"])
        moe.grouped_matmul_wgrad(b["da"], b["xr"], off, out=b["dw1"])
        moe.combine_rows(b["dxr"], lb.pair_row, k, out=b["dx"])

    outs = ("y", "dx", "dw1", "dw2", "dw")
    step()
    torch.cuda.synchronize()
    eager = {n: b[n].clone() for n in outs}
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        for r in range(3):
            for n in outs:
                b[n].fill_(3.0)
            (d["x"] + 1).sum().item()
            say(f"replay {r}")
            cg.replay()
            torch.cuda.synchronize()
            R = int(lb.row_offset[-1])
            for n in outs:
                rows = slice(0, R) if n == "dw" else slice(None)
                assert torch.equal(b[n][rows], eager[n][rows]), n
        return

    # 64-bit autograd of the same function of the same inputs
    R = int(lb.row_offset[-1])
    off = lb.row_offset.cpu().tolist()
    pair, weight = lb.row_pair.cpu().long()[:R], lb.row_weight.cpu().double()[:R]
    X, W1, W2, Wt = (t.clone().requires_grad_() for t in (x.double(), w1.double(), w2.double(), weight))
    rows = X[pair // k]
    parts = []
    for ex in range(L):
        r = slice(off[ex], off[ex + 1])
        a = rows[r] @ W1[ex].t()
        parts.append((torch.nn.functional.silu(a[:, :I]) * a[:, I:] * Wt[r, None]) @ W2[ex].t())
    Y = torch.zeros(N, H, dtype=torch.float64).index_add(0, pair // k, torch.cat(parts))
    (Y * dy.double()).sum().backward()
    # a, h, the expert rows, dh, da and dx rows are each rounded to bf16 on the
    # way: up to five roundings of 2^-8 stand behind an entry of dx or dw1, in
    # sums of independent errors; the bar is five whole ones of the norm
    for n, ref in (("y", Y.detach()), ("dx", X.grad), ("dw1", W1.grad), ("dw2", W2.grad), ("dw", Wt.grad)):
        got = eager[n].double().cpu()[: len(ref)]
        err = (got - ref).norm() / ref.norm()
        say(f"training step {n}: {err:.2e}")
        assert err <= 5 * 2.0 ** -8, n
    # and against differences of the 64-bit function
    f = lambda X_: (torch.zeros(N, H, dtype=torch.float64).index_add(0, pair // k, torch.cat([   # noqa: E731
        (lambda a: (torch.nn.functional.silu(a[:, :I]) * a[:, I:] * weight[off[ex]:off[ex + 1], None]) @ w2[ex].double().t())(
            X_[pair // k][off[ex]:off[ex + 1]] @ w1[ex].double().t()) for ex in range(L)])) * dy.double()).sum()
    v = torch.randn(N, H, generator=g, dtype=torch.float64)
    num = (f(x.double() + 1e-6 * v) - f(x.double() - 1e-6 * v)) / 2e-6
    got = (eager["dx"].double().cpu() * v).sum()
    assert abs(got - num) <= 5 * 2.0 ** -8 * X.grad.norm() * 4   # 4 standard deviations of an error along v


def test_fp8_layer():
    """Quantise, block-scaled product, SwiGLU to e4m3, second product: a dense
    fp8 layer, against 64 bits on the same codes."""
    g = gen(8)
    M, H, I = 37, 512, 256
    x, w1, w2 = normal(g, M, H), normal(g, 2 * I, H, std=0.05), normal(g, H, I, std=0.05)
    qx, sx = moe.quantize_fp8(up(x))
    q1, s1 = moe.quantize_fp8(up(w1), block_rows=128)
    q2, s2 = moe.quantize_fp8(up(w2), block_rows=128)
    a = moe.fp8_matmul(qx, sx, q1, s1)
    qh, sh = moe.swiglu(a, out_dtype=F8)
    y = moe.fp8_matmul(qh, sh, q2, s2)
    torch.cuda.synchronize()
    c = lambda t: t.cpu()   # noqa: E731
    ref, mag = fp8_reference(c(qx), c(sx), c(q1), c(s1), [0, M])
    assert_close(a, ref, BF, mag, H, "first product", DROP)
    ref, mag = fp8_reference(c(qh), c(sh), c(q2), c(s2), [0, M])
    assert_close(y, ref, BF, mag, I, "second product", DROP)
    # the whole layer against the unquantised one: x, w1 and w2, h each carry
    # half-step errors of 2^-4 at most, independent over hundreds of terms
    ad = x.double() @ w1.double().t()
    full = (torch.nn.functional.silu(ad[:, :I]) * ad[:, I:]) @ w2.double().t()
    assert (y.double().cpu() - full).norm() / full.norm() <= 2 * 2.0 ** -4


def test_two_streams_at_once():
    g = gen(15)
    x, w, off = normal(g, 500, 512), normal(g, 4, 512, 512, std=0.05), offsets([100, 150, 50, 200])
    dx, dw, doff = up(x), up(w), up(off)
    want_f = moe.grouped_matmul(dx, dw, doff)
    want_w = moe.grouped_matmul_wgrad(want_f, dx, doff)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        a = moe.grouped_matmul(dx, dw, doff, stream=s1)
        b = moe.grouped_matmul_wgrad(want_f, dx, doff, stream=s2)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want_f) and torch.equal(b, want_w)


def test_checks_hold_for_sizes_seen_before():
    # a call of known sizes skips the checks that sizes settle, and no other
    g = gen(41)
    x, w, off = up(normal(g, 30, 64)), up(normal(g, 2, 32, 64)), up(offsets([10, 20]))
    out = torch.empty(30, 32, dtype=BF, device="cuda")
    want = moe.grouped_matmul(x, w, off).clone()
    for _ in range(2):
        assert torch.equal(moe.grouped_matmul(x, w, off, out=out), want)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w.clone().requires_grad_(), off, out=out)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w, off, out=out.cpu())
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w, off.cpu(), out=out)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w.transpose(0, 1), off, out=out)
    with pytest.raises(ValueError):
        moe.grouped_matmul(x, w, off.long(), out=out)
    with pytest.raises(_lib.MoeError):
        moe.grouped_matmul(x, w, off, out=out, tile=99)
    # an unaligned tensor of the same sizes takes another kernel, same numbers
    buf = torch.empty(30 * 64 + 1, dtype=BF, device="cuda")
    xu = buf[1:].view(30, 64)
    xu.copy_(x)
    got = moe.grouped_matmul(xu, w, off)
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
