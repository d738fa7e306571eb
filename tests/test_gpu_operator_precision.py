"""Scales and sums of the block-scaled e4m3 product, pinned.

Two bars beside the elementwise worst case of the other tests, which for long
sums is several percent of a typical result:

Exact. Codes are whole numbers of -8 to 8, so eight products differ by less than
2^7 in size and none loses a bit in the matrix cores; block sums are whole
numbers under 2^13. Row scales are 1 + j/256 and weight scales 1/2, 1 or 2 (or
the other way round), so every scaled block sum is a multiple of 2^-9; where the
sum of their magnitudes is under 2^15, every partial sum in any order has at most
24 bits: fp32 results are equal to the formula's, bf16 ones to its one rounding.

Norm. With random codes the matrix cores drop bits below 2^-13 of the largest of
eight products, M: at most 2^-13 M of each product. Signs are random, so in the
norm these add up as squares: 2^-13 sqrt(sum of 8 M^2 over the groups of eight),
times the scales, over the outputs; fp32 additions of the block sums add 2^-24 of
what they reach each, far below. The mistakes that this is meant to find (scales,
block sums or accumulator in bf16) are planted in the oracle and lie above it."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def blocks(n):
    return -(-n // 128)


def scaled_block_sums(x, xs, w, ws):
    """[blocks, rows, n] in 64 bits: each block's sum, and with its scales."""
    K, n = x.shape[1], w.shape[0]
    p = torch.stack([x[:, b:b + 128].double() @ w[:, b:b + 128].double().t() for b in range(0, K, 128)])
    s = xs.double().t()[:, :, None] * ws.double()[torch.arange(n) // 128].t()[:, None, :]
    return p, p * s


def exact_inputs(g, rows, n, K, odd):
    whole = lambda *s: torch.randint(-8, 9, s, generator=g).float().to(F8)   # noqa: E731
    fine = lambda *s: 1 + torch.randint(0, 4, s, generator=g) / 256           # noqa: E731
    power = lambda *s: 2.0 ** torch.randint(-1, 2, s, generator=g)            # noqa: E731
    xs, ws = (rows, blocks(K)), (blocks(n), blocks(K))
    return (whole(rows, K), (fine if odd == "rows" else power)(*xs).float(), whole(n, K), (fine if odd == "weights" else power)(*ws).float())


def placed(t, pad, lead, fill=float("nan")):
    """t on the device in a larger buffer of `fill`, and that buffer's view of the
    columns behind every row."""
    shape = (*t.shape[:-1], t.shape[-1] + pad)
    buf = torch.full((lead + torch.Size(shape).numel(),), fill, dtype=F32).to(t.dtype).cuda()
    v = buf[lead:].view(shape)
    v[..., :t.shape[-1]].copy_(t)
    return v[..., :t.shape[-1]], v[..., t.shape[-1]:]


def run(counts, rows, n, K, odd, out_dtype, pad=0, lead=0, tile=0, splits=0):
    g = gen(rows * 7 + n + K)
    experts = counts or [rows]
    R = sum(experts)
    parts = [exact_inputs(g, c, n, K, odd) for c in experts]
    want = torch.zeros(R + 2, n, dtype=torch.float64)
    at = 1
    for part, c in zip(parts, experts):
        if c:
            _, scaled = scaled_block_sums(*part)
            assert scaled.abs().sum(0).max() < 2 ** 15 and (scaled * 2 ** 9).frac().abs().max() == 0
            want[at:at + c] = scaled.sum(0)
        at += c
    row = lambda i, fill: torch.cat([fill, *[p[i].float() for p in parts], fill])   # noqa: E731
    x, xs = row(0, torch.full((1, K), float("nan"))).to(F8), row(1, torch.full((1, blocks(K)), float("nan")))
    w, ws = torch.stack([p[2].float() for p in parts]).to(F8), torch.stack([p[3] for p in parts])
    off = None
    if counts:
        off = torch.cat([torch.tensor([1]), 1 + torch.tensor(experts).cumsum(0)]).to(torch.int32).cuda()
    else:
        x, xs, w, ws, want = x[1:-1], xs[1:-1], w[0], ws[0], want[1:-1]
    out, behind = placed(torch.full((len(x), n), 7.0, dtype=out_dtype), pad, lead)
    print(f"[ops] fp8 exact {counts} rows={rows} n={n} K={K} {odd} {out_dtype} pad={pad} lead={lead} tile={tile} splits={splits}", flush=True)
    moe.fp8_matmul(placed(x, pad, lead)[0], placed(xs, 1 if pad else 0, 0)[0], placed(w, pad, lead)[0], ws.cuda(), row_offset=off, out=out,
                   tile=tile, splits=splits)
    got = out.cpu()
    rows_of = slice(1, -1) if counts else slice(None)
    assert torch.equal(got[rows_of], want[rows_of].float().to(out_dtype))
    assert not counts or ((got[0] == 7).all() and (got[-1] == 7).all())
    assert torch.isnan(behind.float()).all(), "written behind a row's end"


SHAPES = [(None, 1, 136, 8336), (None, 300, 512, 1024), (None, 33, 200, 7168), ([0, 33, 257, 1], 291, 328, 1040), ([128, 0, 256], 384, 512, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("odd", ["rows", "weights"])
@pytest.mark.parametrize("counts,rows,n,K", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_scales_and_sums_are_exact(counts, rows, n, K, odd, out_dtype):
    run(counts, rows, n, K, odd, out_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("pad,lead", [(16, 16), (3, 1)], ids=["aligned", "odd"])
@pytest.mark.parametrize("counts,rows,n,K", SHAPES[1:], ids=lambda v: str(v).replace(" ", ""))
def test_strides_change_no_sum_and_no_padding(counts, rows, n, K, pad, lead, out_dtype):
    run(counts, rows, n, K, "rows", out_dtype, pad=pad, lead=lead)


@pytest.mark.gpu
@pytest.mark.parametrize("tile", range(1, 10))
def test_every_tile_is_exact(tile):
    run([0, 33, 257, 1], 291, 328, 1040, "rows", F32, pad=16, tile=tile)
    run(None, 256, 512, 2048, "weights", BF, pad=16, tile=tile)   # whole tiles
    run(None, 70, 264, 7168, "weights", F32, tile=tile, splits=3)


def random_inputs(K):
    g = gen(K)
    e4m3 = lambda *s: (torch.randn(*s, generator=g) * 110).clamp(-448, 448).to(F8)   # noqa: E731
    scale = lambda *s: (0.5 + torch.rand(*s, generator=g)) * 0.01                    # noqa: E731
    rows, n = 24, 40
    return e4m3(rows, K), scale(rows, blocks(K)), e4m3(n, K), scale(1, blocks(K))


def norm_bar(x, xs, w, ws):
    total = 0.0
    for b in range(0, x.shape[1], 128):
        xb, wb = x[:, b:b + 128].double(), w[:, b:b + 128].double()
        products = (xb[:, None] * wb[None]).abs()
        products = torch.nn.functional.pad(products, (0, -products.shape[2] % 8)).unflatten(2, (-1, 8))
        s = xs[:, b // 128].double()[:, None] * ws[0, b // 128].double()
        total += (8 * products.amax(3).square().sum(2) * s.square()).sum()
    return 2.0 ** -13 * float(total) ** 0.5


@pytest.mark.parametrize("K", [1024, 7168, 8336])
def test_the_norm_bar_finds_sums_and_scales_in_bf16(K):
    x, xs, w, ws = random_inputs(K)
    p, scaled = scaled_block_sums(x, xs, w, ws)
    ref, bar = scaled.sum(0), norm_bar(x, xs, w, ws)
    bf = lambda t: t.float().to(BF).double()   # noqa: E731
    acc = torch.zeros_like(ref)
    for part in scaled:
        acc = bf(acc + part)
    s = scaled / p
    for what, wrong in (("scales", scaled_block_sums(x, bf(xs), w, bf(ws))[1].sum(0)), ("block sums", (bf(p) * s).sum(0)), ("accumulator", acc)):
        assert (wrong - ref).norm() > 2 * bar, what


@pytest.mark.gpu
@pytest.mark.parametrize("tile,splits", [(0, 0), (0, 1), (1, 1), (6, 1), (9, 2)])
@pytest.mark.parametrize("K", [1024, 7168, 8336])
def test_random_sums_stay_in_the_norm_bar(K, tile, splits):
    x, xs, w, ws = random_inputs(K)
    got = moe.fp8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out_dtype=F32, tile=tile, splits=splits).cpu().double()
    ref = scaled_block_sums(x, xs, w, ws)[1].sum(0)
    bar = norm_bar(x, xs, w, ws)
    print(f"[ops] fp8 norm K={K} tile={tile} splits={splits}: {float((got - ref).norm() / ref.norm()):.2e}, bar {bar / float(ref.norm()):.2e}", flush=True)
    assert (got - ref).norm() <= bar
