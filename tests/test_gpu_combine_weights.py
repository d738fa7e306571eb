"""Each token's rows combined with the router's weights, and its gradients,
against plain 64-bit implementations.

Bars, derived: k fused multiply-adds in fp32, each off by half a unit (2^-24) of the
running sum, at most of the magnitudes; then one rounding (bf16 2^-8). A product
w dy rounded to fp32 and to bf16: 2^-24 and 2^-8. A dot product of H columns: a
thread adds up at most ceil(H / 64) + 8 of them (64 threads or more take a row),
six additions join the lanes and three the wavefronts: (ceil(H / 64) + 24) 2^-24
of the magnitudes."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from test_gpu_operators import BF, F32, HALF, gen, normal, routing, say, strided, up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [(1, 1, 1, 1, 8), (1, 8, 16, 2, 7168), (40, 3, 8, 2, 264), (7, 8, 16, 16, 1000), (33, 2, 4, 1, 37), (300, 16, 32, 8, 136),
         (5, 4, 4, 4, 8200), (2, 2, 2, 2, 20001), (1500, 4, 16, 4, 40), (1100, 2, 8, 4, 1000), (1050, 8, 64, 8, 2056), (1030, 3, 8, 2, 7168)]


def case(N, k, E, L, H, dy_dtype=BF):
    _, pair_row, _, R = routing(N, k, E, L, N + H)
    g = gen(N + k)
    rows, weights = normal(g, R + 2, H), torch.rand(N, k, generator=g)
    if pair_row[0] < 0:
        pair_row[0] = R + 2   # past the rows: no row
    here = (pair_row >= 0) & (pair_row < R + 2)
    weights.view(-1)[~here] = float("nan")   # not looked at
    return rows, weights, pair_row, here.view(N, k), normal(g, N, H, std=0.5, dtype=dy_dtype)


def near(got, ref, tol, what):
    bad = ~((got.double().cpu() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("out_dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,k,E,L,H", SIZES)
def test_weighted_combine(N, k, E, L, H, out_dtype):
    rows, weights, pair_row, here, _ = case(N, k, E, L, H)
    at = pair_row.long().view(N, k)
    ref, mag = torch.zeros(N, H, dtype=torch.float64), torch.zeros(N, H, dtype=torch.float64)
    for j in range(k):
        t = rows[at[:, j].clamp(0, len(rows) - 1)].double() * torch.where(here[:, j], weights[:, j], 0.0).double()[:, None]
        ref, mag = ref + t, mag + t.abs()
    say(f"weighted combine {N} {k} {H} {out_dtype}")
    got = moe.combine_rows(up(rows), up(pair_row), k, out_dtype=out_dtype, weights=up(weights))
    near(got, ref, HALF[out_dtype] * 1.01 * ref.abs() + (k + 1) * U * mag + 1e-37, "combine")
    for pad, lead in ((3, 1), (8, 8)):
        out = strided(torch.zeros(N, H, dtype=out_dtype), pad, lead)
        assert torch.equal(moe.combine_rows(strided(rows, pad, lead), up(pair_row), k, out=out, weights=up(weights)), got)
    ones = torch.ones(N, k)
    assert torch.equal(moe.combine_rows(up(rows), up(pair_row), k, out_dtype=out_dtype, weights=up(ones)),
                       moe.combine_rows(up(rows), up(pair_row), k, out_dtype=out_dtype))


@pytest.mark.parametrize("dy_dtype", [BF, F32], ids=["dy_bf16", "dy_fp32"])
@pytest.mark.parametrize("N,k,E,L,H", SIZES)
def test_weighted_combine_backward(N, k, E, L, H, dy_dtype):
    rows, weights, pair_row, here, dy = case(N, k, E, L, H, dy_dtype)
    R = len(rows)
    out = torch.full((R, H), 7.0, dtype=BF)
    say(f"weighted combine backward {N} {k} {H} {dy_dtype}")
    dweights = torch.full((N, k), 9.0)
    got, dw = moe.combine_rows_backward(up(dy), up(rows), up(pair_row), up(weights), out=up(out), dweights=up(dweights))
    n, j = torch.nonzero(here, as_tuple=True)
    r = pair_row.view(N, k)[n, j].long()
    ref = out.double()
    ref[r] = weights[n, j].double()[:, None] * dy[n].double()
    tol = torch.zeros_like(ref)
    tol[r] = (HALF[BF] * 1.01 + U) * ref[r].abs() + 1e-37
    near(got, ref, tol, "rows")
    refw, magw = torch.zeros(N, k, dtype=torch.float64), torch.zeros(N, k, dtype=torch.float64)
    refw[n, j] = (rows[r].double() * dy[n].double()).sum(dim=1)
    magw[n, j] = (rows[r].double() * dy[n].double()).abs().sum(dim=1)
    near(dw, refw, (-(-H // 64) + 24) * U * magw, "weights")
    for pad, lead in ((3, 1), (8, 8)):
        again, dwa = moe.combine_rows_backward(strided(dy, pad, lead), strided(rows, pad, lead), up(pair_row), up(weights), out=strided(out, pad, lead))
        assert torch.equal(again, got)
        near(dwa, refw, (-(-H // 64) + 24) * U * magw, "weights, rows apart")
    both = up(rows)   # written over the rows themselves
    over, dwo = moe.combine_rows_backward(up(dy), both, up(pair_row), up(weights), out=both)
    assert over is both and torch.equal(over[up(r)], got[up(r)]) and torch.equal(dwo, dw)


@pytest.mark.parametrize("N", [40, 1200])
@pytest.mark.parametrize("H", [515, 1027, 2051, 4099, 8195])
def test_rows_whose_end_is_a_wavefronts_first_piece_in_place(H, N):
    # a wavefront may be done with its part of the row before another has read the end of it
    rows, weights, pair_row, here, dy = case(N, 2, 8, 8, H)
    weights = torch.nan_to_num(weights)
    out = up(torch.zeros_like(rows))
    want, dw = moe.combine_rows_backward(up(dy), up(rows), up(pair_row), up(weights), out=out)
    both = up(rows)
    got, dwo = moe.combine_rows_backward(up(dy), both, up(pair_row), up(weights), out=both)
    r = up(pair_row.long()[here.view(-1)])
    assert torch.equal(got[r], want[r]) and torch.equal(dwo, dw)


def test_infinities_stay_in_their_rows():
    N, k, H = 6, 2, 72
    rows, weights, dy = normal(gen(1), 12, H), torch.rand(N, k, generator=gen(2)), normal(gen(3), N, H)
    pair_row = torch.arange(12, dtype=torch.int32)
    want, ww = moe.combine_rows_backward(up(dy), up(rows), up(pair_row), up(weights))
    wy = moe.combine_rows(up(rows), up(pair_row), k, weights=up(weights))
    rows[5], dy[4] = float("nan"), float("inf")
    got, gw = moe.combine_rows_backward(up(dy), up(rows), up(pair_row), up(weights))
    gy = moe.combine_rows(up(rows), up(pair_row), k, weights=up(weights))
    clean = [i for i in range(12) if i not in (8, 9)]
    assert torch.equal(got[clean], want[clean]) and torch.equal(gy[[0, 1, 3, 4, 5]], wy[[0, 1, 3, 4, 5]]) and torch.isnan(gy[2]).all()
    cleanw = [i for i in range(12) if i not in (5, 8, 9)]
    assert torch.equal(gw.view(-1)[cleanw], ww.view(-1)[cleanw]) and torch.isnan(gw.view(-1)[5])


def test_no_tokens_and_no_rows():
    none = torch.zeros(0, 4)
    drows, dw = moe.combine_rows_backward(up(torch.zeros(0, 16, dtype=BF)), up(torch.ones(3, 16, dtype=BF)),
                                          up(torch.zeros(0, dtype=torch.int32)), up(none), out=up(torch.ones(3, 16, dtype=BF)))
    assert (drows == 1).all() and dw.shape == (0, 4)
    drows, dw = moe.combine_rows_backward(up(torch.ones(5, 16, dtype=BF)), up(torch.zeros(0, 16, dtype=BF)),
                                          up(torch.zeros(10, dtype=torch.int32)), up(torch.ones(5, 2)))
    assert drows.shape == (0, 16) and (dw == 0).all()
    y = moe.combine_rows(up(torch.zeros(0, 16, dtype=BF)), up(torch.zeros(10, dtype=torch.int32)), 2, weights=up(torch.ones(5, 2)))
    assert (y == 0).all()


def test_gradient_against_differences():
    N, k, E, L, H = 30, 3, 6, 6, 200
    rows, weights, pair_row, here, dy = case(N, k, E, L, H, F32)
    g = gen(50)
    f = lambda z, w: ((z[pair_row.long().view(N, k)] * w[..., None]).sum(dim=1) * dy.double()).sum()   # noqa: E731
    z, w = rows.double(), weights.double()
    assert here.all()
    dz, dw = moe.combine_rows_backward(up(dy), up(rows), up(pair_row), up(weights), out=torch.zeros(len(rows), H, dtype=BF, device="cuda"))
    vz, vw = torch.randn(z.shape, generator=g, dtype=torch.float64), torch.randn(w.shape, generator=g, dtype=torch.float64)
    h = 1e-3   # f is linear in either
    num = (f(z + h * vz, w) - f(z - h * vz, w)) / (2 * h)
    assert abs((dz.double().cpu() * vz).sum() - num) <= (HALF[BF] * 1.02 * dz.double().cpu().abs() * vz.abs()).sum() + 1e-9
    num = (f(z, w + h * vw) - f(z, w - h * vw)) / (2 * h)
    mag = (rows[pair_row.long().view(N, k)].double() * dy.double()[:, None]).abs().sum(dim=2)
    assert abs((dw.double().cpu() * vw).sum() - num) <= ((-(-H // 64) + 24) * U * mag * vw.abs()).sum() + 1e-9
