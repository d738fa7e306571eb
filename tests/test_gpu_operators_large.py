"""The operators around the expert FFN on buffers past 4 GiB and 2^31
elements: offsets that do not fit 32 bits, checked at the last rows against
64-bit products of slices (bars as in test_gpu_operators.py)."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ULP = 2.0 ** -23


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def randn(*shape, std=1.0, dtype=BF, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def off(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def close(got, ref, mag, terms, drop=0.0):
    err = (got.double() - ref).abs()
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    assert (err <= half * 1.01 * (ref.abs() + drop * mag) + ((terms + 8) * ULP + drop) * mag).all()


R, K, N = 70_000, 32_768, 64   # x: 4.6 GB


@pytest.mark.parametrize("tile", [0, 1, 5])
def test_grouped_rows_past_4_gib(tile):
    x, w = randn(R, K), randn(2, N, K, std=0.02)
    o = off(0, 30, R)
    print("[large] forward", flush=True)
    y = moe.grouped_matmul(x, w, o, tile=tile)
    torch.cuda.synchronize()
    for r, e in ((slice(0, 8), 0), (slice(30, 38), 1), (slice(R - 8, R), 1)):
        a, b = x[r].double(), w[e].double()
        close(y[r], a @ b.t(), a.abs() @ b.abs().t(), K)
    print("[large] wgrad", flush=True)
    dw = moe.grouped_matmul_wgrad(y, x, o, out_dtype=F32, tile=tile)
    torch.cuda.synchronize()
    for c in (slice(0, 16), slice(K - 16, K)):
        a, b = y[30:].double(), x[30:, c].double()
        close(dw[1][:, c], a.t() @ b, a.abs().t() @ b.abs(), R)
    print("[large] dgrad", flush=True)
    dx = moe.grouped_matmul_dgrad(y, w, o, out=x, tile=tile)
    torch.cuda.synchronize()
    for r, e in ((slice(0, 8), 0), (slice(R - 8, R), 1)):
        a, b = y[r].double(), w[e].double()
        close(dx[r], a @ b, a.abs() @ b.abs(), N)


def test_grouped_weights_past_4_gib():
    L, n = 40, 2048   # w: 5.4 GB
    w = randn(L, n, K, std=0.02)
    x = randn(20, K)
    o = off(*([0] * L), 20)   # every row belongs to the last expert
    y = moe.grouped_matmul(x, w, o)
    torch.cuda.synchronize()
    a, b = x.double(), w[-1].double()
    close(y, a @ b.t(), a.abs() @ b.abs().t(), K)
    dw = moe.grouped_matmul_wgrad(y, x, o, out=w)
    torch.cuda.synchronize()
    a, b = y[:, -16:].double(), x.double()
    close(dw[-1][-16:], a.t() @ b, a.abs().t() @ b.abs(), 20)
    assert not dw[0].any() and not dw[L - 2].any()


def test_fp8_and_quantize_past_4_gib():
    rows = 140_000   # codes: 4.6 GB, the values 9.2 GB
    x = randn(rows, K)
    q, s = moe.quantize_fp8(x)
    torch.cuda.synchronize()
    for r in (slice(0, 4), slice(rows - 4, rows)):
        amax = x[r].float().abs().view(4, -1, 128).amax(2)
        assert torch.equal(s[r], amax / torch.full_like(amax, 448.0))
        want = (x[r].float() / s[r].repeat_interleave(128, 1)).to(F8)
        assert torch.equal(q[r].view(torch.uint8), want.view(torch.uint8))
    del x
    w = randn(N, K, std=100.0).clamp_(-448, 448).to(F8)
    ws = torch.rand(1, K // 128, device="cuda") * 0.01
    y = moe.fp8_matmul(q, s, w, ws)
    torch.cuda.synchronize()
    for r in (slice(0, 8), slice(rows - 8, rows)):
        a = q[r].double() * s[r].double().repeat_interleave(128, 1)
        b = w.double() * ws.double().repeat_interleave(128, 1)
        close(y[r], a @ b.t(), a.abs() @ b.abs().t(), K, drop=7 * 2.0 ** -13)


def test_rows_past_4_gib():
    T, k = 40_000, 2
    x = randn(T, K)   # 2.6 GB
    pairs = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    rows = moe.dispatch_rows(x, pairs, off(0, T * k), k)   # 5.2 GB
    torch.cuda.synchronize()
    assert torch.equal(rows[:4], x[[T - 1, T - 1, T - 2, T - 2]]) and torch.equal(rows[-2:], x[[0, 0]])
    y = moe.combine_rows(rows, pairs, k, out=x)
    torch.cuda.synchronize()
    # token n's slots are rows T k - 1 - 2n and one before: twice its own row
    assert torch.equal(y[-1], (2 * rows[0].float()).to(BF)) and torch.equal(y[0], (2 * rows[-1].float()).to(BF))


def test_swiglu_past_4_gib():
    rows, I = 40_000, 32_768   # gate and up: 5.2 GB
    a = randn(rows, 2 * I)
    h = moe.swiglu(a)
    torch.cuda.synchronize()
    last = slice(rows - 3, rows)
    g, u = a[last, :I].double(), a[last, I:].double()
    want = g / (1 + torch.exp(-g)) * u
    assert ((h[last].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()
    da, _ = moe.swiglu_backward(a, h, out=a)   # in place
    torch.cuda.synchronize()
    s = 1 / (1 + torch.exp(-g))
    du = h[last].double() * g * s
    assert ((da[last, I:].double() - du).abs() <= du.abs() * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()
