"""RMS norm of the residual stream and its gradients against plain 64-bit
implementations.

Bars, derived. A thread adds up n = max(32, 8 ceil(H / 8192)) squares in fp32, ten
more additions join the threads (four behind a wavefront in order): relative
error at most (n + 16) 2^-24 of a sum of positive terms, half of that in its
square root, and less than 8 more roundings to y: y is off by at most
Y = ((n + 16) / 2 + 8) 2^-24 of its value before it is rounded (bf16: 2^-8).
dx adds two such sums and 16 roundings over the magnitudes |dres| + r (|g| +
|s| r^2 mean |g s|): at most (2 (n + 16) + 16) 2^-24 of them. dw adds up to R
terms in any order, each off by Y: (R + 16) 2^-24 + Y of the magnitudes."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from test_gpu_operators import BF, F32, F8, HALF, gen, normal, say, strided, up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def steps(H):
    return max(32, 8 * -(-H // 8192)) + 16


def bar_y(H):
    return (steps(H) / 2 + 8) * U


def reference(x, w, res, eps):
    """(stream as stored, y in 64 bits, r)"""
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    v = s.double()
    r = (v.square().mean(dim=1, keepdim=True) + eps).rsqrt()
    return s, v * r * (1.0 if w is None else w.double()), r


def inputs(R, H, dtype, seed, residual=True, wdtype=BF):
    g = gen(seed)
    x = normal(g, R, H, dtype=dtype)
    res = normal(g, R, H, std=3.0, dtype=dtype) if residual else None
    w = None if wdtype is None else (1 + normal(g, H, std=0.2, dtype=F32)).to(wdtype)
    return x, res, w, g


def near(got, ref, tol, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / tol).max():.3g} of the bar"


SIZES = [(1, 1), (1, 7168), (3, 7), (5, 64), (33, 100), (2, 128), (70, 129), (17, 1000), (300, 2048), (3, 2049), (5, 2056), (9, 4096), (4, 4104),
         (130, 7168), (3, 8192), (3, 8193), (2, 8200), (2, 16384), (3, 32768), (2, 32769), (2, 40000), (1, 131080), (2100, 64)]


@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,H", SIZES)
def test_rms_norm_matches_64_bits(R, H, dtype, residual):
    x, res, w, _ = inputs(R, H, dtype, R + H, residual, wdtype=[BF, F32, None][(R + H) % 3])
    s, ref, _ = reference(x, w, res, 1e-5)
    for out_dtype in (BF, F32):
        say(f"rms_norm {R} x {H} {dtype} residual={residual} {out_dtype}")
        got = moe.rms_norm(up(x), up(w), residual=up(res), eps=1e-5, out_dtype=out_dtype)
        if residual:
            got, stream = got
            assert torch.equal(stream.cpu(), s)
        near(got, ref, (HALF[out_dtype] * 1.01 + bar_y(H)) * ref.abs() + 1e-37, "y")


@pytest.mark.parametrize("pad,lead", [(0, 1), (8, 8), (3, 0), (5, 3)])
@pytest.mark.parametrize("quantize", [None, "fp8", "mx_e4m3", "mx_e2m1"])
def test_rms_norm_strides_and_alignment(quantize, pad, lead):
    R, H = 11, 328
    x, res, w, _ = inputs(R, H, BF, 5)
    want = moe.rms_norm(up(x), up(w), residual=up(res), quantize=quantize)
    out = torch.empty(R, want[0].shape[1] + pad, dtype=want[0].dtype, device="cuda")[:, :want[0].shape[1]]
    scales = None if quantize is None else torch.empty(R, want[1].shape[1] + pad, dtype=want[1].dtype, device="cuda")[:, :want[1].shape[1]]
    stream = strided(torch.zeros(R, H, dtype=BF), pad, lead)
    got = moe.rms_norm(strided(x, pad, lead), strided(w[None], 0, lead)[0], residual=strided(res, pad, lead), quantize=quantize, out=out,
                       scales=scales, residual_out=stream)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("H", [1, 37, 128, 1000, 2050, 7168, 16392, 40000])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_quantised_outputs_are_those_of_the_fp32_values(dtype, H):
    R = 9
    x, res, w, _ = inputs(R, H, dtype, H)
    x[2], res[2] = 0, 0   # a row of zeros
    y, s = moe.rms_norm(up(x), up(w), residual=up(res), out_dtype=F32)
    for quantize in ("fp8", "mx_e4m3", "mx_e2m1"):
        say(f"quantised norm {H} {dtype} {quantize}")
        q, scales, stream = moe.rms_norm(up(x), up(w), residual=up(res), quantize=quantize)
        wq, ws = moe.quantize_fp8(y) if quantize == "fp8" else moe.quantize_mx(y, quantize[3:])
        assert torch.equal(q.contiguous().view(torch.uint8), wq.contiguous().view(torch.uint8))
        assert torch.equal(scales.contiguous(), ws.contiguous())
        assert torch.equal(stream, s)


def test_in_place_and_rows_apart():
    x, res, w, _ = inputs(40, 520, BF, 3)
    y, s = moe.rms_norm(up(x), up(w), residual=up(res))
    for which in (0, 1):
        dx, dr = up(x), up(res)
        got, stream = moe.rms_norm(dx, up(w), residual=dr, residual_out=(dx, dr)[which])
        assert torch.equal(got, y) and torch.equal(stream, s) and stream is (dx, dr)[which]
    alone = moe.rms_norm(up(s.cpu()), up(w))
    d = up(s.cpu())
    assert moe.rms_norm(d, up(w), out=d) is d and torch.equal(d, alone) and torch.equal(alone, y)
    long = inputs(3, 40000, F32, 4)[0]
    want = moe.rms_norm(up(long), out_dtype=F32)
    d = up(long)
    assert torch.equal(moe.rms_norm(d, out=d), want)


@pytest.mark.parametrize("H", [515, 1027, 2051, 4099, 8195, 16387, 33283])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_whose_end_is_a_wavefronts_first_piece_in_place(dtype, H):
    # a wavefront may be done with its part of the row before another has read the end of it
    R = 600 if H < 16000 else 60
    x, res, w, g = inputs(R, H, dtype, H)
    dy, dx, dr = up(normal(g, R, H, dtype=dtype)), up(x), up(res)
    say(f"in place {R} x {H} {dtype}")
    y, s = moe.rms_norm(up(x), up(w), residual=dr)
    got, stream = moe.rms_norm(dx, up(w), residual=dr, residual_out=dx)
    assert torch.equal(got, y) and torch.equal(stream, s)
    want, dw = moe.rms_norm_backward(dy, s, up(w), dresidual=dr)
    for over in (0, 1, 2):
        t = [dy.clone(), s.clone(), dr.clone()]
        got, dwo = moe.rms_norm_backward(t[0], t[1], up(w), dresidual=t[2], out=t[over])
        assert torch.equal(got, want) and torch.equal(dwo, dw)
    d = s.clone()
    assert torch.equal(moe.rms_norm(d, up(w), out=d, out_dtype=dtype), moe.rms_norm(s, up(w), out_dtype=dtype))


def test_zero_infinite_and_large_rows():
    H = 264
    x = normal(gen(9), 6, H, dtype=F32)
    x[1], x[2, 5], x[3, 7], x[4] = 0, float("inf"), float("nan"), 1e20
    got = moe.rms_norm(up(x), out_dtype=F32).cpu()
    _, ref, _ = reference(x[[0, 1, 5]], None, None, 1e-6)
    near(got[[0, 1, 5]], ref, bar_y(H) * ref.abs(), "other rows")
    assert torch.isnan(got[2, 5]) and torch.isnan(got[3]).all() and (got[4] == 0).all()
    q, s = moe.rms_norm(up(x), quantize="mx_e4m3")
    assert (s[1] == 127).all() and (s[3] == 255).all() and (q[1].float() == 0).all() and torch.isnan(q[3].float()).all()
    q, s = moe.rms_norm(up(x), quantize="fp8")
    assert (s[1] == 1).all() and torch.isnan(s[3]).all() and torch.isnan(q[3].float()).all()


def test_no_rows_and_eps():
    x, _, w, _ = inputs(0, 64, BF, 1, residual=False)
    assert moe.rms_norm(up(x), up(w)).shape == (0, 64)
    dx, dw = moe.rms_norm_backward(up(x), up(x), up(w))
    assert dx.shape == (0, 64) and (dw == 0).all()
    a = moe.rms_norm(torch.full((1, 64), 2.0, device="cuda"), eps=12.0, out_dtype=F32)
    assert ((a - 0.5).abs() <= 8 * U).all()
    b = moe.rms_norm(torch.full((1, 64), 2.0, device="cuda"), eps=5.0, out_dtype=F32)   # the same sizes, another eps
    assert ((b - 2 / 3).abs() <= 8 * U).all()


# ---- gradients ---------------------------------------------------------------------

def gradients(dy, s, w, dres, eps):
    v, d = s.double(), dy.double()
    r = (v.square().mean(dim=1, keepdim=True) + eps).rsqrt()
    g = d * (1.0 if w is None else w.double())
    along = (g * v).mean(dim=1, keepdim=True)
    dx = r * (g - v * r * r * along)
    mag = r * (g.abs() + v.abs() * r * r * (g * v).abs().mean(dim=1, keepdim=True))
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    terms = d * v * r
    return dx, mag, terms.sum(dim=0), terms.abs().sum(dim=0)


def check_gradients(got, dy, s, w, dres, eps):
    R, H = s.shape
    dx, mag, dw, wmag = gradients(dy, s, w, dres, eps)
    near(got[0], dx, HALF[got[0].dtype] * 1.01 * dx.abs() + (2 * steps(H) + 16) * U * mag + 1e-37, "dx")
    if got[1] is not None:
        near(got[1], dw, ((R + 16) * U + bar_y(H)) * wmag + 1e-37, "dw")


@pytest.mark.parametrize("dy_dtype", [BF, F32], ids=["dy_bf16", "dy_fp32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,H", SIZES)
def test_rms_norm_backward_matches_64_bits(R, H, dtype, dy_dtype):
    s, dres, w, g = inputs(R, H, dtype, 2 * R + H, wdtype=[BF, F32, None][(R + H) % 3])
    dy = normal(g, R, H, std=0.3, dtype=dy_dtype)
    say(f"rms_norm_backward {R} x {H} {dtype} {dy_dtype}")
    args = up(dy), up(s), up(w)
    dweight = torch.full((H,), 7.0, device="cuda") if w is None else None   # asked for without a weight too
    got = moe.rms_norm_backward(*args, eps=1e-5, dresidual=up(dres), dweight=dweight)
    check_gradients(got, dy, s, w, dres, 1e-5)
    got = moe.rms_norm_backward(*args, eps=1e-5)
    assert (got[1] is None) == (w is None)
    check_gradients(got, dy, s, w, None, 1e-5)


@pytest.mark.parametrize("pad,lead", [(0, 1), (8, 8), (3, 0)])
def test_rms_norm_backward_strides_and_places(pad, lead):
    R, H = 70, 328
    s, dres, w, g = inputs(R, H, BF, 8)
    dy = normal(g, R, H)
    want = moe.rms_norm_backward(up(dy), up(s), up(w), dresidual=up(dres))
    t = [strided(v, pad, lead) for v in (dy, s, dres)]
    out = strided(torch.zeros(R, H, dtype=BF), pad, lead)
    got = moe.rms_norm_backward(t[0], t[1], strided(w[None], 0, lead)[0], dresidual=t[2], out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for i in range(3):   # written over dy, the stream or dresidual
        t = [up(v) for v in (dy, s, dres)]
        got = moe.rms_norm_backward(t[0], t[1], up(w), dresidual=t[2], out=t[i])
        assert got[0] is t[i] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H", [40, 1000, 8200, 33000])
def test_gradient_against_differences(H):
    R, eps = 12, 1e-5
    s, _, w, g = inputs(R, H, F32, H, residual=False, wdtype=F32)
    dy = normal(g, R, H, dtype=F32)
    f = lambda v, u: (v * (v.square().mean(dim=1, keepdim=True) + eps).rsqrt() * u * dy.double()).sum()   # noqa: E731
    dx, dw = moe.rms_norm_backward(up(dy), up(s), up(w), eps=eps)
    v, u = torch.randn(R, H, generator=g, dtype=torch.float64), torch.randn(H, generator=g, dtype=torch.float64)
    h = 1e-6
    num = (f(s.double() + h * v, w.double()) - f(s.double() - h * v, w.double())) / (2 * h)
    got = (dx.double().cpu() * v).sum()
    # dx is off by its bar, and the difference by rounding (2^-52 of f over h) and h^2
    _, mag, _, wmag = gradients(dy, s, w, None, eps)
    bar = ((2 * steps(H) + 17) * U * mag * v.abs()).sum() + 1e-7 * mag.sum()
    assert abs(got - num) <= bar
    num = (f(s.double(), w.double() + h * u) - f(s.double(), w.double() - h * u)) / (2 * h)
    assert abs((dw.double().cpu() * u).sum() - num) <= (((R + 17) * U + bar_y(H)) * wmag * u.abs()).sum() + 1e-7 * wmag.sum()


def test_weight_gradient_does_not_depend_on_timing():
    s, _, w, g = inputs(5000, 1032, BF, 12, residual=False)
    dy = normal(g, 5000, 1032)
    t = up(dy), up(s), up(w)
    want = moe.rms_norm_backward(*t)
    for _ in range(5):
        got = moe.rms_norm_backward(*t)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
