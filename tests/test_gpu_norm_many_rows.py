"""RMS norm and its gradients with several rows to a workgroup, for every shape in
which a row is held (one and two pieces a thread, 256, 512 and 1024 threads, rows
side by side, whole eights and not) and for rows past what is held. Each workgroup
then walks its rows with the next one on its way and its reduction buffers in turn,
which few rows never show. Against 64 bits, with test_gpu_norm's bars. And tensors
of more than 2^31 elements."""
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from test_gpu_norm import HALF, U, bar_y, check_gradients, gradients, inputs, near, reference, steps
from test_gpu_operators import BF, F32, gen, normal, say, up

pytestmark = pytest.mark.gpu

# rows, hidden: more than the largest grid takes at once, mostly twice or three times
MANY = [(70000, 64), (70001, 61), (20000, 500), (9001, 1000), (5000, 2048), (5001, 2047), (3300, 4096), (3301, 4095), (3100, 7168), (3101, 7167),
        (1600, 8200), (1601, 8199), (1100, 16384), (1200, 16500)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,H", MANY)
def test_forward(R, H, dtype):
    x, res, w, _ = inputs(R, H, dtype, R + H, wdtype=[BF, F32, None][(R + H) % 3])
    s, ref, _ = reference(x, w, res, 1e-5)
    dx, dw, dr = up(x), up(w), up(res)
    say(f"norm of many rows {R} x {H} {dtype}")
    got = {}
    for out_dtype in (BF, F32):
        got[out_dtype], stream = moe.rms_norm(dx, dw, residual=dr, eps=1e-5, out_dtype=out_dtype)
        assert torch.equal(stream.cpu(), s)
        near(got[out_dtype], ref, (HALF[out_dtype] * 1.01 + bar_y(H)) * ref.abs() + 1e-37, "y")
        assert torch.equal(moe.rms_norm(stream, dw, eps=1e-5, out_dtype=out_dtype), got[out_dtype])   # without a residual
    for quantize in ("fp8", "mx_e4m3", "mx_e2m1"):
        q, scales, s2 = moe.rms_norm(dx, dw, residual=dr, eps=1e-5, quantize=quantize)
        wq, ws = moe.quantize_fp8(got[F32]) if quantize == "fp8" else moe.quantize_mx(got[F32], quantize[3:])
        assert torch.equal(s2, stream)
        assert torch.equal(q.contiguous().view(torch.uint8), wq.contiguous().view(torch.uint8)) and torch.equal(scales.contiguous(), ws.contiguous())
    over, same = moe.rms_norm(dx, dw, residual=dr, eps=1e-5, residual_out=dx)   # written over x
    assert same is dx and torch.equal(dx, stream) and torch.equal(over, got[BF])


@pytest.mark.parametrize("dy_dtype", [BF, F32], ids=["dy_bf16", "dy_fp32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("R,H", MANY)
def test_backward(R, H, dtype, dy_dtype):
    s, dres, w, g = inputs(R, H, dtype, 2 * R + H, wdtype=[BF, F32][(R + H) % 2])
    dy = normal(g, R, H, std=0.3, dtype=dy_dtype)
    say(f"gradients of many rows {R} x {H} {dtype} {dy_dtype}")
    t = up(dy), up(s), up(w), up(dres)
    got = moe.rms_norm_backward(*t[:3], eps=1e-5, dresidual=t[3])
    check_gradients(got, dy, s, w, dres, 1e-5)
    plain = moe.rms_norm_backward(*t[:3], eps=1e-5)
    assert torch.equal(plain[1], got[1])   # dw knows no dresidual
    over = moe.rms_norm_backward(*t[:3], eps=1e-5, dresidual=t[3], out=t[3])
    assert over[0] is t[3] and torch.equal(over[0], got[0]) and torch.equal(over[1], got[1])
    over = moe.rms_norm_backward(*t[:3], eps=1e-5, out=t[1])   # over the stream
    assert torch.equal(over[0], plain[0]) and torch.equal(over[1], got[1])


# ---- past 2^31 elements -------------------------------------------------------------------

@pytest.fixture
def memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R,H", [(300_000, 7168), (140_000, 16_392)], ids=["held", "two_passes"])
def test_past_2_31_elements(memory, R, H):
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)   # noqa: E731
    x, w = randn(R, H), randn(H)
    # rows of both ends and around the 2^31st element
    mid = 2 ** 31 // H
    at = torch.cat([torch.arange(40), torch.arange(mid - 20, mid + 20), torch.arange(R - 40, R)])
    rows, wc = x[at.cuda()].cpu(), w.cpu()
    say(f"large norm {R} x {H}")
    y = moe.rms_norm(x, w)
    _, ref, _ = reference(rows, wc, None, 1e-6)
    near(y[at.cuda()], ref, (HALF[BF] * 1.01 + bar_y(H)) * ref.abs(), "rows")
    q, sc = moe.rms_norm(x, w, quantize="mx_e4m3")
    for r in (at[:40], at[40:80], at[80:]):   # the same rows in a tensor of their own, of the same kernel's shape
        part = torch.cat([x[r.cuda()], x[:600]])
        wq, ws = moe.rms_norm(part, w, quantize="mx_e4m3")
        assert torch.equal(q.view(torch.uint8)[r.cuda()], wq.view(torch.uint8)[:len(r)]) and torch.equal(sc[r.cuda()], ws[:len(r)])
    del q, sc
    say(f"large norm's gradients {R} x {H}")
    y.zero_()   # dy: zeros but for these rows, whose weight gradient is the whole one
    dyr = normal(gen(3), len(at), H)
    y[at.cuda()] = dyr.cuda()
    dx, dw = moe.rms_norm_backward(y, x, w, dresidual=x, out=y)
    ref, mag, refw, wmag = gradients(dyr, rows, wc, rows, 1e-6)
    near(dx[at.cuda()], ref, HALF[BF] * 1.01 * ref.abs() + (2 * steps(H) + 16) * U * mag, "dx")
    near(dw, refw, ((len(at) + 16) * U + bar_y(H)) * wmag + 1e-37, "dw")   # zeros add nothing and round nothing
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[at.cuda()] = False
    for n in range(0, R, 20000):   # a row without a gradient of its own passes dresidual on
        part = slice(n, n + 20000)
        assert torch.equal(dx[part][rest[part]], x[part][rest[part]])
