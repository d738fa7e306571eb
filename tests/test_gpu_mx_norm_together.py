"""RMS norm, MX quantisation and products, and the weighted combination as one
layer uses them -- serving in MX formats, and a training step -- against 64 bits,
as eager calls and captured and replayed; on several streams; on tensors past
4 GiB; and what the outputs' versions and the checks of known sizes say."""
import numpy as np
import pytest
import torch

import moe_expert_ffn_persistent_amd as moe
from moe_expert_ffn_persistent_amd import _lib
from oracle import moe_oracle as mo
from test_gpu_mx import operand, values
from test_gpu_norm import U, bar_y, gradients, near, reference, steps
from test_gpu_operators import BF, DROP, F32, F8, HALF, assert_close, gen, normal, offsets, say, up

pytestmark = pytest.mark.gpu


def zeros(*s, dt=BF):
    return torch.zeros(*s, dtype=dt, device="cuda")


def captured(step):
    """A graph of step, after torch's recipe"""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        step()
    return cg


def replays(step, fill, outs, rows, what):
    """Three replays with other inputs and eager work between, each bitwise as the eager calls; rows(): how many rows a per-row output has."""
    fill(1)
    cg = captured(step)
    for r in range(3):
        fill(10 + r)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.view(torch.uint8).fill_(0x3C)
        (want[-1].float() + 1).sum().item()
        say(f"{what}, replay {r}")
        cg.replay()
        torch.cuda.synchronize()
        n, cap = rows()
        for t, v in zip(outs, want):
            keep = n if len(t) == cap else len(t)
            assert torch.equal(t[:keep].contiguous().view(torch.uint8), v[:keep].contiguous().view(torch.uint8))


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("element", ["e4m3", "e2m1"])
def test_mx_layer(element, graph):
    S, T, E, k, L, H, I = 2, 40, 16, 4, 5, 512, 288
    N, cap, g = S * T, S * T * k, gen(9)
    w1, s1, v1 = operand(g, "e2m1", L, 2 * I, H)
    w2, s2, v2 = operand(g, "e2m1", L, H, I)
    # weights as a trained layer's: their products of the size of what goes in
    s1, s2, v1, v2 = s1 - 5, s2 - 4, v1 / 32, v2 / 16
    wn = up((1 + 0.2 * torch.randn(H, generator=g)).to(BF))
    x, res, logits = zeros(N, H), zeros(N, H), zeros(N, E, dt=F32)
    ffn = moe.MoeExpertFFN(S, T, E, k, 0, L, H, 128)
    codes = lambda r, c: zeros(r, c, dt=F8) if element == "e4m3" else zeros(r, c // 2, dt=torch.uint8)   # noqa: E731
    sc = lambda r, c: zeros(r, c // 32, dt=torch.uint8)   # noqa: E731
    qx, sx, qr, sr, qh, sh = codes(N, H), sc(N, H), codes(cap, H), sc(cap, H), codes(cap, I), sc(cap, I)
    stream, a, h, yr, y = zeros(N, H), zeros(cap, 2 * I), zeros(cap, I), zeros(cap, H), zeros(N, H)

    def step():
        lay = ffn.layout(logits=logits)
        off = lay.row_offset
        moe.rms_norm(x, wn, residual=res, quantize="mx_" + element, out=qx, scales=sx, residual_out=stream)
        moe.dispatch_rows(qx, lay.row_pair, off, k, out=qr)
        moe.dispatch_rows(sx, lay.row_pair, off, k, out=sr)
        moe.mx_matmul(qr, sr, w1, s1, row_offset=off, out=a, expected_rows=cap * L // E)
        moe.swiglu(a, row_offset=off, out=h)
        moe.quantize_mx(h, element, row_offset=off, out=qh, scales=sh)
        moe.mx_matmul(qh, sh, w2, s2, row_offset=off, out=yr, expected_rows=cap * L // E)
        moe.combine_rows(yr, lay.pair_row, k, out=y, weights=lay.topk_w)
        return lay

    def fill(seed):
        x.copy_(torch.randn(N, H, generator=gen(seed)))
        res.copy_(torch.randn(N, H, generator=gen(seed + 2)) * 2)
        logits.copy_(torch.randn(N, E, generator=gen(seed + 1)))

    if graph:
        rows = lambda: (int(ffn.layout(logits=logits).row_offset[-1]), cap)   # noqa: E731
        replays(step, fill, [qx, sx, stream, qr, sr, a, h, qh, sh, yr, y], rows, f"mx layer {element}")
        return
    fill(1)
    say(f"mx layer {element}")
    lay = step()
    torch.cuda.synchronize()
    off, pair, R = lay.row_offset.cpu(), lay.row_pair.cpu().long(), int(lay.row_offset[-1])
    assert 0 < R < cap
    tok = (pair[:R] // k).cuda()
    assert torch.equal(qr[:R].view(torch.uint8), qx[tok].view(torch.uint8)) and torch.equal(sr[:R], sx[tok])
    # the norm's codes are those of quantize_mx of its fp32 output
    assert torch.equal(stream, (x.float() + res.float()).to(BF))
    q, s = moe.quantize_mx(moe.rms_norm(stream, wn, out_dtype=F32), element)
    assert torch.equal(q.view(torch.uint8), qx.view(torch.uint8)) and torch.equal(s, sx)
    val = lambda c, s_, cols: torch.from_numpy(np.ascontiguousarray(values(c, element, cols))) * \
        torch.from_numpy(mo.e8m0_to_f64(s_.cpu().numpy())).repeat_interleave(32, dim=1)   # noqa: E731, E127

    def product(xv, wv):
        out, mag = torch.zeros(R, wv.shape[1], dtype=torch.float64), torch.zeros(R, wv.shape[1], dtype=torch.float64)
        for e in range(L):
            r = slice(int(off[e]), int(off[e + 1]))
            out[r], mag[r] = xv[r] @ wv[e].t(), xv[r].abs() @ wv[e].abs().t()
        return out, mag

    ref, mag = product(val(qr[:R], sr[:R], H), v1)
    assert_close(a[:R], ref, BF, mag, H, "first product", DROP)
    q, s = moe.quantize_mx(h[:R].contiguous(), element)
    assert torch.equal(q.view(torch.uint8), qh[:R].view(torch.uint8)) and torch.equal(s, sh[:R])
    ref, mag = product(val(qh[:R], sh[:R], I), v2)
    assert_close(yr[:R], ref, BF, mag, I, "second product", DROP)
    # the whole layer against the unquantised one: a value within the codes' range is
    # off by half a step (2^-4, 2^-2), one that a scale rounded down leaves above it by
    # 1/8 (448 of 512) or 1/4 (6 of 8) at most; x and h each, over hundreds of terms
    v = stream.double().cpu()
    n = v * (v.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * wn.double().cpu()
    ad, _ = product(n[pair[:R] // k], v1)
    rows, _ = product(torch.nn.functional.silu(ad[:, :I]) * ad[:, I:], v2)
    full = torch.zeros(N, H, dtype=torch.float64).index_add(0, pair[:R] // k, rows * lay.topk_w.cpu().double().view(-1)[pair[:R], None])
    err = (y.double().cpu() - full).norm() / full.norm()
    say(f"mx layer {element}: {err:.3f} of the unquantised one")
    assert err <= (2 * 2.0 ** -3 if element == "e4m3" else 2 * 2.0 ** -2)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_training_step(graph):
    """The residual stream's addition and norm, rows to the experts, their products
    with SwiGLU between, the router's weights, and every gradient."""
    S, T, E, k, L, H, I = 2, 30, 8, 3, 4, 264, 128
    N, cap, g = S * T, S * T * k, gen(78)
    w1, w2 = up(normal(g, L, 2 * I, H, std=0.06)), up(normal(g, L, H, I, std=0.06))
    wn = up((1 + 0.2 * torch.randn(H, generator=g)).float())
    x, res, dy, ds, logits = zeros(N, H), zeros(N, H), zeros(N, H), zeros(N, H), zeros(N, E, dt=F32)
    ffn = moe.MoeExpertFFN(S, T, E, k, 0, L, 256, 128)
    b = dict(s=zeros(N, H), n=zeros(N, H), xr=zeros(cap, H), a=zeros(cap, 2 * I), h=zeros(cap, I), yr=zeros(cap, H), y=zeros(N, H, dt=F32),
             dyr=zeros(cap, H), dwt=zeros(N, k, dt=F32), dh=zeros(cap, I), da=zeros(cap, 2 * I), dxr=zeros(cap, H), dn=zeros(N, H, dt=F32),
             dx=zeros(N, H), dwn=zeros(H, dt=F32), dw1=zeros(L, 2 * I, H, dt=F32), dw2=zeros(L, H, I, dt=F32))

    def step():
        lay = ffn.layout(logits=logits)
        off = lay.row_offset
        moe.rms_norm(x, wn, residual=res, out=b["n"], residual_out=b["s"])
        moe.dispatch_rows(b["n"], lay.row_pair, off, k, out=b["xr"])
        moe.grouped_matmul(b["xr"], w1, off, out=b["a"])
        moe.swiglu(b["a"], row_offset=off, out=b["h"])
        moe.grouped_matmul(b["h"], w2, off, out=b["yr"])
        moe.combine_rows(b["yr"], lay.pair_row, k, out=b["y"], weights=lay.topk_w)
        moe.combine_rows_backward(dy, b["yr"], lay.pair_row, lay.topk_w, out=b["dyr"], dweights=b["dwt"])
        moe.grouped_matmul_dgrad(b["dyr"], w2, off, out=b["dh"])
        moe.grouped_matmul_wgrad(b["dyr"], b["h"], off, out=b["dw2"])
        moe.swiglu_backward(b["a"], b["dh"], row_offset=off, out=b["da"])
        moe.grouped_matmul_dgrad(b["da"], w1, off, out=b["dxr"])
        moe.grouped_matmul_wgrad(b["da"], b["xr"], off, out=b["dw1"])
        moe.combine_rows(b["dxr"], lay.pair_row, k, out=b["dn"])
        moe.rms_norm_backward(b["dn"], b["s"], wn, dresidual=ds, out=b["dx"], dweight=b["dwn"])
        return lay

    def fill(seed):
        for i, t in enumerate((x, res, dy, ds, logits)):
            t.copy_(torch.randn(t.shape, generator=gen(seed + 100 * i)))

    if graph:
        rows = lambda: (int(ffn.layout(logits=logits).row_offset[-1]), cap)   # noqa: E731
        replays(step, fill, list(b.values()), rows, "training step")
        return
    fill(1)
    say("training step")
    lay = step()
    torch.cuda.synchronize()
    R, off = int(lay.row_offset[-1]), lay.row_offset.cpu().tolist()
    pair = lay.row_pair.cpu().long()[:R]
    c = lambda t: t.double().cpu()   # noqa: E731
    dyd, dsd = c(dy), c(ds)

    def loss(s_, wn_, w1_, w2_, wt_):
        n = s_ * (s_.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * wn_
        rows, parts = n[pair // k], []
        for e in range(L):
            r = slice(off[e], off[e + 1])
            a = rows[r] @ w1_[e].t()
            parts.append((torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ w2_[e].t())
        y = torch.zeros(N, H, dtype=torch.float64).index_add(0, pair // k, torch.cat(parts) * wt_.reshape(-1)[pair, None])
        return y, (y * dyd).sum() + (s_ * dsd).sum()

    args = [c(t).requires_grad_() for t in (b["s"], wn, w1, w2, lay.topk_w)]
    y, total = loss(*args)
    total.backward()
    # the norm's output, a, h, the expert rows, dy rows, dh, da and dx rows are each
    # rounded to bf16 on the way: up to six roundings of 2^-8 stand behind an entry
    # of a gradient, in sums of independent errors; the bar is six whole ones of the norm
    bar = 6 * 2.0 ** -8
    grads = dict(zip(("dx", "dwn", "dw1", "dw2", "dwt"), (t.grad for t in args)))
    for n, ref in (("y", y.detach()), *grads.items()):
        err = (c(b[n]) - ref).norm() / ref.norm()
        say(f"training step {n}: {err:.2e}")
        assert err <= bar, n
    # and against differences of the 64-bit function, along one direction of each input
    with torch.no_grad():
        for i, n in enumerate(grads):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            move = lambda t: loss(*[a + t * v if j == i else a for j, a in enumerate(args)])[1]   # noqa: E731, B023
            num = (move(1e-6) - move(-1e-6)) / 2e-6
            # 4 standard deviations of an error along v
            assert abs((c(b[n]) * v).sum() - num) <= bar * grads[n].norm() * 4 + 1e-6, n


def operators():
    """name: (call(stream), tensors read, tensors written)"""
    g = gen(3)
    R, H, n = 24, 96, 40
    x, res, w, dy = (up(normal(g, *s)) for s in ((R, H), (R, H), (H,), (R, H)))
    off = up(offsets([10, 14]))
    qx, sx = moe.quantize_mx(x)
    x4, s4 = moe.quantize_mx(x, "e2m1")
    qw, sw = moe.quantize_mx(up(normal(g, 2, n, H)), "e2m1")
    at, wt = up(torch.arange(R, dtype=torch.int32)), up(torch.rand(R // 2, 2, generator=g))
    y, s, q, qs = zeros(R, H), zeros(R, H), zeros(R, H, dt=F8), zeros(R, H // 32, dt=torch.uint8)
    q4, f8s, dw, out, tok, dwt = zeros(R, H // 2, dt=torch.uint8), zeros(R, 1, dt=F32), zeros(H, dt=F32), zeros(R, n), zeros(R // 2, H), zeros(R // 2, 2, dt=F32)
    norm = lambda q_, o, sc: lambda st: moe.rms_norm(x, w, residual=res, quantize=q_, out=o, scales=sc, residual_out=s, stream=st)   # noqa: E731
    return {
        "rms_norm": (norm(None, y, None), (x, w, res), (y, s)),
        "rms_norm_fp8": (norm("fp8", q, f8s), (x, w, res), (q, f8s, s)),
        "rms_norm_mx_e4m3": (norm("mx_e4m3", q, qs), (x, w, res), (q, qs, s)),
        "rms_norm_mx_e2m1": (norm("mx_e2m1", q4, qs), (x, w, res), (q4, qs, s)),
        "rms_norm_backward": (lambda st: moe.rms_norm_backward(dy, x, w, dresidual=res, out=y, dweight=dw, stream=st), (dy, x, w, res), (y, dw)),
        "quantize_mx": (lambda st: moe.quantize_mx(x, out=q, scales=qs, stream=st), (x,), (q, qs)),
        "quantize_mx_experts": (lambda st: moe.quantize_mx(x, "e2m1", row_offset=off, out=q4, scales=qs, stream=st), (x, off), (q4, qs)),
        "mx_matmul": (lambda st: moe.mx_matmul(qx, sx, qw, sw, row_offset=off, out=out, stream=st), (qx, sx, qw, sw, off), (out,)),
        "mx_matmul_e2m1_in_ranges": (lambda st: moe.mx_matmul(x4, s4, qw, sw, row_offset=off, out=out, splits=2, stream=st), (x4, s4, qw, sw, off), (out,)),
        "combine_rows": (lambda st: moe.combine_rows(x, at, 2, out=tok, weights=wt, stream=st), (x, at, wt), (tok,)),
        "combine_rows_backward": (lambda st: moe.combine_rows_backward(dy[:R // 2], x, at, wt, out=y, dweights=dwt, stream=st), (dy, x, at, wt), (y, dwt)),
    }


NAMES = ["rms_norm", "rms_norm_fp8", "rms_norm_mx_e4m3", "rms_norm_mx_e2m1", "rms_norm_backward", "quantize_mx", "quantize_mx_experts", "mx_matmul",
         "mx_matmul_e2m1_in_ranges", "combine_rows", "combine_rows_backward"]


@pytest.mark.parametrize("stream", ["current", "other"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_get_a_new_version_and_inputs_keep_theirs(name, stream):
    call, read, written = operators()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):   # the first call of these sizes, and calls of sizes seen before
        before = [t._version for t in read], [t._version for t in written]
        call(side if stream == "other" else None)
        assert [t._version for t in read] == before[0]
        assert all(t._version > v for t, v in zip(written, before[1]))
    torch.cuda.synchronize()


def test_two_streams_at_once():
    g = gen(16)
    R, H, n = 700, 1024, 520
    x, w, dy = up(normal(g, R, H)), up(normal(g, H)), up(normal(g, R, H))
    qw, sw = moe.quantize_mx(up(normal(g, 3, n, H)), "e2m1")
    off = up(offsets([300, 150, 250]))
    qx, sx = moe.rms_norm(x, w, quantize="mx_e4m3")
    calls = [lambda s: moe.rms_norm_backward(dy, x, w, stream=s), lambda s: (moe.mx_matmul(qx, sx, qw, sw, row_offset=off, splits=3, stream=s),),
             lambda s: moe.rms_norm(x, w, quantize="fp8", stream=s), lambda s: moe.quantize_mx(x, "e2m1", stream=s)]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[f(s) for f, s in zip(calls, streams[i % 2:] + streams[:i % 2])] for i in range(8)]
    torch.cuda.synchronize()
    for turn in got:
        for a, b in zip(turn, want):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_checks_hold_for_sizes_seen_before():
    ops = operators()
    for name in NAMES:
        ops[name][0](None)
    R, H = 24, 96
    x, w, y, s = zeros(R, H), zeros(H), zeros(R, H), zeros(R, H)
    for _ in range(2):
        moe.rms_norm(x, w, residual=s, out=y, residual_out=s)
    for bad in (dict(weight=w.cpu()), dict(weight=w[:-1]), dict(residual=s.float()), dict(residual=s.clone().requires_grad_()), dict(out=y.t()),
                dict(out=y.cpu()), dict(residual_out=y.int())):
        with pytest.raises(ValueError):
            moe.rms_norm(**{**dict(x=x, weight=w, residual=s, out=y, residual_out=s), **bad})
    q, qs = moe.quantize_mx(x)
    qw, sw = moe.quantize_mx(zeros(40, H), "e2m1")
    out = moe.mx_matmul(q, qs, qw, sw)
    for bad in (dict(x_scales=qs.float()), dict(w=q), dict(w_scales=sw[:-1]), dict(out=out.cpu()), dict(x=q.clone().view(torch.uint8)), dict(out=out.half())):
        with pytest.raises(ValueError):
            moe.mx_matmul(**{**dict(x=q, x_scales=qs, w=qw, w_scales=sw, out=out), **bad})
    with pytest.raises(_lib.MoeError):
        moe.mx_matmul(q, qs, qw, sw, out=out, tile=99)
    with pytest.raises(ValueError):
        moe.quantize_mx(x, out=q, scales=qs[:, :-1])


# ---- past 4 GiB and 2^31 elements ---------------------------------------------------------

@pytest.fixture
def memory():
    yield
    torch.cuda.empty_cache()


def randn(*shape, dtype=BF, seed=1):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=dtype)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_norm_past_4_gib(memory):
    R, H = 140_000, 16_392   # 4.6 GB of bf16, of codes 2.3
    x, w = randn(R, H), randn(H)
    last = slice(R - 70, R)
    tail = x[last].clone()
    say("large norm")
    y, s = moe.rms_norm(x, w, residual=x)
    assert same(s[last], (2 * tail.float()).to(BF))
    _, ref, _ = reference(s[last].cpu(), w.cpu(), None, 1e-6)
    near(y[last], ref, (HALF[BF] * 1.01 + bar_y(H)) * ref.abs(), "last rows")
    say("large norm, MX")
    q, sc = moe.rms_norm(x, w, quantize="mx_e4m3")
    tq, tsc = moe.quantize_mx(moe.rms_norm(tail, w, out_dtype=F32))
    # sums of another order: off by 2^-15 at most, against borders 2^-4 apart
    assert (q[last].view(torch.uint8) != tq.view(torch.uint8)).float().mean() <= 2e-3 and (sc[last] != tsc).float().mean() <= 2e-3
    say("large norm's gradients")
    ty = y[last].clone()
    dx, dw = moe.rms_norm_backward(y, x, w, dresidual=x, out=y)
    ref, mag, _, _ = gradients(ty.cpu(), tail.cpu(), w.cpu(), tail.cpu(), 1e-6)
    near(dx[last], ref, HALF[BF] * 1.01 * ref.abs() + (2 * steps(H) + 16) * U * mag, "last rows' gradients")
    assert torch.isfinite(dw).all()


def test_mx_past_4_gib(memory):
    R, K, n = 140_000, 32_768, 72   # values: 9.2 GB, codes 4.6
    x = randn(R, K)
    last = slice(R - 70, R)
    tail = x[last].clone()
    say("large quantize_mx")
    q, sc = moe.quantize_mx(x)
    tq, tsc = moe.quantize_mx(tail)
    assert same(q[last], tq) and same(sc[last], tsc)
    del x
    w, ws = moe.quantize_mx(randn(n, K), "e2m1")
    want = moe.mx_matmul(tq, tsc, w, ws, tile=1, splits=1)
    for tile in (0, 1, 5, 8, 9):
        say(f"large mx product, tile {tile}")
        y = moe.mx_matmul(q, sc, w, ws, tile=tile, splits=1 if tile else 0)
        d = (y[last].float() - want.float()).abs().max() / want.float().abs().max()
        assert d <= 2.0 ** -7, tile   # another order of the sums and one rounding each
    del q, y
    L, rows = 90, 3200   # weights: 4.7 GB
    w, ws = moe.quantize_mx(randn(L, rows, K), "e2m1")
    off = up(offsets([0] * (L - 1) + [20]))
    want = moe.mx_matmul(tq[:20], tsc[:20], w[-1].clone(), ws[-1].clone())
    for pad in (0, 1):   # the last expert's, read by the tile kernels and by the one of any alignment
        say(f"large mx weights {pad}")
        xb = torch.zeros(20, K + 16 + pad, dtype=torch.uint8, device="cuda")[:, :K]
        xb.copy_(tq[:20].view(torch.uint8))
        y = moe.mx_matmul(xb.view(F8), tsc[:20], w, ws, row_offset=off)
        d = (y.float() - want.float()).abs().max() / want.float().abs().max()
        assert d <= 2.0 ** -7


def test_weighted_combine_past_4_gib(memory):
    R, H, k = 140_000, 16_392, 2
    rows, N = randn(R, H), R // k
    at = torch.arange(R, dtype=torch.int32, device="cuda").flip(0).contiguous()
    wt = torch.rand(N, k, device="cuda")
    say("large weighted combine")
    y = moe.combine_rows(rows, at, k, weights=wt)
    few = slice(0, 50)   # the first tokens own the last rows
    tail = rows[R - 100:].clone()
    tat = torch.arange(100, dtype=torch.int32, device="cuda").flip(0).contiguous()
    assert same(y[few], moe.combine_rows(tail, tat, k, weights=wt[few].contiguous()))
    say("large weighted combine's gradients")
    d, dw = moe.combine_rows_backward(y, rows, at, wt)
    td, tdw = moe.combine_rows_backward(y[few].contiguous(), tail, tat, wt[few].contiguous())
    mag = (y[few].double()[:, None] * rows[at[:100].long()].double().view(50, k, H)).abs().sum(dim=2)
    assert same(d[R - 100:], td) and ((dw[few] - tdw).abs() <= 2 * (-(-H // 64) + 24) * U * mag).all()
