"""The operators before, within and behind an expert layer in microscaled formats, as a user's program calls them: the
RMS norm of the residual stream with the stream's addition and an output in 8 or 4 bits, forward and backward;
quantisation to the OCP Microscaling (MX) formats; the product of MX operands, dense and grouped by expert; and each
token's rows combined with its router weights, forward and backward.

`own` false: each operator in plain torch operations in 32 bits. `own` true: the framework's kernels."""
import math
import random

import torch

own = False

MX = 32     # elements of one power-of-two scale
FP8 = 128   # elements of one fp32 scale
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the norm before the experts of a decode batch, written in the fp8 format (e4m3, fp32 scales)
        {"name": "norm_decode_fp8", "op": "norm", "form": "forward", "rows": 128, "hidden": 7168, "type": "bf16", "residual": True, "out": "fp8"},
        # a prefill batch's, written as MX e4m3 for 4-bit weights
        {"name": "norm_prefill_mx", "op": "norm", "form": "forward", "rows": 8192, "hidden": 7168, "type": "bf16", "residual": True, "out": "mx_e4m3"},
        # a training step's norm, forward and backward, with the gradient that passes it by
        {"name": "norm_train", "op": "norm", "form": "train", "rows": 16384, "hidden": 7168, "type": "bf16", "residual": True, "out": "bf16"},
        # an odd-sized layer's with the residual stream in fp32
        {"name": "norm_odd_train", "op": "norm", "form": "train", "rows": 1777, "hidden": 1000, "type": "fp32", "residual": True, "out": "bf16"},
        # activations of a decode batch to MX e4m3
        {"name": "mx_quantize_decode", "op": "quantize", "rows": 128, "cols": 2048, "type": "bf16"},
        # the routed rows of a prefill batch to MX e4m3
        {"name": "mx_quantize_prefill", "op": "quantize", "rows": 32768, "cols": 7168, "type": "bf16"},
        # one token through a dense layer with 4-bit weights
        {"name": "mx_token", "op": "product", "experts": 0, "rows": 1, "k": 7168, "n": 4096, "x": "e4m3", "skew": 0.0, "empty": 0},
        # a decode batch's rows through 4-bit experts: few rows, the weights read once
        {"name": "mx_decode", "op": "product", "experts": 32, "rows": 128, "k": 7168, "n": 4096, "x": "e4m3", "skew": 0.3, "empty": 1},
        # a prefill batch through a dense layer with 4-bit weights
        {"name": "mx_prefill", "op": "product", "experts": 0, "rows": 8192, "k": 7168, "n": 4096, "x": "e4m3", "skew": 0.0, "empty": 0},
        # the experts' second product over ragged rows, activations quantised to four bits on the way
        {"name": "mx_grouped_4bit", "op": "product", "experts": 32, "rows": 16384, "k": 2048, "n": 7168, "x": "e2m1", "skew": 0.3, "empty": 1},
        # a decode batch's rows back from one GPU's experts with the router's weights
        {"name": "combine_decode", "op": "combine", "form": "forward", "tokens": 128, "top_k": 8, "experts": 128, "local": 16, "hidden": 4096},
        # a training step's, with the gradients of the rows and of the router's weights
        {"name": "combine_train", "op": "combine", "form": "train", "tokens": 16384, "top_k": 8, "experts": 256, "local": 32, "hidden": 7168},
    ]


def _size(rng, lo, hi, step=1):
    """A size of lo..hi, even over its logarithm, a multiple of `step`."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "quantize", "product", "product", "product", "combine", "combine"])
    if op == "norm":
        train = rng.random() < 0.5
        kind = rng.choice(["bf16", "bf16", "fp32"])
        c = {"op": op, "form": "train" if train else "forward", "rows": _size(rng, 1, 16384),
             "hidden": _size(rng, 64, 7168, rng.choice([1, 8, 8])), "type": kind, "residual": rng.random() < 0.7,
             "out": "bf16" if train else rng.choice(["bf16", "fp8", "mx_e4m3"])}
        if kind == "fp32":
            c["rows"] = max(1, c["rows"] // 2)
        return c
    if op == "quantize":
        return {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 64, 7168, rng.choice([1, 8, 8])), "type": rng.choice(["bf16", "fp32"])}
    if op == "product":
        experts = 0 if rng.random() < 0.5 else _size(rng, 1, 32)
        c = {"op": op, "experts": experts, "rows": _size(rng, 1, 16384), "k": _size(rng, 128, 7168, rng.choice([2, 32, 32])),
             "n": _size(rng, 64, 7168, 8), "x": rng.choice(["e4m3", "e2m1"]), "skew": rng.choice([0.0, 0.3, 0.6]) if experts else 0.0,
             "empty": rng.randrange(0, experts // 4 + 1)}
        while max(1, experts) * c["k"] * c["n"] > 32 * 7168 * 4096 or c["rows"] * c["k"] * c["n"] > 8192 * 7168 * 4096:
            c["n"] = max(64, c["n"] // 16 * 8)
            if c["n"] == 64:
                break
        return c
    top_k, experts = rng.randrange(1, 9), rng.choice([8, 16, 32, 64, 128, 256])
    return {"op": op, "form": rng.choice(["forward", "train"]), "tokens": _size(rng, 1, 16384), "top_k": top_k, "experts": experts,
            "local": max(1, experts // rng.choice([1, 2, 4, 8])) if top_k < 3 else max(1, experts // 8),
            "hidden": _size(rng, 64, 7168, rng.choice([1, 8, 8]))}


def _counts(case, seed):
    """Rows of each expert: drawn with weights exp(skew * normal), `empty` experts without any."""
    rng = random.Random(seed * 7919 + 17)
    experts, empty = max(1, case["experts"]), case["empty"]
    weight = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(experts)]
    for e in rng.sample(range(experts), min(empty, experts - 1)):
        weight[e] = 0.0
    counts = [0] * experts
    for e in rng.choices(range(experts), weight, k=case["rows"]):
        counts[e] += 1
    return counts


def _work_counts(case):
    """Experts with a row, as drawn on average: each is read once."""
    experts = max(1, case["experts"]) - case["empty"]
    return experts * (1.0 - (1.0 - 1.0 / experts) ** case["rows"])


def _rows(shape, dtype, step, dev):
    """An uninitialised tensor whose rows start `step` elements apart or a multiple of that, as the framework lays out MX operands."""
    return torch.empty(*shape[:-1], -(-shape[-1] // step) * step, dtype=dtype, device=dev)[..., :shape[-1]]


def _mx_buffers(rows, cols, element, dev):
    """Codes (rows of whole 16 bytes apart) and scale bytes (of whole four)."""
    codes = _rows((rows, cols), torch.float8_e4m3fn, 16, dev) if element == "e4m3" else _rows((rows, -(-cols // 2)), torch.uint8, 16, dev)
    return codes, _rows((rows, -(-cols // MX)), torch.uint8, 4, dev)


def prepare(case, seed):
    dev, op = torch.device("cuda"), case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *shape, std=1.0, dtype=torch.bfloat16: torch.randn(shape, generator=gen, device=dev, dtype=dtype).mul_(std)  # noqa: E731
    s = {"case": case}
    if op == "norm":
        R, H, dtype = case["rows"], case["hidden"], torch.float32 if case["type"] == "fp32" else torch.bfloat16
        s["x"] = normal(R, H, dtype=dtype)
        # rows of different sizes: the stream grows along the layers
        s["residual"] = normal(R, H, std=2.0, dtype=dtype).mul_(torch.exp(0.5 * normal(R, 1, dtype=torch.float32)).to(dtype)) if case["residual"] else None
        s["stream"] = torch.empty(R, H, dtype=dtype, device=dev) if case["residual"] else None
        s["weight"] = 1.0 + normal(H, std=0.1)
        if case["out"] == "fp8":
            s["y"], s["scales"] = torch.empty(R, H, dtype=torch.float8_e4m3fn, device=dev), torch.empty(R, -(-H // FP8), dtype=torch.float32, device=dev)
        elif case["out"] == "bf16":
            s["y"], s["scales"] = torch.empty(R, H, dtype=torch.bfloat16, device=dev), None
        else:
            s["y"], s["scales"] = _mx_buffers(R, H, case["out"][3:], dev)
        if case["form"] == "train":
            s["dy"] = normal(R, H, std=0.1)
            s["dstream"] = normal(R, H, std=0.1, dtype=dtype) if case["residual"] else None
            s["dx"], s["dweight"] = torch.empty(R, H, dtype=dtype, device=dev), torch.empty(H, dtype=torch.float32, device=dev)
    elif op == "quantize":
        R, C = case["rows"], case["cols"]
        s["x"] = normal(R, C, dtype=torch.float32 if case["type"] == "fp32" else torch.bfloat16)
        s["x"] *= torch.exp(normal(R, 1, dtype=torch.float32)).to(s["x"].dtype)  # rows of different sizes
        s["q"], s["scales"] = _mx_buffers(R, C, "e4m3", dev)
    elif op == "product":
        L, R, K, N = max(1, case["experts"]), case["rows"], case["k"], case["n"]
        counts = _counts(case, seed)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        s["row_offset"] = torch.tensor(offsets, dtype=torch.int32, device=dev) if case["experts"] else None
        s["most"] = max(counts)  # rows of the largest expert, known where its buffers were sized
        s["w"], s["ws"] = _rows((L, N, K // 2), torch.uint8, 16, dev), _rows((L, N, -(-K // MX)), torch.uint8, 4, dev)
        for e in range(L):
            q, scales = _mx(normal(N, K, std=0.02, dtype=torch.float32), "e2m1")
            s["w"][e], s["ws"][e] = _packed(q), scales
        if not case["experts"]:
            s["w"], s["ws"] = s["w"][0], s["ws"][0]
        x = normal(R, K, dtype=torch.float32).mul_(torch.exp(normal(R, 1, dtype=torch.float32)))
        s["x"], s["xs"] = _mx_buffers(R, K, case["x"], dev)
        if case["x"] == "e4m3":
            q, scales = _mx(x, "e4m3")
            s["x"].copy_(q.to(torch.float8_e4m3fn))
            s["xs"].copy_(scales)
        else:
            s["a"] = x.to(torch.bfloat16)  # what the product's activations are quantised from
        s["y"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    else:
        T, k, E, L, H = case["tokens"], case["top_k"], case["experts"], case["local"], case["hidden"]
        score = torch.rand(T, E, generator=gen, device=dev)
        best = score.topk(k, dim=1)
        expert = best.indices.reshape(-1)  # of each (token, slot) pair
        order = torch.sort(expert, stable=True).indices
        local = order[expert[order] < L]  # this GPU owns experts 0..L-1
        R = local.numel()
        s["rows_used"] = R
        s["weights"] = torch.softmax(4.0 * best.values, dim=1)
        s["pair_row"] = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
        s["pair_row"][local] = torch.arange(R, dtype=torch.int32, device=dev)
        s["z"] = normal(T * k, H)  # room for every pair: this GPU's rows come first
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        if case["form"] == "train":
            s["dy"] = normal(T, H, std=0.1)
            s["dz"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=dev)
            s["dweights"] = torch.empty(T, k, dtype=torch.float32, device=dev)
    return s


def _power(e):
    """2^e in fp32 for whole e of -127..127, to the bit (pow and ldexp are not)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _round(a, lowest, bits, most):
    """Magnitudes to the nearest value of a format with `bits` bits behind the leading one, even on a tie: steps as of 2^lowest below that."""
    step = _power(torch.frexp(a).exponent.clamp(min=lowest + 1) - 1 - bits)
    return (torch.round(a / step) * step).clamp(max=most)


def _blocks(v, block):
    """[R, C] as [R, blocks, block] with zeros behind the last column."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % block)).view(v.shape[0], -1, block)


def _mx(v, element):
    """fp32 v in the MX format: the elements' values (fp32) and the scale bytes."""
    R, C = v.shape
    b = _blocks(v, MX)
    amax = b.abs().amax(dim=2)
    e = (torch.frexp(amax).exponent - 1 - (8 if element == "e4m3" else 2)).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    a = b * _power(-e)[:, :, None]
    q = _round(a.abs(), -6, 3, 448.0) if element == "e4m3" else _round(a.abs(), 0, 1, 6.0)
    return torch.copysign(q, b).view(R, -1)[:, :C], (e + 127).to(torch.uint8)


def _packed(q):
    """e2m1 values as bytes of two codes, the first in the low bits."""
    code = torch.searchsorted(torch.tensor(E2M1, device=q.device), q.abs().contiguous()).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    code = torch.nn.functional.pad(code, (0, code.shape[1] % 2))
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpacked(w):
    """The values (fp32) of bytes of two e2m1 codes."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=w.device)
    return torch.stack((table[(w & 15).int()], table[(w >> 4).int()]), dim=-1).flatten(-2)


def _scaled(values, scales):
    """MX elements (fp32) times their blocks' scales."""
    return values * _power(scales.int() - 127).repeat_interleave(MX, dim=-1)[..., :values.shape[-1]]


def _e4m3_blocks(v):
    """fp32 v as e4m3 values with fp32 scales for each row and 128 columns."""
    R, C = v.shape
    b = _blocks(v, FP8)
    amax = b.abs().amax(dim=2)
    scale = amax / torch.full_like(amax, 448.0)
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    a = b / scale[:, :, None]
    return torch.copysign(_round(a.abs(), -6, 3, 448.0), a).view(R, -1)[:, :C].to(torch.float8_e4m3fn), scale


def _padded(s, t):
    """[R, C] as [L, most, C] with zeros behind an expert's rows, and where row r went."""
    off = s["row_offset"].long()
    r = torch.arange(t.shape[0], device=off.device)
    e = torch.searchsorted(off[1:], r, right=True)
    p = torch.zeros(off.numel() - 1, s["most"], t.shape[1], dtype=torch.float32, device=off.device)
    p[e, r - off[e]] = t
    return p, (e, r - off[e])


def _as_scales(t):
    """Scale bytes as the powers of two that they stand for."""
    return t.view(torch.float8_e8m0fnu)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        stream, out = s["x"], {}
        if case["residual"]:
            stream = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
            out["stream"] = stream
        v, w = stream.float(), s["weight"].float()
        r = 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        n = v * r
        y = n * w
        if case["out"] == "bf16":
            out["y"] = y.to(torch.bfloat16)
        elif case["out"] == "fp8":
            out["y"], out["scales"] = _e4m3_blocks(y)
        else:
            q, scales = _mx(y, "e4m3")
            out["y"], out["scales"] = q.to(torch.float8_e4m3fn), _as_scales(scales)
        if case["form"] == "train":
            dy = s["dy"].float()
            g = dy * w
            dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
            if case["residual"]:
                dx = dx + s["dstream"].float()
            out["dx"] = dx.to(s["x"].dtype)
            out["dweight"] = (dy * n).sum(dim=0)
        return out
    if op == "quantize":
        q, scales = _mx(s["x"].float(), "e4m3")
        return {"q": q.to(torch.float8_e4m3fn), "scales": _as_scales(scales)}
    if op == "product":
        if case["x"] == "e4m3":
            x = _scaled(s["x"].float(), s["xs"])
        else:
            x = _scaled(*_mx(s["a"].float(), "e2m1"))
        w = _scaled(_unpacked(s["w"]), s["ws"])
        if not case["experts"]:
            return {"y": (x @ w.t()).to(torch.bfloat16)}
        x, at = _padded(s, x)
        return {"y": torch.bmm(x, w.transpose(1, 2))[at].to(torch.bfloat16)}
    at = s["pair_row"].long().view(-1, case["top_k"])
    here = at >= 0
    z = torch.where(here[..., None], s["z"][at.clamp(min=0)].float(), 0.0)
    out = {"y": (z * s["weights"][..., None]).sum(dim=1).to(torch.bfloat16)}
    if case["form"] == "train":
        R, dy = s["rows_used"], s["dy"].float()
        pair = torch.nonzero(here.view(-1)).view(-1)
        pair = pair[torch.argsort(at.view(-1)[pair])]  # the pair of each row
        s["dz"][:R] = s["weights"].view(-1)[pair][:, None] * dy[pair // case["top_k"]]
        out["dz"] = s["dz"]
        out["dweights"] = (z * dy[:, None, :]).sum(dim=2)
    return out


def _kernels(s):
    import moe_expert_ffn_persistent_amd as moe

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        got = moe.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out=s["y"], scales=s["scales"], residual_out=s["stream"],
                           quantize=None if case["out"] == "bf16" else case["out"])
        out = {"y": s["y"]}
        if case["residual"]:
            out["stream"] = got[-1]
        if case["out"] != "bf16":
            out["scales"] = s["scales"] if case["out"] == "fp8" else _as_scales(s["scales"])
        if case["form"] == "train":
            out["dx"], out["dweight"] = moe.rms_norm_backward(s["dy"], s["stream"] if case["residual"] else s["x"], s["weight"], eps=EPS,
                                                              dresidual=s["dstream"], out=s["dx"], dweight=s["dweight"])
        return out
    if op == "quantize":
        q, scales = moe.quantize_mx(s["x"], "e4m3", out=s["q"], scales=s["scales"])
        return {"q": q, "scales": _as_scales(scales)}
    if op == "product":
        if case["x"] == "e2m1":
            moe.quantize_mx(s["a"], "e2m1", out=s["x"], scales=s["xs"])
        return {"y": moe.mx_matmul(s["x"], s["xs"], s["w"], s["ws"], row_offset=s["row_offset"], out=s["y"])}
    out = {"y": moe.combine_rows(s["z"], s["pair_row"], case["top_k"], out=s["y"], weights=s["weights"])}
    if case["form"] == "train":
        out["dz"], out["dweights"] = moe.combine_rows_backward(s["dy"], s["z"], s["pair_row"], s["weights"], out=s["dz"], dweights=s["dweights"])
    return out


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "norm":
        R, H, t = case["rows"], case["hidden"], 4 if case["type"] == "fp32" else 2
        b = R * H * (t * (3 if case["residual"] else 1) + (2 if case["out"] == "bf16" else 1)) + 2 * H
        b += R * (4 * -(-H // FP8) if case["out"] == "fp8" else -(-H // MX) if case["out"] == "mx_e4m3" else 0)
        f = 5 * R * H
        if case["form"] == "train":
            b += R * H * (2 + t * (2 if case["residual"] else 1)) + 4 * H  # the stream is already counted
            f += 10 * R * H
        return {"bytes": b, "flops": f}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        return {"bytes": R * C * (5 if case["type"] == "fp32" else 3) + R * -(-C // MX), "flops": 3 * R * C}
    if op == "product":
        R, K, N, L = case["rows"], case["k"], case["n"], _work_counts(case)
        kb = -(-K // MX)
        # activations of four bits are quantised from bf16
        x = R * (K + kb) if case["x"] == "e4m3" else 2 * R * K
        return {"bytes": x + L * N * (K // 2 + kb) + 2 * R * N, "flops": 2 * R * K * N}
    T, k, H = case["tokens"], case["top_k"], case["hidden"]
    share = case["local"] / case["experts"]
    R = T * k * share
    read = T * (1.0 - (1.0 - share) ** k)  # tokens with a local slot
    b, f = 2 * H * (R + T) + 8 * T * k, 2 * R * H
    if case["form"] == "train":
        b += 2 * H * (read + R) + 4 * T * k
        f += 3 * R * H
    return {"bytes": b, "flops": f}


def _exact_two(exponent):
    """2^exponent in 64 bits, put together from its bits."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _exact_exponent(y):
    """floor(log2 |y|) of normal 64-bit numbers, read from their bits; zero gives -1023."""
    return ((y.contiguous().view(torch.int64) >> 52) & 2047) - 1023


def _exact_code(y, lowest, bits, most):
    """The nearest value of the format, even on a tie, in 64 bits."""
    step = _exact_two(_exact_exponent(y).clamp(min=lowest) - bits)
    return (y / step).round().mul(step).clamp(-most, most)


def _exact_mx(v, element):
    """The MX format's definition in 64 bits: elements and scales."""
    R, C = v.shape
    cb = -(-C // MX)
    full = torch.zeros(R, cb * MX, dtype=torch.float64, device=v.device)
    full[:, :C] = v
    blocks = full.reshape(R, cb, MX)
    amax = blocks.abs().max(dim=2).values
    scale = torch.where(amax > 0, _exact_two((_exact_exponent(amax) - (8 if element == "e4m3" else 2)).clamp(min=-127)), torch.ones_like(amax))
    y = (blocks / scale.unsqueeze(2)).reshape(R, cb * MX)[:, :C]
    return (_exact_code(y, -6, 3, 448) if element == "e4m3" else _exact_code(y, 0, 1, 6)), scale


def _exact_values(w, scales):
    """Bytes of two e2m1 codes with their scales, in 64 bits."""
    code = torch.empty(*w.shape[:-1], 2 * w.shape[-1], dtype=torch.int64, device=w.device)
    code[..., 0::2], code[..., 1::2] = (w & 15).long(), (w >> 4).long()
    exponent, fraction = (code >> 1) & 3, code & 1
    value = torch.where(exponent > 0, (2.0 + fraction) * _exact_two(exponent - 2), 0.5 * fraction)
    value = torch.where(code >= 8, -value, value)
    column = torch.arange(value.shape[-1], device=w.device) // MX
    return value * _exact_two(scales.long() - 127).index_select(-1, column)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        out, stream = {}, s["x"].double()
        if case["residual"]:
            stream = stream + s["residual"].double()
            out["stream"] = stream
            stream = stream.to(s["x"].dtype).double()  # what is stored is normalised
        w, H = s["weight"].double(), case["hidden"]
        rms = torch.sqrt(torch.linalg.vector_norm(stream, dim=1).square() / H + EPS).unsqueeze(1)
        unit = stream / rms
        if case["out"] == "bf16":
            out["y"] = unit * w
        elif case["out"] == "fp8":
            cb = -(-H // FP8)
            full = torch.zeros(case["rows"], cb * FP8, dtype=torch.float64, device=w.device)
            full[:, :H] = unit * w
            blocks = full.reshape(-1, cb, FP8)
            scale = (blocks.abs().max(dim=2).values / 448).float().double()
            scale[scale == 0] = 1
            out["y"], out["scales"] = _exact_code((blocks / scale.unsqueeze(2)).reshape(case["rows"], -1)[:, :H], -6, 3, 448), scale
        else:
            out["y"], out["scales"] = _exact_mx(unit * w, "e4m3")
        if case["form"] == "train":
            dy = s["dy"].double()
            along = torch.einsum("rh,rh->r", dy * w, unit).unsqueeze(1) / H
            out["dx"] = (dy * w - unit * along) / rms
            if case["residual"]:
                out["dx"] += s["dstream"].double()
            out["dweight"] = torch.einsum("rh,rh->h", dy, unit)
        return out
    if op == "quantize":
        q, scales = _exact_mx(s["x"].double(), "e4m3")
        return {"q": q, "scales": scales}
    if op == "product":
        if case["x"] == "e4m3":
            column = torch.arange(case["k"], device="cuda") // MX
            x = s["x"].float().double() * _exact_two(s["xs"].long() - 127).index_select(1, column)
        else:
            q, scales = _exact_mx(s["a"].double(), "e2m1")
            x = q * scales.index_select(1, torch.arange(case["k"], device="cuda") // MX)
        if not case["experts"]:
            return {"y": x @ _exact_values(s["w"], s["ws"]).t()}
        off, y = s["row_offset"].tolist(), torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            r = slice(off[e], off[e + 1])
            y[r] = x[r] @ _exact_values(s["w"][e], s["ws"][e]).t()
        return {"y": y}
    k, R = case["top_k"], s["rows_used"]
    pair = torch.empty(R, dtype=torch.int64, device="cuda")
    here = torch.nonzero(s["pair_row"] >= 0).view(-1)
    pair[s["pair_row"][here].long()] = here
    token, weight = torch.div(pair, k, rounding_mode="floor"), s["weights"].double().view(-1)[pair].unsqueeze(1)
    z = s["z"][:R].double()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    y.index_add_(0, token, z * weight)
    out = {"y": y}
    if case["form"] == "train":
        dy = s["dy"].double().index_select(0, token)
        out["dz"] = torch.zeros(s["dz"].shape, dtype=torch.float64, device="cuda")
        out["dz"][:R] = dy * weight
        dweights = torch.zeros(case["tokens"] * k, dtype=torch.float64, device="cuda")
        dweights[pair] = torch.einsum("rh,rh->r", dy, z)
        out["dweights"] = dweights.view(-1, k)
    return out
