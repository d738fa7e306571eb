"""The operators around the expert FFN, as a user's program calls them: rows dispatched to and combined from the
experts, matrix products grouped by expert (forward, input gradient, weight gradient), SwiGLU with router weights,
quantisation to e4m3 with block scales, and the block-scaled e4m3 matrix product, dense and grouped by expert.

`own` false: each operator in plain torch operations in 32 bits. `own` true: the framework's kernels."""
import math
import random

import torch

own = False

BLOCK = 128  # columns of one fp32 scale


def listed():
    return [
        # the experts' first product for a decode batch: few rows, the weights read once
        {"name": "grouped_decode", "op": "grouped", "form": "forward", "experts": 32, "rows": 128, "k": 7168, "n": 4096,
         "skew": 0.3, "empty": 1, "grad": "bf16"},
        # forward, input gradient and weight gradient of an odd-sized layer: ragged experts, two without a row
        {"name": "grouped_odd_train", "op": "grouped", "form": "train", "experts": 7, "rows": 1777, "k": 1000, "n": 520,
         "skew": 0.6, "empty": 2, "grad": "fp32"},
        # a training step's expert products at the sizes of one GPU's share
        {"name": "grouped_train", "op": "grouped", "form": "train", "experts": 32, "rows": 32768, "k": 7168, "n": 4096,
         "skew": 0.3, "empty": 0, "grad": "bf16"},
        # the activation of a decode batch, written as e4m3 for the fp8 second product
        {"name": "swiglu_decode_fp8", "op": "swiglu", "form": "forward", "rows": 128, "inter": 2048, "weights": False, "out": "fp8"},
        # the activation's forward and backward pass in a training step
        {"name": "swiglu_train", "op": "swiglu", "form": "train", "rows": 32768, "inter": 2048, "weights": True, "out": "bf16"},
        # a decode batch's tokens to and from one GPU's experts
        {"name": "rows_decode", "op": "rows", "tokens": 128, "top_k": 8, "experts": 128, "local": 16, "hidden": 4096},
        # a prefill batch's
        {"name": "rows_prefill", "op": "rows", "tokens": 16384, "top_k": 8, "experts": 256, "local": 32, "hidden": 7168},
        # activations of a decode batch to e4m3 with a scale for each row and 128 columns
        {"name": "quantize_decode", "op": "quantize", "rows": 128, "cols": 7168, "block_rows": 1, "type": "bf16"},
        # a weight matrix to e4m3 with a scale for each 128 x 128 block
        {"name": "quantize_weights", "op": "quantize", "rows": 32768, "cols": 7168, "block_rows": 128, "type": "bf16"},
        # one token through a dense layer
        {"name": "fp8_token", "op": "fp8", "experts": 0, "rows": 1, "k": 7168, "n": 4096, "skew": 0.0, "empty": 0},
        # a prefill batch through a dense layer
        {"name": "fp8_prefill", "op": "fp8", "experts": 0, "rows": 8192, "k": 7168, "n": 4096, "skew": 0.0, "empty": 0},
        # the experts' second product over ragged rows
        {"name": "fp8_grouped", "op": "fp8", "experts": 32, "rows": 16384, "k": 2048, "n": 7168, "skew": 0.3, "empty": 1},
    ]


def _size(rng, lo, hi, step=1):
    """A size of lo..hi, even over its logarithm, a multiple of `step`."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "swiglu", "rows", "quantize", "fp8", "fp8"])
    if op in ("grouped", "fp8"):
        train = op == "grouped" and rng.random() < 0.6
        experts = 0 if op == "fp8" and rng.random() < 0.5 else _size(rng, 1, 32)
        c = {"op": op, "experts": experts, "rows": _size(rng, 1, 32768 if train else 16384),
             "k": _size(rng, 128, 7168, 8 if op == "grouped" else 16), "n": _size(rng, 64, 7168, 8),
             "skew": rng.choice([0.0, 0.3, 0.6]) if experts else 0.0, "empty": rng.randrange(0, experts // 4 + 1)}
        while max(1, experts) * c["k"] * c["n"] > 32 * 7168 * 4096 or c["rows"] * c["k"] * c["n"] > 32768 * 7168 * 4096:
            c["n"] = max(64, c["n"] // 16 * 8)
        if op == "grouped":
            c |= {"form": "train" if train else "forward", "grad": rng.choice(["bf16", "fp32"])}
        return c
    if op == "swiglu":
        train = rng.random() < 0.5
        return {"op": op, "form": "train" if train else "forward", "rows": _size(rng, 1, 32768), "inter": _size(rng, 64, 4096, 8),
                "weights": rng.random() < 0.7, "out": "bf16" if train else rng.choice(["bf16", "fp8"])}
    if op == "rows":
        top_k, experts = rng.randrange(1, 9), rng.choice([8, 16, 32, 64, 128, 256])
        return {"op": op, "tokens": _size(rng, 1, 16384), "top_k": top_k, "experts": experts,
                "local": max(1, experts // rng.choice([1, 2, 4, 8])) if top_k < 3 else max(1, experts // 8), "hidden": _size(rng, 64, 7168, 8)}
    return {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 64, 7168, 8), "block_rows": rng.choice([1, 1, 128]),
            "type": rng.choice(["bf16", "fp32"])}


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
    """Experts with a row, as drawn on average: each is read (or its gradient written) once."""
    experts = max(1, case["experts"]) - case["empty"]
    return experts * (1.0 - (1.0 - 1.0 / experts) ** case["rows"])


def _codes(shape, gen):
    """e4m3 values as quantised activations and weights have them: a bell over the whole range."""
    return (torch.randn(shape, generator=gen, device="cuda") * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev, op = torch.device("cuda"), case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *shape, std=1.0, dtype=torch.bfloat16: torch.randn(shape, generator=gen, device=dev, dtype=dtype).mul_(std)  # noqa: E731
    s = {"case": case}
    if op in ("grouped", "fp8"):
        counts = _counts(case, seed)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        s["row_offset"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
        s["most"] = max(counts)  # rows of the largest expert, known where its buffers were sized
    if op == "grouped":
        L, R, K, N = case["experts"], case["rows"], case["k"], case["n"]
        s["x"], s["w"] = normal(R, K), normal(L, N, K, std=0.02)
        s["y"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
        if case["form"] == "train":
            s["dy"] = normal(R, N, std=0.1)
            s["dx"] = torch.empty(R, K, dtype=torch.bfloat16, device=dev)
            s["dw"] = torch.empty(L, N, K, dtype=torch.float32 if case["grad"] == "fp32" else torch.bfloat16, device=dev)
    elif op == "swiglu":
        R, I = case["rows"], case["inter"]
        s["a"] = normal(R, 2 * I)
        s["weight"] = torch.rand(R, generator=gen, device=dev) if case["weights"] else None
        if case["form"] == "train":
            s["dh"] = normal(R, I, std=0.1)
            s["da"] = torch.empty(R, 2 * I, dtype=torch.bfloat16, device=dev)
            s["dweight"] = torch.empty(R, dtype=torch.float32, device=dev) if case["weights"] else None
        s["h"] = torch.empty(R, I, dtype=torch.float8_e4m3fn if case["out"] == "fp8" else torch.bfloat16, device=dev)
        s["scales"] = torch.empty(R, -(-I // BLOCK), dtype=torch.float32, device=dev) if case["out"] == "fp8" else None
    elif op == "rows":
        T, k, E, L, H = case["tokens"], case["top_k"], case["experts"], case["local"], case["hidden"]
        expert = torch.rand(T, E, generator=gen, device=dev).topk(k, dim=1).indices.reshape(-1)  # of each (token, slot) pair
        order = torch.sort(expert, stable=True).indices
        local = order[expert[order] < L]  # this GPU owns experts 0..L-1
        R = local.numel()
        s["rows_used"] = R
        s["row_pair"] = torch.zeros(T * k, dtype=torch.int32, device=dev)
        s["row_pair"][:R] = local.to(torch.int32)
        s["pair_row"] = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
        s["pair_row"][local] = torch.arange(R, dtype=torch.int32, device=dev)
        counts = torch.bincount(expert, minlength=E)[:L]
        s["row_offset"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["x"], s["z"] = normal(T, H), normal(T * k, H)
        s["rows"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=dev)  # room for every pair: this GPU's come first
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    elif op == "quantize":
        R, C, b = case["rows"], case["cols"], case["block_rows"]
        s["x"] = normal(R, C, dtype=torch.float32 if case["type"] == "fp32" else torch.bfloat16)
        s["x"] *= torch.exp(normal(R, 1, dtype=torch.float32)).to(s["x"].dtype)  # rows of different sizes
        s["q"] = torch.empty(R, C, dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.empty(-(-R // b), -(-C // BLOCK), dtype=torch.float32, device=dev)
    else:
        L, R, K, N = max(1, case["experts"]), case["rows"], case["k"], case["n"]
        kb = -(-K // BLOCK)
        s["x"], s["w"] = _codes((R, K), gen), _codes((L, N, K), gen)
        s["xs"] = (0.5 + torch.rand(R, kb, generator=gen, device=dev)) * 0.01
        s["ws"] = (0.5 + torch.rand(L, -(-N // BLOCK), kb, generator=gen, device=dev)) * 2e-4
        if not case["experts"]:
            s["w"], s["ws"], s["row_offset"] = s["w"][0], s["ws"][0], None
        s["y"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    return s


def _padded(s, *tensors):
    """Each [R, C] tensor as [L, most, C] fp32 with zeros behind an expert's rows, and where row r went."""
    off = s["row_offset"].long()
    r = torch.arange(tensors[0].shape[0], device=off.device)
    e = torch.searchsorted(off[1:], r, right=True)
    at = (e, r - off[e])
    out = []
    for t in tensors:
        p = torch.zeros(off.numel() - 1, s["most"], t.shape[1], dtype=torch.float32, device=off.device)
        p[at] = t.float()
        out.append(p)
    return out, at


def _e4m3(y):
    """y to the nearest e4m3 value (even on a tie), at most 448."""
    a = y.abs()
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a).exponent.clamp(min=-5) - 4)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), y).to(torch.float8_e4m3fn)


def _quantized(v, block_rows):
    """fp32 v as e4m3 values and the scales of its block_rows x 128 blocks."""
    R, C = v.shape
    pad = torch.nn.functional.pad(v, (0, -C % BLOCK, 0, -R % block_rows))
    amax = pad.abs().view(pad.shape[0] // block_rows, block_rows, pad.shape[1] // BLOCK, BLOCK).amax(dim=(1, 3))
    scale = amax / torch.full_like(amax, 448.0)  # a quotient: times 1/448 is not the same
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return _e4m3(v / _spread(scale, block_rows, R, C)), scale


def _spread(scale, block_rows, R, C):
    """Block scales as one for each element."""
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :C].repeat_interleave(block_rows, dim=-2)[..., :R, :]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "grouped":
        w = s["w"].float()
        (x,), at = _padded(s, s["x"])
        y = torch.bmm(x, w.transpose(1, 2))[at].to(torch.bfloat16)
        if case["form"] == "forward":
            return {"y": y}
        (dy,), at = _padded(s, s["dy"])
        return {"y": y, "dx": torch.bmm(dy, w)[at].to(torch.bfloat16), "dw": torch.bmm(dy.transpose(1, 2), x).to(s["dw"].dtype)}
    if op == "swiglu":
        I = case["inter"]
        g, u = s["a"][:, :I].float(), s["a"][:, I:].float()
        weight = s["weight"][:, None] if case["weights"] else 1.0
        sig = 1.0 / (1.0 + torch.exp(-g))
        act = g * sig * u
        h = act * weight
        if case["out"] == "fp8":
            q, scales = _quantized(h, 1)
            return {"h": q, "scales": scales}
        out = {"h": h.to(torch.bfloat16)}
        if case["form"] == "train":
            dh = s["dh"].float()
            back = dh * weight
            out["da"] = torch.cat([back * u * sig * (1.0 + g * (1.0 - sig)), back * g * sig], dim=1).to(torch.bfloat16)
            if case["weights"]:
                out["dweight"] = (dh * act).sum(dim=1)
        return out
    if op == "rows":
        k, R = case["top_k"], s["rows_used"]
        at = s["pair_row"].long().view(-1, k)
        picked = torch.where((at >= 0)[..., None], s["z"][at.clamp(min=0)].float(), 0.0)
        s["rows"][:R] = s["x"][s["row_pair"][:R].long() // k]
        return {"rows": s["rows"], "y": picked.sum(dim=1).to(torch.bfloat16)}
    if op == "quantize":
        q, scales = _quantized(s["x"].float(), case["block_rows"])
        return {"q": q, "scales": scales}
    x = s["x"].float() * _spread(s["xs"], 1, *s["x"].shape)
    w = s["w"].float() * _spread(s["ws"], BLOCK, *s["w"].shape[-2:])
    if not case["experts"]:
        return {"y": (x @ w.t()).to(torch.bfloat16)}
    (x,), at = _padded(s, x)
    return {"y": torch.bmm(x, w.transpose(1, 2))[at].to(torch.bfloat16)}


def _kernels(s):
    import moe_expert_ffn_persistent_amd as moe

    case, op = s["case"], s["case"]["op"]
    if op == "grouped":
        out = {"y": moe.grouped_matmul(s["x"], s["w"], s["row_offset"], out=s["y"])}
        if case["form"] == "train":
            out["dx"] = moe.grouped_matmul_dgrad(s["dy"], s["w"], s["row_offset"], out=s["dx"])
            out["dw"] = moe.grouped_matmul_wgrad(s["dy"], s["x"], s["row_offset"], out=s["dw"])
        return out
    if op == "swiglu":
        if case["out"] == "fp8":
            q, scales = moe.swiglu(s["a"], row_weight=s["weight"], out=s["h"], scales=s["scales"])
            return {"h": q, "scales": scales}
        out = {"h": moe.swiglu(s["a"], row_weight=s["weight"], out=s["h"])}
        if case["form"] == "train":
            da, dweight = moe.swiglu_backward(s["a"], s["dh"], row_weight=s["weight"], out=s["da"], drow_weight=s["dweight"])
            out["da"] = da
            if case["weights"]:
                out["dweight"] = dweight
        return out
    if op == "rows":
        rows = moe.dispatch_rows(s["x"], s["row_pair"], s["row_offset"], case["top_k"], out=s["rows"])
        return {"rows": rows, "y": moe.combine_rows(s["z"], s["pair_row"], case["top_k"], out=s["y"])}
    if op == "quantize":
        q, scales = moe.quantize_fp8(s["x"], block_rows=case["block_rows"], out=s["q"], scales=s["scales"])
        return {"q": q, "scales": scales}
    return {"y": moe.fp8_matmul(s["x"], s["xs"], s["w"], s["ws"], row_offset=s["row_offset"], out=s["y"])}


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "grouped":
        R, K, N, L = case["rows"], case["k"], case["n"], _work_counts(case)
        b, f = 2 * (R * K + L * N * K + R * N), 2 * R * K * N
        if case["form"] == "train":
            # dy and the second output; the weight gradient of every expert is written
            b += 2 * (R * N + R * K) + case["experts"] * N * K * (4 if case["grad"] == "fp32" else 2)
            f *= 3
        return {"bytes": b, "flops": f}
    if op == "swiglu":
        R, I = case["rows"], case["inter"]
        b = R * I * (4 + (1 if case["out"] == "fp8" else 2)) + (4 * R if case["weights"] else 0)
        if case["out"] == "fp8":
            b += 4 * R * -(-I // BLOCK)
        f = 5 * R * I
        if case["form"] == "train":
            b += R * I * 6 + (4 * R if case["weights"] else 0)
            f += 12 * R * I
        return {"bytes": b, "flops": f}
    if op == "rows":
        T, k, H = case["tokens"], case["top_k"], case["hidden"]
        share = case["local"] / case["experts"]
        R = T * k * share
        read = T * (1.0 - (1.0 - share) ** k)  # tokens with a local slot
        return {"bytes": 2 * H * (read + 2 * R + T) + 8 * T * k, "flops": R * H}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        return {"bytes": R * C * (5 if case["type"] == "fp32" else 3) + 4 * -(-R // case["block_rows"]) * -(-C // BLOCK), "flops": 3 * R * C}
    R, K, N, L = case["rows"], case["k"], case["n"], _work_counts(case)
    kb = -(-K // BLOCK)
    return {"bytes": R * K + L * N * K + 2 * R * N + 4 * (R * kb + L * -(-N // BLOCK) * kb), "flops": 2 * R * K * N}


def _exact_codes(v, block_rows):
    """The definition in 64 bits: scale = fp32(amax / 448), code = the e4m3 value nearest to the fp32 quotient."""
    R, C = v.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    full = torch.zeros(rb * block_rows, cb * BLOCK, dtype=torch.float64, device=v.device)
    full[:R, :C] = v
    blocks = full.reshape(rb, block_rows, cb, BLOCK).transpose(1, 2)
    scale = (blocks.abs().flatten(2).max(dim=2).values / 448).float().double()
    scale[scale == 0] = 1
    y = (blocks / scale[:, :, None, None]).float().double().transpose(1, 2).reshape(full.shape)[:R, :C]
    exponent = torch.floor(torch.log2(y.abs().clamp(min=2.0**-20)))
    exponent += (torch.pow(2.0, exponent + 1) <= y.abs()).double() - (torch.pow(2.0, exponent) > y.abs()).double()
    step = torch.pow(2.0, exponent.clamp(min=-6) - 3)
    return (y / step).round().mul(step).clamp(-448, 448), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "grouped":
        off = s["row_offset"].tolist()
        y = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
        out = {"y": y}
        if case["form"] == "train":
            out["dx"] = torch.empty(s["dx"].shape, dtype=torch.float64, device="cuda")
            out["dw"] = torch.empty(s["dw"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            r = slice(off[e], off[e + 1])
            x, w = s["x"][r].double(), s["w"][e].double()
            y[r] = x @ w.t()
            if case["form"] == "train":
                dy = s["dy"][r].double()
                out["dx"][r] = dy @ w
                out["dw"][e] = dy.t() @ x
        return out
    if op == "swiglu":
        g, u = (t.double() for t in s["a"].chunk(2, dim=1))
        weight = s["weight"].double().unsqueeze(1) if case["weights"] else torch.ones(1, 1, dtype=torch.float64, device="cuda")
        sig = torch.reciprocal(1 + torch.exp(-g))
        silu = g * sig
        if case["out"] == "fp8":
            q, scales = _exact_codes(silu * u * weight, 1)
            return {"h": q, "scales": scales}
        out = {"h": silu * u * weight}
        if case["form"] == "train":
            dh = s["dh"].double()
            out["da"] = torch.cat([dh * weight * u * (sig + silu * (1 - sig)), dh * weight * silu], dim=1)
            if case["weights"]:
                out["dweight"] = torch.einsum("ri,ri->r", dh, silu * u)
        return out
    if op == "rows":
        k, R = case["top_k"], s["rows_used"]
        token = torch.div(s["row_pair"][:R], k, rounding_mode="floor").long()
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        y.index_add_(0, token, s["z"][:R].double())
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
        rows[:R] = s["x"].double().index_select(0, token)
        return {"rows": rows, "y": y}
    if op == "quantize":
        q, scales = _exact_codes(s["x"].double(), case["block_rows"])
        return {"q": q, "scales": scales}
    x, w = s["x"].float().double(), s["w"].float().double()
    K, N = case["k"], case["n"]
    column, feature = torch.arange(K, device="cuda") // BLOCK, torch.arange(N, device="cuda") // BLOCK
    x = x * s["xs"].double()[:, column]
    y = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
    off = s["row_offset"].tolist() if case["experts"] else [0, case["rows"]]
    for e in range(max(1, case["experts"])):
        we, se = (w[e], s["ws"][e]) if case["experts"] else (w, s["ws"])
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ (we * se.double()[feature][:, column]).t()
    return {"y": y}
