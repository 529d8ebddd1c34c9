"""The measured cases of the operators on 8-bit floating point codes with a
scale for each block of 128: the codes themselves (of activations and of
weights), the gated activation between two products with its 8-bit checkpoint
and its gradient from that checkpoint, the product of such codes, the same
grouped by expert, and the weights' gradient from checkpointed codes.

`run` computes them in plain torch operations in 32 bits, or, where `own` is
true, through this package's public calls."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3fn": torch.float8_e4m3fn,
          "e5m2": torch.float8_e5m2, "e8m0": torch.float8_e8m0fnu}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3fn": 1, "e5m2": 1, "e8m0": 1}
LARGEST = {"e4m3fn": 448.0, "e5m2": 57344.0}
LEAST_SCALE = 2.0 ** -126
B = 128


def listed():
    return [
        # a prompt's activations at the projection's width, an odd number of them, before a product
        {"name": "quant_prompt", "op": "quant", "T": 2047, "n": 1920, "x": "bf16", "out": "e4m3fn", "scale": "e8m0",
         "rows": 1, "E": 1},
        # the weights of eight experts after an optimizer's step, kept in 32 bits; scales as checkpoints hold them
        {"name": "quant_weights", "op": "quant", "T": 4096, "n": 4096, "x": "fp32", "out": "e4m3fn", "scale": "fp32",
         "rows": 128, "E": 8},
        # a prompt of odd length through the gate of a layer that is served: nothing is kept
        {"name": "swiglu_prompt", "op": "swiglu", "T": 1023, "F": 1925, "x": "bf16", "out": "e4m3fn", "scale": "fp32",
         "keep": False},
        # a training batch; gate and up are kept in 8 bits, and the gradient comes from those
        {"name": "swiglu_grad_batch", "op": "swiglu_grad", "T": 8192, "F": 8192, "x": "bf16", "out": "e4m3fn",
         "scale": "e8m0"},
        # one decoded token through the projection, scales as checkpoints hold them: the weights are read once
        {"name": "mm_one_token", "op": "mm", "M": 1, "N": 5760, "K": 1920, "a": "e4m3fn", "w": "e4m3fn", "scale": "fp32",
         "out": "bf16", "bias": False},
        # a ragged batch of prompts under scales as checkpoints hold them
        {"name": "mm_ragged", "op": "mm", "M": 2047, "N": 4096, "K": 4096, "a": "e4m3fn", "w": "e4m3fn", "scale": "fp32",
         "out": "fp16", "bias": True},
        # the benchmark's square, a gradient in e5m2 against weights
        {"name": "mm_square", "op": "mm", "M": 8192, "N": 8192, "K": 8192, "a": "e5m2", "w": "e4m3fn", "scale": "e8m0",
         "out": "bf16", "bias": False},
        # a decoded batch's rows over sixteen experts: latency and the weights' bytes
        {"name": "grouped_decode", "op": "grouped", "T": 32, "E": 16, "N": 4096, "K": 2048, "a": "e4m3fn", "w": "e4m3fn",
         "scale": "fp32", "out": "bf16"},
        # prompts over many small experts, ragged, some of them without a row
        {"name": "grouped_prompt", "op": "grouped", "T": 4095, "E": 64, "N": 2048, "K": 1920, "a": "e4m3fn", "w": "e4m3fn",
         "scale": "e8m0", "out": "bf16"},
        # a training batch over a few large experts
        {"name": "grouped_batch", "op": "grouped", "T": 16384, "E": 8, "N": 8192, "K": 4096, "a": "e4m3fn", "w": "e4m3fn",
         "scale": "e8m0", "out": "bf16"},
        # one layer's weights from a short batch, odd sizes, summed over in 32 bits
        {"name": "weight_grad_odd", "op": "weight_grad", "T": 1023, "E": 0, "N": 1925, "K": 1920, "g": "bf16", "a": "e4m3fn",
         "out": "fp32"},
        # the same training batch's gradient of the experts' weights
        {"name": "weight_grad_batch", "op": "weight_grad", "T": 16384, "E": 8, "N": 8192, "K": 4096, "g": "bf16",
         "a": "e4m3fn", "out": "bf16"},
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of low..high, odd or round."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.4 and v >= 64:
        v = v // 64 * 64
    return v


def draw(rng):
    op = rng.choice(["quant", "swiglu", "swiglu_grad", "mm", "mm", "grouped", "grouped", "weight_grad", "weight_grad"])
    code = lambda: rng.choice(["e4m3fn", "e4m3fn", "e4m3fn", "e5m2"])  # noqa: E731
    real = lambda: rng.choice(["bf16", "bf16", "fp16", "fp32"])  # noqa: E731
    while True:
        if op == "quant":
            rows = rng.choice([1, 1, 128])
            c = {"op": op, "T": _log(rng, 1, 16384), "n": _log(rng, 64, 16384), "x": real(), "out": code(),
                 "scale": rng.choice(["e8m0", "fp32"]), "rows": rows, "E": rng.choice([1, 1, 5]) if rows == 128 else 1}
            fits = c["E"] * c["T"] * c["n"] <= 2 ** 27
        elif op in ("swiglu", "swiglu_grad"):
            c = {"op": op, "T": _log(rng, 1, 8192), "F": _log(rng, 64, 16384), "x": real(), "out": code(),
                 "scale": rng.choice(["e8m0", "fp32"])}
            if op == "swiglu":
                c["keep"] = rng.random() < 0.6
            fits = c["T"] * c["F"] <= 2 ** 26
        elif op == "mm":
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 64, 16384), "a": code(),
                 "w": code(), "scale": rng.choice(["e8m0", "fp32"]), "out": real(), "bias": rng.random() < 0.3}
            fits = c["M"] * c["N"] * c["K"] <= 2 ** 38
        else:
            c = {"op": op, "T": _log(rng, 1, 16384), "E": _log(rng, 1, 128), "N": _log(rng, 64, 8192),
                 "K": _log(rng, 64, 8192), "a": code(), "out": real()}
            if op == "grouped":
                c.update(w="e4m3fn", scale=rng.choice(["e8m0", "fp32"]))
            else:
                c.update(g=real(), E=rng.choice([0, c["E"]]))
            fits = c["T"] * c["N"] * c["K"] <= 2 ** 38 and max(1, c["E"]) * c["N"] * c["K"] <= 2 ** 28
        if fits:
            return c


# ---- codes and scales in plain operations, for inputs and for the plain forms ----

def _blocks(n):
    return (n + B - 1) // B


def _scales(most, out, scale):
    """Scales of blocks whose largest magnitude is `most`, in 32 bits."""
    if scale == "fp32":
        return (most / LARGEST[out]).clamp_min(LEAST_SCALE)
    # the least power of two that brings `most` within the type: both largest values are 7/8 of one
    digits, power = torch.frexp(most)
    power = power - (9 if out == "e4m3fn" else 16) + (digits > 0.875)
    return torch.ldexp(torch.ones_like(most), torch.where(most > 0, power, -126).clamp_min(-126))


def _spread(s, n, dim):
    """Each block's scale in the places of its values."""
    return s.repeat_interleave(B, dim).narrow(dim, 0, n)


def _codes(x, rows, out, scale):
    """Codes and 32-bit scales of x [.., T, n] in blocks of `rows` x 128."""
    T, n = x.shape[-2:]
    pad = torch.nn.functional.pad(x.float().abs(), (0, _blocks(n) * B - n, 0, -T % rows))
    most = pad.unflatten(-1, (-1, B)).amax(-1).unflatten(-2, (-1, rows)).amax(-2)
    s = _scales(most, out, scale)
    at = _spread(s if rows == 1 else s.repeat_interleave(rows, -2).narrow(-2, 0, T), n, -1)
    return (x.float() / at).clamp(-LARGEST[out], LARGEST[out]).to(DTYPES[out]), s


def _values(codes, s, rows=1):
    """What codes and their blocks' scales stand for, in 32 bits."""
    T, n = codes.shape[-2:]
    s = s.float()
    if rows > 1:
        s = s.repeat_interleave(rows, -2).narrow(-2, 0, T)
    return codes.float() * _spread(s, n, -1)


# ---- inputs ----

def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _stream(gen, T, n, std, dtype=torch.float32):
    """Activations: tokens of different size, a few channels far above the rest."""
    loud = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    size = torch.exp(torch.randn(T, 1, generator=gen, device="cuda") * 0.5)
    return (torch.randn(T, n, generator=gen, device="cuda") * std * loud * size).to(dtype)


def _weights(gen, E, N, K, out, scale):
    """Codes [E, N, K] and scales [E, blocks of N, blocks of K] of experts' weights, one after the other."""
    codes = torch.empty(E, N, K, dtype=DTYPES[out], device="cuda")
    scales = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
    for e in range(E):
        codes[e], scales[e] = _codes(_normal(gen, (N, K), K ** -0.5), B, out, scale)
    return codes, scales.to(DTYPES[scale])


def _routing(seed, T, E):
    """Rows of each expert, skewed as routers leave them: every eighth expert
    has none, and a buffer of fixed size has a few rows behind the last one's."""
    gen = torch.Generator().manual_seed(seed)
    likely = torch.exp(torch.randn(E, generator=gen) * 0.7)
    if E >= 8:
        likely[torch.randperm(E, generator=gen)[:E // 8]] = 0
    used = T - T // 50
    return torch.bincount(torch.multinomial(likely, used, replacement=True, generator=gen), minlength=E).tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    op, s = case["op"], dict(case)
    if op == "quant":
        T, n = case["T"], case["n"]
        if case["rows"] == 1:
            s["v"] = _stream(gen, T, n, 0.8, DTYPES[case["x"]])
        elif case["E"] == 1:
            s["v"] = _normal(gen, (T, n), n ** -0.5, DTYPES[case["x"]])
        else:
            s["v"] = _normal(gen, (case["E"], T, n), n ** -0.5, DTYPES[case["x"]])
    elif op == "swiglu":
        # one product makes both halves
        both = _stream(gen, case["T"], 2 * case["F"], 1.0, DTYPES[case["x"]])
        s["gate"], s["up"] = both[:, :case["F"]], both[:, case["F"]:]
    elif op == "swiglu_grad":
        T, F = case["T"], case["F"]
        s["g"] = _normal(gen, (T, F), 1e-2, DTYPES[case["x"]])
        halves = [_codes(_stream(gen, T, F, 1.0, DTYPES[case["x"]]), 1, case["out"], case["scale"]) for _ in range(2)]
        s["kept"] = torch.cat([h[0].view(torch.uint8) for h in halves], 1).view(DTYPES[case["out"]])
        s["kept_scale"] = torch.cat([h[1] for h in halves], 1).to(DTYPES[case["scale"]])
    elif op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        s["codes"], scale = _codes(_stream(gen, M, K, 0.8), 1, case["a"], case["scale"])
        s["sa"] = scale.to(DTYPES[case["scale"]])
        w, sw = _weights(gen, 1, N, K, case["w"], case["scale"])
        s["weights"], s["sw"] = w[0], sw[0]
        s["b"] = _normal(gen, (N,), 1.0, DTYPES[case["out"]]) if case["bias"] else None
    else:
        T, K = case["T"], case["K"]
        s["codes"], scale = _codes(_stream(gen, T, K, 0.8), 1, case["a"], case.get("scale", "e8m0"))
        s["sa"] = scale.to(DTYPES[case.get("scale", "e8m0")])
        s["count"] = _routing(int(seed) * 31 + 5, T, case["E"]) if case["E"] else None
        s["ends"] = torch.tensor(s["count"], device="cuda").cumsum(0).int() if case["E"] else None
        if op == "grouped":
            s["weights"], s["sw"] = _weights(gen, case["E"], case["N"], K, case["w"], case["scale"])
        else:
            s["grad"] = _normal(gen, (T, case["N"]), 1e-2, DTYPES[case["g"]])
    return s


# ---- the plain forms ----

def _swiglu(s):
    gate, up = s["gate"].float(), s["up"].float()
    codes, scale = _codes(gate / (1 + torch.exp(-gate)) * up, 1, s["out"], s["scale"])
    got = [(codes, scale)]
    if s["keep"]:
        halves = [_codes(v, 1, s["out"], s["scale"]) for v in (s["gate"], s["up"])]
        got.append((torch.cat([h[0].view(torch.uint8) for h in halves], 1).view(codes.dtype),
                    torch.cat([h[1] for h in halves], 1)))
    return got


def _halves(s):
    F, blocks = s["F"], _blocks(s["F"])
    return [_values(s["kept"][:, i * F:i * F + F], s["kept_scale"][:, i * blocks:i * blocks + blocks]) for i in (0, 1)]


def _swiglu_grad(s):
    gate, up = _halves(s)
    g, p = s["g"].float(), 1 / (1 + torch.exp(-gate))
    return torch.cat([g * up * p * (1 + gate * (1 - p)), g * gate * p], 1).to(s["g"].dtype)


def _mm(s):
    y = _values(s["codes"], s["sa"]) @ _values(s["weights"], s["sw"], B).t()
    return (y if s["b"] is None else y + s["b"].float()).to(DTYPES[s["out"]])


def _grouped(s):
    a = _values(s["codes"], s["sa"])
    out = torch.zeros(s["T"], s["N"], dtype=DTYPES[s["out"]], device=a.device)
    at = 0
    for e, rows in enumerate(s["count"]):
        out[at:at + rows] = a[at:at + rows] @ _values(s["weights"][e], s["sw"][e], B).t()
        at += rows
    return out


def _weight_grad(s):
    a, g = _values(s["codes"], s["sa"]), s["grad"].float()
    if s["count"] is None:
        return (g.t() @ a).to(DTYPES[s["out"]])
    out = torch.zeros(s["E"], s["N"], s["K"], dtype=DTYPES[s["out"]], device=a.device)
    at = 0
    for e, rows in enumerate(s["count"]):
        out[e] = g[at:at + rows].t() @ a[at:at + rows]
        at += rows
    return out


def _standing_for(pairs):
    """Codes of computed values as the values they stand for: a value next to a
    border may fall to either side, a scale with it."""
    return [_values(codes, scale).to(torch.bfloat16) for codes, scale in pairs]


def run(state):
    s, op = state, state["op"]
    if own:
        import bit_exact_fp8_amd as fw
        if op == "quant":
            return fw.block_quant(s["v"], block_rows=s["rows"], out_dtype=DTYPES[s["out"]], scale_dtype=DTYPES[s["scale"]])
        if op == "swiglu":
            r = fw.swiglu_block_quant(s["gate"], s["up"], out_dtype=DTYPES[s["out"]], scale_dtype=DTYPES[s["scale"]],
                                      keep=s["keep"])
            if not s["keep"]:
                return _standing_for([(r.codes, r.scale)])
            return _standing_for([(r.codes, r.scale)]) + [r.kept, r.kept_scale]
        if op == "swiglu_grad":
            return fw.swiglu_block_backward(s["g"], s["kept"], s["kept_scale"])
        if op == "mm":
            return fw.block_scaled_mm(s["codes"], s["weights"].t(), s["sa"], s["sw"].t(), bias=s["b"],
                                      out_dtype=DTYPES[s["out"]])
        if op == "grouped":
            return fw.grouped_block_scaled_mm(s["codes"], s["weights"].transpose(1, 2), s["sa"], s["sw"].transpose(1, 2),
                                              s["ends"], out_dtype=DTYPES[s["out"]])
        return fw.block_weight_grad(s["grad"], s["codes"], s["sa"], s["ends"], out_dtype=DTYPES[s["out"]])
    if op == "quant":
        codes, scale = _codes(s["v"], s["rows"], s["out"], s["scale"])
        return codes, scale.to(DTYPES[s["scale"]])
    if op == "swiglu":
        got = _swiglu(s)
        if not s["keep"]:
            return _standing_for(got)
        return _standing_for(got[:1]) + [got[1][0], got[1][1].to(DTYPES[s["scale"]])]
    return {"swiglu_grad": _swiglu_grad, "mm": _mm, "grouped": _grouped, "weight_grad": _weight_grad}[op](s)


def work(case):
    op = case["op"]
    if op == "quant":
        T, n = case["E"] * case["T"], case["n"]
        scales = case["E"] * (-(-case["T"] // case["rows"])) * _blocks(n) * BYTES[case["scale"]]
        return {"bytes": T * n * (BYTES[case["x"]] + 1) + scales, "flops": 2 * T * n}
    if op == "swiglu":
        T, F, parts = case["T"], case["F"], 3 if case["keep"] else 1
        return {"bytes": T * F * (2 * BYTES[case["x"]] + parts) + parts * T * _blocks(F) * BYTES[case["scale"]],
                "flops": 8 * T * F}
    if op == "swiglu_grad":
        T, F = case["T"], case["F"]
        return {"bytes": T * F * (3 * BYTES[case["x"]] + 2) + 2 * T * _blocks(F) * BYTES[case["scale"]], "flops": 14 * T * F}
    E, N, K = case.get("E", 1), case["N"], case["K"]
    if op == "mm":
        M, scale = case["M"], BYTES[case["scale"]]
        return {"bytes": M * K + N * K + M * N * BYTES[case["out"]] + (M + _blocks(N)) * _blocks(K) * scale +
                (N * BYTES[case["out"]] if case["bias"] else 0), "flops": 2 * M * N * K}
    T = case["T"]
    used = T - T // 50 if E else T
    if op == "grouped":
        # an expert without a row is not read
        read = min(E - E // 8, used)
        return {"bytes": used * K + read * N * K + T * N * BYTES[case["out"]] +
                (used + read * _blocks(N)) * _blocks(K) * BYTES[case["scale"]], "flops": 2 * used * N * K}
    return {"bytes": used * (K + N * BYTES[case["g"]] + _blocks(K)) + max(1, E) * N * K * BYTES[case["out"]],
            "flops": 2 * used * N * K}


# ---- the same from the definitions, in 64 bits ----

def _grid(v, out):
    """The nearest value of an 8-bit type, ties to even, cut at its largest."""
    bits, low = (3, -6) if out == "e4m3fn" else (2, -14)
    exponent = torch.frexp(v)[1].long() - 1
    step = torch.exp2((exponent.clamp_min(low) - bits).double())
    return (torch.round(v / step) * step).clamp(-LARGEST[out], LARGEST[out])


def _block_of(n, device):
    return torch.arange(n, device=device) // B


def _exact_codes(x, rows, out, scale):
    """By one block of columns after the other."""
    x = x.double()
    T, n = x.shape
    values, scales = torch.empty_like(x), []
    group = torch.arange(T, device=x.device) // rows
    for c in range(0, n, B):
        v = x[:, c:c + B]
        row = torch.maximum(v.amax(1), -v.amin(1))
        most = torch.zeros(-(-T // rows), dtype=torch.float64, device=x.device).scatter_reduce_(0, group, row, "amax")
        if scale == "fp32":
            q = (most / LARGEST[out]).float().double()
        else:
            q = torch.exp2(torch.ceil(torch.log2(most / LARGEST[out])))
            q = torch.where(most > q * LARGEST[out], q * 2, torch.where(most <= q / 2 * LARGEST[out], q / 2, q))
        q = q.clamp_min(LEAST_SCALE)
        values[:, c:c + B] = _grid(v / q[group][:, None], out)
        scales.append(q)
    return values, torch.stack(scales, 1)


def _exact_values(codes, s, rows=1):
    T, n = codes.shape
    return codes.double() * s.double()[torch.arange(T, device=s.device) // rows][:, _block_of(n, s.device)]


def exact(case, seed):
    s = prepare(case, seed)
    op, f = s["op"], torch.float64
    if op == "quant":
        if case["E"] == 1:
            return _exact_codes(s["v"], case["rows"], case["out"], case["scale"])
        parts = [_exact_codes(v, case["rows"], case["out"], case["scale"]) for v in s["v"]]
        return tuple(torch.stack(p) for p in zip(*parts))
    if op == "swiglu":
        gate, up = s["gate"].to(f), s["up"].to(f)
        h, q = _exact_codes(torch.sigmoid(gate) * gate * up, 1, case["out"], case["scale"])
        got = [h * q[:, _block_of(case["F"], q.device)]]
        if case["keep"]:
            kept = [_exact_codes(v, 1, case["out"], case["scale"]) for v in (gate, up)]
            got += [torch.cat([k[0] for k in kept], 1), torch.cat([k[1] for k in kept], 1)]
        return got
    if op == "swiglu_grad":
        F, blocks = case["F"], _blocks(case["F"])
        gate = _exact_values(s["kept"][:, :F], s["kept_scale"][:, :blocks])
        up = _exact_values(s["kept"][:, F:], s["kept_scale"][:, blocks:])
        p, g = torch.sigmoid(gate), s["g"].to(f)
        return torch.cat([g * up * (p + gate * p * torch.sigmoid(-gate)), g * gate * p], 1)
    a = _exact_values(s["codes"], s["sa"])
    if op == "mm":
        y = torch.matmul(a, _exact_values(s["weights"], s["sw"], B).t().contiguous())
        return y if s["b"] is None else y + s["b"].to(f)
    ends = [0] + s["ends"].tolist() if s["ends"] is not None else [0, case["T"]]
    spans = list(zip(ends, ends[1:]))
    if op == "grouped":
        out = torch.zeros(case["T"], case["N"], dtype=f, device=a.device)
        for e, (first, end) in enumerate(spans):
            if end > first:
                w = _exact_values(s["weights"][e], s["sw"][e], B).t().contiguous()
                torch.matmul(a[first:end], w, out=out[first:end])
        return out
    out = torch.stack([torch.matmul(s["grad"][first:end].to(f).t().contiguous(), a[first:end]) for first, end in spans])
    return out if case["E"] else out[0]
