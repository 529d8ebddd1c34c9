"""The measured cases of the operators beside the FP8 product: the residual's
addition with the RMS norm and an 8-bit output (and its gradient), the int8
product with scales per token and channel, and the log probabilities of given
tokens with entropy and top alternatives (and their gradient).

`run` computes them in plain torch operations in 32 bits, or, where `own` is
true, through this package's public calls."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "int8": torch.int8, "e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3fn": 1, "e5m2": 1}
QMAX = {"int8": 127.0, "e4m3fn": 448.0, "e5m2": 57344.0}
LEAST_SCALE = 2.0 ** -126
EPS = 1e-6


def listed():
    return [
        # one decoded token entering a layer: latency
        {"name": "norm_one_token", "op": "norm", "T": 1, "n": 4096, "x": "bf16", "res": "bf16", "out": "e4m3fn",
         "given": False},
        # a prompt with an odd number of tokens, at the projection's width, for the int8 product
        {"name": "norm_prompt_int8", "op": "norm", "T": 2047, "n": 1920, "x": "bf16", "res": "fp32", "out": "int8",
         "given": False},
        # a packed batch of prompts; one calibrated scale, as the FP8 product takes it
        {"name": "norm_batch", "op": "norm", "T": 16384, "n": 8192, "x": "bf16", "res": "bf16", "out": "e4m3fn",
         "given": True},
        # a short training batch, an odd width, the residual stream in 32 bits
        {"name": "norm_grad_odd", "op": "norm_grad", "T": 1023, "n": 1925, "g": "bf16", "h": "fp32", "gh": True},
        # a training batch of a wide model
        {"name": "norm_grad_batch", "op": "norm_grad", "T": 8192, "n": 8192, "g": "bf16", "h": "bf16", "gh": True},
        # one decoded token through the projection: the weights are read once
        {"name": "mm_one_token", "op": "mm", "M": 1, "N": 5760, "K": 1920, "out": "bf16", "bias": False},
        # a chunk of a prompt, ragged, with a bias
        {"name": "mm_chunk", "op": "mm", "M": 250, "N": 4096, "K": 4096, "out": "fp16", "bias": True},
        # the benchmark's square
        {"name": "mm_square", "op": "mm", "M": 8192, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # one decoded token under a grammar that masks a third of an odd vocabulary
        {"name": "logp_one_token", "op": "logp", "T": 1, "V": 50257, "z": "bf16", "C": 1, "k": 20, "masked": True},
        # scoring a batch of prompts over a large vocabulary
        {"name": "logp_batch", "op": "logp", "T": 4096, "V": 131072, "z": "bf16", "C": 1, "k": 5, "masked": False},
        # a policy's update on a short batch, an odd vocabulary, logits in 32 bits
        {"name": "logp_grad_odd", "op": "logp_grad", "T": 509, "V": 32001, "z": "fp32", "C": 1, "k": 0},
        # a policy's update on a training batch
        {"name": "logp_grad_batch", "op": "logp_grad", "T": 4096, "V": 65536, "z": "bf16", "C": 1, "k": 0},
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of low..high, odd or round."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.4 and v >= 64:
        v = v // 64 * 64
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "mm", "mm", "logp", "logp_grad"])
    while True:
        if op == "norm":
            x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            c = {"op": op, "T": _log(rng, 1, 16384), "n": _log(rng, 64, 16384), "x": x,
                 "res": rng.choice([x, x, "fp32", "none"]), "out": rng.choice(["e4m3fn", "e5m2", "int8"]),
                 "given": rng.random() < 0.4}
            fits = c["T"] * c["n"] <= 2 ** 26
        elif op == "norm_grad":
            g = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            c = {"op": op, "T": _log(rng, 1, 8192), "n": _log(rng, 64, 16384), "g": g,
                 "h": rng.choice([g, g, "fp32"]), "gh": rng.random() < 0.7}
            fits = c["T"] * c["n"] <= 2 ** 25
        elif op == "mm":
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 64, 16384),
                 "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "bias": rng.random() < 0.3}
            fits = c["M"] * c["N"] * c["K"] <= 2 ** 38
        else:
            z = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            c = {"op": op, "T": _log(rng, 1, 4096), "V": _log(rng, 512, 262144), "z": z,
                 "C": rng.choice([1, 1, 1, 4]), "k": rng.choice([0, 1, 5, 20])}
            if op == "logp":
                c["masked"] = rng.random() < 0.3
            fits = c["T"] * c["V"] <= 2 ** 27
        if fits:
            return c


def _normal(gen, shape, std=1.0, dtype=torch.float32):
    """Normal values, made in slices so that the largest case needs no copy of itself in 32 bits."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    rows = max(1, 2 ** 26 // max(1, shape[-1]))
    if len(shape) == 1 or dtype == torch.float32:
        return out.copy_(torch.randn(shape, generator=gen, device="cuda").mul_(std))
    for i in range(0, shape[0], rows):
        part = out[i:i + rows]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(std))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op, s = case["op"], dict(case)
    if op in ("norm", "norm_grad"):
        T, n = case["T"], case["n"]
        # a residual stream has a few channels far above the rest
        loud = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
        s["weight"] = (1.0 + _normal(gen, (n,), 0.2)).to(DTYPES[case["x" if op == "norm" else "g"]])
        if op == "norm":
            s["x"] = _normal(gen, (T, n), 0.7, DTYPES[case["x"]])
            s["res"] = None
            if case["res"] != "none":
                s["res"] = _normal(gen, (T, n), 1.5, DTYPES[case["res"]]).mul_(loud.to(DTYPES[case["res"]]))
            # a scale that a calibration run would have left: it clips a few values in ten thousand
            s["scale"] = torch.full((1,), 10.0 / QMAX[case["out"]], device="cuda") if case["given"] else None
        else:
            s["g"] = _normal(gen, (T, n), 1e-2, DTYPES[case["g"]])
            s["h"] = _normal(gen, (T, n), 1.5, DTYPES[case["h"]]).mul_(loud.to(DTYPES[case["h"]]))
            s["gh"] = _normal(gen, (T, n), 1e-2, DTYPES[case["g"]]) if case["gh"] else None
    elif op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"] = _normal(gen, (M, K), 30.0, torch.float16).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = _normal(gen, (N, K), 35.0, torch.float16).round_().clamp_(-127, 127).to(torch.int8)
        s["sa"] = torch.rand(M, 1, generator=gen, device="cuda") * 0.05 + 0.01
        s["sw"] = torch.rand(1, N, generator=gen, device="cuda") * 2e-3 + 1e-4
        s["bias"] = _normal(gen, (N,), 1.0, DTYPES[case["out"]]) if case["bias"] else None
    else:
        T, V, C = case["T"], case["V"], case["C"]
        z = _normal(gen, (T, V), 2.5, DTYPES[case["z"]])
        tokens = torch.randint(0, V, (T, C), generator=gen, device="cuda")
        # the text's own token is mostly a likely one
        lift = torch.rand(T, 1, generator=gen, device="cuda").mul_(16.0).to(z.dtype)
        z.scatter_add_(1, tokens[:, :1], lift)
        if case.get("masked"):
            hidden = torch.rand(V, generator=gen, device="cuda") < 1 / 3
            z.masked_fill_(hidden, -math.inf)
            z.scatter_(1, tokens[:, :1], lift)
        # positions of a padded batch have no token
        pad = (torch.rand(T, C, generator=gen, device="cuda") < 0.03) & (torch.arange(T, device="cuda") > 0)[:, None]
        s["z"], s["tokens"] = z, tokens.masked_fill(pad, -1)
        if op == "logp_grad":
            s["g"] = torch.randn(T, C, generator=gen, device="cuda")
            s["gH"] = torch.randn(T, generator=gen, device="cuda") * 0.01
            # what the forward call left: the log of the sum, the entropy and the alternatives
            s["lse"], s["H"] = _lse_entropy(z)
            s["top"] = torch.stack([(torch.arange(T, device="cuda") * 31 + 7 * i) % V for i in range(case["k"])], 1) \
                if case["k"] else None
            s["gtop"] = torch.randn(T, case["k"], generator=gen, device="cuda") if case["k"] else None
    return s


def _lse_entropy(z):
    """What a forward call hands to the backward one, by rows in slices."""
    lse, ent = [], []
    rows = max(1, 2 ** 26 // z.shape[1])
    for i in range(0, z.shape[0], rows):
        lp = torch.log_softmax(z[i:i + rows].double(), 1)
        lse.append((z[i:i + rows, 0].double() - lp[:, 0]).float())
        ent.append(-(lp.exp() * lp).nan_to_num_(nan=0.0).sum(1).float())
    return torch.cat(lse), torch.cat(ent)


def _values(q, scale):
    """The numbers that int8 codes and their rows' scales stand for."""
    return torch.mul(q, scale, out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))


# ---- the plain forms ----

def _norm(s):
    v = s["x"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    y = v * rstd * s["weight"].float()
    q = QMAX[s["out"]]
    scale = s["scale"] if s["scale"] is not None else (y.abs().amax(1, keepdim=True) / q).clamp_min(LEAST_SCALE)
    y = (y / scale).clamp(-q, q)
    codes = torch.round(y).to(torch.int8) if s["out"] == "int8" else y.to(DTYPES[s["out"]])
    return codes, scale, None if s["res"] is None else v.to(s["res"].dtype)


def _norm_grad(s):
    g, h, w = s["g"].float(), s["h"].float(), s["weight"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * rstd
    u = g * w
    d = rstd * (u - n * (u * n).mean(1, keepdim=True))
    if s["gh"] is not None:
        d = d + s["gh"].float()
    return d.to(s["g"].dtype), (g * n).sum(0).to(s["weight"].dtype)


def _mm(s):
    y = (s["a"].float() @ s["w"].float().t()) * s["sa"] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(DTYPES[s["out"]])


def _logp(s):
    z, t, k = s["z"].float(), s["tokens"], s["k"]
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    ent = log_total - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total
    lse = m + log_total
    lp = z.gather(1, t.clamp_min(0)) - lse
    out = [torch.where(t < 0, 0.0, lp), ent[:, 0], lse[:, 0]]
    if k:
        # one whole number orders value first and lower index before higher
        bits = (z + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32
        key += 2 ** 32 - 1 - torch.arange(z.shape[1], device=z.device)
        top = 2 ** 32 - 1 - (torch.topk(key, k, 1).values & (2 ** 32 - 1))
        out += [z.gather(1, top) - lse, top]
    return tuple(out)


def _logp_grad(s):
    z, t = s["z"].float(), s["tokens"]
    g = torch.where(t < 0, 0.0, s["g"])
    lp = z - s["lse"][:, None]
    p = torch.exp(lp)
    total = g.sum(1, keepdim=True)
    if s["top"] is not None:
        total = total + s["gtop"].sum(1, keepdim=True)
    d = -p * (total + s["gH"][:, None] * (lp + s["H"][:, None]))
    d.scatter_add_(1, t.clamp_min(0), g)
    if s["top"] is not None:
        d.scatter_add_(1, s["top"], s["gtop"])
    return d.to(s["z"].dtype)


def run(state):
    s, op = state, state["op"]
    if own:
        import bit_exact_fp8_amd as fw
        if op == "norm":
            q, scale, h = fw.add_rms_norm_quant(s["x"], s["weight"], s["res"], eps=EPS, out_dtype=DTYPES[s["out"]],
                                                scale=s["scale"])
        elif op == "norm_grad":
            return fw.add_rms_norm_backward(s["g"], s["h"], s["weight"], eps=EPS, grad_h=s["gh"])
        elif op == "mm":
            return fw.int8_scaled_mm(s["a"], s["w"].t(), s["sa"], s["sw"], bias=s["bias"],
                                     out_dtype=DTYPES[s["out"]])
        elif op == "logp":
            r = fw.token_logprobs(s["z"], s["tokens"], top_k=s["k"])
            return (r.logprobs, r.entropy, r.lse) + ((r.top_logprobs, r.top_tokens) if s["k"] else ())
        else:
            return fw.token_logprobs_backward(s["z"], s["tokens"], s["lse"], s["H"], s["g"], s["gH"],
                                              top_tokens=s["top"], grad_top=s["gtop"])
    elif op == "norm":
        q, scale, h = _norm(s)
    else:
        return {"norm_grad": _norm_grad, "mm": _mm, "logp": _logp, "logp_grad": _logp_grad}[op](s)
    return [_values(q, scale) if s["out"] == "int8" else q, scale] + ([] if h is None else [h])


def work(case):
    op = case["op"]
    if op == "norm":
        T, n, e = case["T"], case["n"], BYTES[case["x"]]
        r = 0 if case["res"] == "none" else BYTES[case["res"]]
        return {"bytes": T * n * (e + 2 * r + 1) + n * e + 4 * T, "flops": 6 * T * n}
    if op == "norm_grad":
        T, n, e, r = case["T"], case["n"], BYTES[case["g"]], BYTES[case["h"]]
        return {"bytes": T * n * (e * (3 if case["gh"] else 2) + r) + 2 * n * e, "flops": 10 * T * n}
    if op == "mm":
        M, N, K, e = case["M"], case["N"], case["K"], BYTES[case["out"]]
        return {"bytes": M * K + N * K + M * N * e + 4 * (M + N) + (N * e if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, V, C, k, e = case["T"], case["V"], case["C"], case["k"], BYTES[case["z"]]
    if op == "logp":
        return {"bytes": T * V * e + T * (12 * C + 8 + 12 * k), "flops": 6 * T * V}
    return {"bytes": 2 * T * V * e + T * (12 * C + 12 + 12 * k), "flops": 6 * T * V}


# ---- the same from the definitions, in 64 bits ----

def _grid(v, out):
    """The nearest value of an 8-bit type, ties to even, cut at its largest."""
    if out == "int8":
        return torch.round(v).clamp(-127, 127)
    bits, low = (3, -6) if out == "e4m3fn" else (2, -14)
    exponent = torch.frexp(v)[1].long() - 1
    step = torch.exp2((exponent.clamp_min(low) - bits).double())
    return (torch.round(v / step) * step).clamp(-QMAX[out], QMAX[out])


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f = torch.float64
    if op == "norm":
        v = s["x"].to(f)
        if s["res"] is not None:
            v += s["res"].to(f)
        y = v / (v.pow(2).sum(1, keepdim=True) / case["n"] + EPS).sqrt() * s["weight"].to(f)
        scale = s["scale"].to(f) if case["given"] else \
            torch.maximum(y.amax(1, keepdim=True), -y.amin(1, keepdim=True)).div(QMAX[case["out"]]).clamp_min(LEAST_SCALE)
        q = _grid(y / scale, case["out"])
        return [q * scale if case["out"] == "int8" else q, scale] + ([] if s["res"] is None else [v])
    if op == "norm_grad":
        g, h, w = s["g"].to(f), s["h"].to(f), s["weight"].to(f)
        m = h.pow(2).sum(1, keepdim=True) / case["n"] + EPS
        dot = (g * w * h).sum(1, keepdim=True)
        d = g * w / m.sqrt() - h * dot / (case["n"] * m ** 1.5)
        return (d if s["gh"] is None else d + s["gh"].to(f)), (g * h / m.sqrt()).sum(0)
    if op == "mm":
        y = torch.matmul(s["a"].to(f), s["w"].to(f).t().contiguous())
        y = y * (s["sa"].to(f) * s["sw"].to(f))
        return y if s["bias"] is None else y + s["bias"].to(f)
    parts, rows = [], max(1, 2 ** 26 // case["V"])
    for i in range(0, case["T"], rows):
        z, t = s["z"][i:i + rows].to(f), s["tokens"][i:i + rows]
        if op == "logp":
            lse = torch.logsumexp(z, 1, keepdim=True)
            lp = z - lse
            given = torch.where(t < 0, torch.zeros((), dtype=f, device="cuda"), lp.gather(1, t.clamp_min(0)))
            part = [given, torch.special.entr(lp.exp()).sum(1), lse[:, 0]]
            if case["k"]:
                order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["k"]]
                part += [lp.gather(1, order), order]
        else:
            # the gradient's definition, with the same saved log-sum and entropy
            p = torch.exp(z - s["lse"][i:i + rows, None].to(f))
            hot = torch.zeros_like(z).scatter_add_(1, t.clamp_min(0), torch.where(t < 0, 0.0, s["g"][i:i + rows]).to(f))
            if case["k"]:
                hot.scatter_add_(1, s["top"][i:i + rows], s["gtop"][i:i + rows].to(f))
            part = [hot - p * hot.sum(1, keepdim=True) + s["gH"][i:i + rows, None].to(f) *
                    (torch.special.entr(p) - p * s["H"][i:i + rows, None].to(f))]
        parts.append(part)
    whole = [torch.cat(c) for c in zip(*parts)]
    return tuple(whole) if op == "logp" else whole[0]
