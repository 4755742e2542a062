"""The float training operators' cases: what is timed and compared for each of them.

The operators are those that train a float residual MLP block beside the integer layers: the
matrix product with bias, activation and residual (forward and backward), layer norm (forward
and backward), the log probabilities of given tokens with their entropy and top alternatives
(forward and backward), and the AdamW step over many tensors with states in 32 or 8 bits.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, where
`own` is true, through the library's entry points; `exact` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SEED = 20177        # of the 8-bit states' stochastic rounding
BLOCK = 128         # elements of an 8-bit state that share an exponent
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01
START = 100         # steps that the states have behind them


def listed():
    return [
        # one token's layer while answering: latency and the weights' bytes
        dict(name="linear fwd 1 token", op="linear_fwd", b=1, ic=4096, oc=4096, type="bf16", act="gelu", bias=True,
             residual=True, z=False),
        # a layer of the 4096-wide MLP on a full training batch, keeping what the backward pass needs
        dict(name="linear fwd 8192", op="linear_fwd", b=8192, ic=4096, oc=4096, type="bf16", act="gelu", bias=True,
             residual=True, z=True),
        # a ragged batch through a layer whose rows are not 16-byte multiples
        dict(name="linear fwd odd", op="linear_fwd", b=333, ic=787, oc=1000, type="f16", act="silu", bias=True,
             residual=False, z=True),
        # the backward pass of such a layer on a quarter of the batch
        dict(name="linear bwd 2048", op="linear_bwd", b=2048, ic=4096, oc=4096, type="bf16", act="gelu", bias=True),
        # a few rows of an odd width in 32 bits: latency
        dict(name="layer norm fwd odd", op="layer_norm_fwd", rows=3, cols=787, type="f32"),
        # the norm before a 4096-wide layer on the full batch, and its backward pass
        dict(name="layer norm fwd 8192", op="layer_norm_fwd", rows=8192, cols=4096, type="bf16"),
        dict(name="layer norm bwd 8192", op="layer_norm_bwd", rows=8192, cols=4096, type="bf16"),
        # one answer over a large vocabulary with its alternatives: latency
        dict(name="logprobs fwd 1 token", op="logprobs_fwd", rows=1, classes=131072, type="bf16", k=8, masked=False),
        # the labels' log probabilities of a training batch
        dict(name="logprobs fwd 4096", op="logprobs_fwd", rows=4096, classes=32768, type="bf16", k=4, masked=False),
        # the loss's gradient, classes padded with masked ones, an odd row length
        dict(name="logprobs bwd odd", op="logprobs_bwd", rows=2047, classes=50001, type="f32", masked=True),
        # one step of a small model's 14 tensors: latency
        dict(name="adamw 32 small", op="adamw", width=64, depth=2, classes=10, bits=32, grad="f32"),
        # one step of four 4096-wide residual blocks, states in 8 bits
        dict(name="adamw 8 large", op="adamw", width=4096, depth=4, classes=1000, bits=8, grad="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd ones as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear_fwd", "linear_bwd", "layer_norm_fwd", "layer_norm_bwd", "logprobs_fwd", "logprobs_bwd",
                     "adamw"))
    if op in ("linear_fwd", "linear_bwd"):
        while True:
            b, ic, oc = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 10, 8192)
            if rng.random() < 0.5:
                ic, oc = max(64, ic // 64 * 64), max(64, oc // 64 * 64)
            if b * ic * oc <= (2 if op == "linear_bwd" else 4) << 35:
                break
        case = dict(op=op, b=b, ic=ic, oc=oc, type=rng.choice(("bf16", "f16")), act=rng.choice(ACTS),
                    bias=rng.random() < 0.7)
        if op == "linear_fwd":
            case.update(residual=rng.random() < 0.5, z=rng.random() < 0.5)
        return case
    if op in ("layer_norm_fwd", "layer_norm_bwd"):
        while True:
            rows, cols = _log(rng, 1, 65536), _log(rng, 16, 16384)
            if rows * cols <= 8192 * 4096:
                return dict(op=op, rows=rows, cols=cols, type=rng.choice(("f32", "bf16", "f16")))
    if op in ("logprobs_fwd", "logprobs_bwd"):
        while True:
            rows, classes = _log(rng, 1, 8192), _log(rng, 10, 160000)
            if rows * classes <= (4096 * 32768 if op == "logprobs_fwd" else 2047 * 50001):
                break
        case = dict(op=op, rows=rows, classes=classes, type=rng.choice(("f32", "bf16", "f16")),
                    masked=rng.random() < 0.3)
        if op == "logprobs_fwd":
            case["k"] = min(classes, rng.choice((0, 1, 2, 5, 8, 20, 32)))
        return case
    while True:
        width, depth, classes = _log(rng, 16, 4096), rng.randint(1, 12), _log(rng, 2, 32768)
        if 2 * width * width * depth + width * classes <= 2 * 4096 * 4096 * 4:
            return dict(op=op, width=width, depth=depth, classes=classes, bits=rng.choice((32, 8)),
                        grad=rng.choice(("f32", "bf16", "f16")))


def _shapes(case):
    """The parameter tensors of a residual MLP: per block a norm and two square layers, then the classes."""
    w = case["width"]
    return [(w,), (w,), (w, w), (w,), (w, w), (w,)] * case["depth"] + [(case["classes"], w), (case["classes"],)]


def _sizes(case):
    return [math.prod(s) for s in _shapes(case)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op = case["op"]

    def normal(shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(dtype)

    s = {"case": case}
    if op in ("linear_fwd", "linear_bwd"):
        b, ic, oc, t = case["b"], case["ic"], case["oc"], TYPES[case["type"]]
        s["x"] = normal((b, ic), 1.0, t)
        s["w"] = normal((oc, ic), ic ** -0.5, t)
        if op == "linear_fwd":
            s["bias"] = normal((oc,), 0.1, t) if case["bias"] else None
            s["residual"] = normal((b, oc), 1.0, t) if case["residual"] else None
        else:
            s["z"] = normal((b, oc), 1.0, t) if case["act"] != "none" else None
            s["dy"] = normal((b, oc), 1.0, t)
    elif op in ("layer_norm_fwd", "layer_norm_bwd"):
        rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]
        s["x"] = (normal((rows, cols), 1.5) + normal((rows, 1), 0.5)).to(t)
        s["gamma"] = 1.0 + normal((cols,), 0.1)
        s["beta"] = normal((cols,), 0.1)
        if op == "layer_norm_bwd":
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + 1e-5)
            s["dy"] = normal((rows, cols), 1.0, t)
    elif op in ("logprobs_fwd", "logprobs_bwd"):
        rows, classes, t = case["rows"], case["classes"], TYPES[case["type"]]
        x = normal((rows, classes), 2.5, t)
        tgt = torch.randint(0, classes, (rows,), generator=gen, device=DEVICE, dtype=torch.int32)
        if case["masked"]:       # padding classes at the end, a row that the mask leaves nothing, a row without a token
            x[:, classes - classes // 8:] = -math.inf
            tgt %= max(1, classes - classes // 8)
            x[rows // 3] = -math.inf
            tgt[rows // 2] = -1
        s["logits"], s["targets"] = x, tgt
        if op == "logprobs_bwd":
            xf = x.float()
            top = xf.amax(1)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            e = torch.exp(xf - top[:, None])
            total = e.sum(1)
            s["lse"] = top + torch.log(total)
            shifted = torch.where(e > 0, (xf - top[:, None]) * e, torch.zeros_like(e)).sum(1)
            s["entropy"] = torch.where(total > 0, torch.log(total) - shifted / total, torch.zeros_like(total))
            s["g_logp"] = -torch.rand((rows,), generator=gen, device=DEVICE) / rows
            s["g_entropy"] = normal((rows,), 0.1 / rows)
    else:
        n, sizes = sum(_sizes(case)), _sizes(case)
        s["w"] = normal((n,), 0.02)
        s["g"] = normal((n,), 1e-3, TYPES[case["grad"]])
        s["copy"] = s["w"].to(torch.bfloat16)
        s["steps"] = START
        blocks = [-(-k // BLOCK) for k in sizes]
        if case["bits"] == 32:
            s["m"] = normal((n,), 3e-4)
            s["v"] = normal((n,), 1e-3).square()
        else:                    # codes and shared exponents as the steps before leave them
            s["m"] = torch.randint(0, 256, (n,), generator=gen, device=DEVICE, dtype=torch.int32).to(torch.uint8)
            s["v"] = torch.randint(200, 256, (n,), generator=gen, device=DEVICE, dtype=torch.int32).to(torch.uint8)
            s["m_exp"] = torch.randint(-12, -9, (sum(blocks),), generator=gen, device=DEVICE).to(torch.int8)
            s["v_exp"] = torch.randint(-20, -17, (sum(blocks),), generator=gen, device=DEVICE).to(torch.int8)
        if own:
            import integer_only_nn_gb300 as ito

            def cut(t, lengths):
                return list(torch.split(t, lengths))

            state = [cut(s["m"], sizes), cut(s["v"], sizes)]
            if case["bits"] == 8:
                state += [cut(s["m_exp"], blocks), cut(s["v_exp"], blocks)]
            s["grads"] = cut(s["g"], sizes)
            s["optimizer"] = ito.AdamW(cut(s["w"], sizes), bits=case["bits"], betas=(BETA1, BETA2), eps=EPS,
                                       weight_decay=DECAY, copies=cut(s["copy"], sizes), states=state, step=START,
                                       seed=SEED)
        elif case["bits"] == 8:  # where each tensor's elements and blocks lie in the flat buffers
            s["where"] = _where(sizes)
    return s


def _where(sizes):
    """Per element of the flat buffers: its block, its index in its tensor and its tensor's number."""
    n = torch.tensor(sizes, device=DEVICE)
    first = torch.cumsum(n, 0) - n
    blocks = (n + BLOCK - 1) // BLOCK
    first_block = torch.cumsum(blocks, 0) - blocks
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEVICE), n)
    index = torch.arange(int(n.sum()), device=DEVICE) - first[tensor]
    return first_block[tensor] + index // BLOCK, index, tensor


# ------------------------------------------------------------ plain forms

def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    return torch.ones_like(z)


def _plain_linear_fwd(s, c):
    t = TYPES[c["type"]]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(t), "z": z.to(t)} if c["z"] else {"y": y.to(t)}


def _plain_linear_bwd(s, c):
    t = TYPES[c["type"]]
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(c["act"], s["z"].float())
    r = {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.T @ s["x"].float()).to(t)}
    if c["bias"]:
        r["dbias"] = dz.sum(0)
    return r


def _plain_layer_norm_fwd(s, c):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + 1e-5)
    return {"y": (d * rstd[:, None] * s["gamma"] + s["beta"]).to(TYPES[c["type"]]), "mean": mean, "rstd": rstd}


def _plain_layer_norm_bwd(s, c):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (s["x"].float() - s["mean"][:, None]) * rstd
    a = dy * s["gamma"]
    dx = (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True)) * rstd
    return {"dx": dx.to(TYPES[c["type"]]), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}


def _plain_logprobs_fwd(s, c):
    x, tgt = s["logits"].float(), s["targets"].long()
    top = x.amax(1)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    d = x - top[:, None]
    e = torch.exp(d)
    total = e.sum(1)
    lse = top + torch.log(total)
    shifted = torch.where(e > 0, d * e, torch.zeros_like(e)).sum(1)
    entropy = torch.where(total > 0, torch.log(total) - shifted / total, torch.zeros_like(total))
    empty = torch.full_like(lse, -math.inf)
    logp = torch.where(total > 0, x.gather(1, tgt.clamp(min=0)[:, None])[:, 0] - lse, empty)
    logp = torch.where(tgt >= 0, logp, torch.zeros_like(logp))
    # keys whose order is the values' (largest first) and among equal values the index's (lowest first)
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    ids = torch.arange(x.shape[1], device=x.device)
    keys = order * (1 << 32) + ((1 << 31) - ids)
    ids = torch.topk(keys, c["k"], dim=1).indices if c["k"] else ids[:0].expand(x.shape[0], 0)
    top_logp = torch.where(total[:, None] > 0, x.gather(1, ids) - lse[:, None], empty[:, None])
    return {"logp": logp, "entropy": entropy, "lse": lse, "top_ids": ids.to(torch.int32), "top_logp": top_logp}


def _plain_logprobs_bwd(s, c):
    x, tgt, lse = s["logits"].float(), s["targets"].long(), s["lse"][:, None]
    some = lse > -math.inf
    lp = torch.where(some & (x > -math.inf), x - lse, torch.zeros_like(x))
    p = torch.where(some & (x > -math.inf), torch.exp(lp), torch.zeros_like(x))
    g = torch.where(tgt >= 0, s["g_logp"], torch.zeros_like(s["g_logp"]))[:, None]
    hot = (torch.arange(x.shape[1], device=x.device) == tgt[:, None]) & some
    dx = g * (hot.float() - p) - s["g_entropy"][:, None] * p * (lp + s["entropy"][:, None])
    return {"dlogits": dx.to(TYPES[c["type"]])}


def _random(index, tensor, step):
    """The 32-bit words of the states' stochastic rounding: a mix of seed, step, tensor and element."""
    m32 = 0xFFFFFFFF
    h = (SEED + step * 0x9E3779B1 + tensor * 0x510E527F) & m32
    h = ((index & m32) * 0x6A09E667 + (index >> 32) * 0xBB67AE85 + h) & m32
    h = h ^ (h >> 16)
    h = (h * 0xBB67AE85) & m32
    h = h ^ (h >> 15)
    h = (h * 0x6A09E667) & m32
    h = h ^ (h >> 16)
    return h & 0xFFFFF, ((h * 0x510E527F) & m32) >> 12


def _unpack(code, exp, block, signed):
    c, e = code.to(torch.int32), exp[block].to(torch.int32)
    mag = c & 127 if signed else c
    value = (((e + (112 if signed else 96)) << 23) + (mag << 20)).view(torch.float32)
    value = torch.where(mag > 0, value, torch.zeros_like(value))
    if signed:
        value = torch.where(c >= 128, -value, value)
    return torch.where(e == -128, torch.full_like(value, math.nan), value)


def _pack(x, block, blocks, rnd, signed):
    bits = x.view(torch.int32).long()
    mag = bits & 0x7FFFFFFF
    top = torch.zeros(blocks, dtype=torch.int64, device=x.device).scatter_reduce(0, block, mag, "amax")
    bad = top >= 0x7F800000
    top = torch.clamp(top, max=0x7F700000)
    low = -111 if signed else -95
    exp = torch.clamp(((top + 0xFFFFF) >> 23) - 127, min=low)
    t = torch.clamp(mag, max=0x7F700000) - ((exp[block] + (112 if signed else 96)) << 23)
    code = torch.where(t >= 0, (t + rnd) >> 20, torch.zeros_like(t))
    if signed:
        code = torch.where((bits != mag) & (code > 0), code + 128, code)
    else:
        code = torch.where(mag > 0, torch.clamp(code, min=1), code)
    exp = torch.where(bad, torch.full_like(exp, -128), exp)
    code = torch.where(bad[block], torch.zeros_like(code), code)
    return code.to(torch.uint8), exp.to(torch.int8)


def _f32(v):
    return float(np.float32(v))


def _plain_adamw(s, c):
    s["steps"] += 1
    t, small = s["steps"], c["bits"] == 8
    g = s["g"].float()
    m, v = s["m"], s["v"]
    if small:
        block, index, tensor = s["where"]
        m, v = _unpack(m, s["m_exp"], block, True), _unpack(v, s["v_exp"], block, False)
    m = m * _f32(BETA1) + g * _f32(1 - BETA1)
    v = v * _f32(BETA2) + (g * g) * _f32(1 - BETA2)
    den = torch.sqrt(v) * _f32(1 / math.sqrt(1 - BETA2 ** t)) + _f32(EPS)
    w = s["w"] * _f32(1 - LR * DECAY) - (m * _f32(LR / (1 - BETA1 ** t))) / den
    s["w"].copy_(w)
    s["copy"].copy_(w)
    if small:
        rnd_m, rnd_v = _random(index, tensor, t)
        mc, me = _pack(m, block, s["m_exp"].numel(), rnd_m, True)
        vc, ve = _pack(v, block, s["v_exp"].numel(), rnd_v, False)
        for key, value in (("m", mc), ("v", vc), ("m_exp", me), ("v_exp", ve)):
            s[key].copy_(value)
        m = _unpack(mc, me, block, True).to(torch.bfloat16)      # exact: a code has four significant bits
        v = _unpack(vc, ve, block, False).to(torch.bfloat16)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return {"w": s["w"], "copy": s["copy"], "m": m, "v": v}


PLAIN = {"linear_fwd": _plain_linear_fwd, "linear_bwd": _plain_linear_bwd, "layer_norm_fwd": _plain_layer_norm_fwd,
         "layer_norm_bwd": _plain_layer_norm_bwd, "logprobs_fwd": _plain_logprobs_fwd,
         "logprobs_bwd": _plain_logprobs_bwd, "adamw": _plain_adamw}


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](state, c)
    import integer_only_nn_gb300 as ito
    if op == "linear_fwd":
        r = ito.ito_fp_linear_fwd(state["x"], state["w"], bias=state["bias"], act=c["act"], residual=state["residual"],
                                  save_z=c["z"])
        return {"y": r[0], "z": r[1]} if c["z"] else {"y": r}
    if op == "linear_bwd":
        dx, dw, dbias = ito.ito_fp_linear_bwd(state["dy"], state["x"], state["w"], z=state["z"], act=c["act"],
                                              need_dbias=c["bias"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if c["bias"] else {"dx": dx, "dw": dw}
    if op == "layer_norm_fwd":
        y, mean, rstd = ito.ito_layer_norm_fwd(state["x"], state["gamma"], state["beta"], eps=1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layer_norm_bwd":
        dx, dgamma, dbeta = ito.ito_layer_norm_bwd(state["dy"], state["x"], state["gamma"], state["mean"], state["rstd"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "logprobs_fwd":
        logp, entropy, lse, ids, top = ito.ito_token_logprobs_fwd(state["logits"], state["targets"], k=c["k"])
        return {"logp": logp, "entropy": entropy, "lse": lse, "top_ids": ids, "top_logp": top}
    if op == "logprobs_bwd":
        return {"dlogits": ito.ito_token_logprobs_bwd(state["logits"], state["targets"], state["lse"], state["entropy"],
                                                      state["g_logp"], state["g_entropy"])}
    opt = state["optimizer"]
    opt.step(state["grads"], lr=LR)
    m, v = (state["m"], state["v"]) if c["bits"] == 32 else opt.moments()
    return {"w": state["w"], "copy": state["copy"], "m": m, "v": v}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op in ("linear_fwd", "linear_bwd"):
        b, ic, oc = case["b"], case["ic"], case["oc"]
        if op == "linear_fwd":
            n = b * ic + oc * ic + b * oc * (1 + case["residual"] + case["z"]) + oc * case["bias"]
            return {"bytes": 2 * n, "flops": 2 * b * ic * oc}
        n = 2 * (b * ic + oc * ic) + b * oc * (2 if case["act"] != "none" else 1)
        return {"bytes": 2 * n + 4 * oc * case["bias"], "flops": 4 * b * ic * oc}
    if op in ("layer_norm_fwd", "layer_norm_bwd"):
        size = 4 if case["type"] == "f32" else 2
        rows, cols = case["rows"], case["cols"]
        if op == "layer_norm_fwd":
            return {"bytes": 2 * size * rows * cols + 8 * rows + 8 * cols, "flops": 7 * rows * cols}
        return {"bytes": 3 * size * rows * cols + 8 * rows + 12 * cols, "flops": 14 * rows * cols}
    if op in ("logprobs_fwd", "logprobs_bwd"):
        size = 4 if case["type"] == "f32" else 2
        rows, n = case["rows"], case["rows"] * case["classes"]
        if op == "logprobs_fwd":
            return {"bytes": size * n + rows * (16 + 8 * case["k"]), "flops": 6 * n}
        return {"bytes": 2 * size * n + 20 * rows, "flops": 8 * n}
    n = sum(_sizes(case))
    g = 4 if case["grad"] == "f32" else 2
    # weight read and written, gradient read, copy written, states read and written (8 bits: their values written too)
    states = 16 if case["bits"] == 32 else 4 + 4 / BLOCK + 4
    return {"bytes": n * (8 + g + 2 + states), "flops": 14 * n}


# ----------------------------------------------------------------- exact

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    return EXACT[case["op"]](s, case)


def _exact_act(name, z, slope):
    """act(z) or its slope in 64 bits, from the normal distribution function and the logistic one."""
    one = torch.ones_like(z)
    if name == "none":
        return one if slope else z
    if name == "relu":
        gate = torch.where(z > 0, one, 0 * one)
        return gate if slope else gate * z
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if slope else z * cdf
    if name == "gelu_tanh":          # (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        q = torch.sigmoid(u2)
        return q + z * q * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2) if slope else z * q
    q = torch.sigmoid(z)
    return q + z * q * torch.sigmoid(-z) if slope else z * q


def _exact_linear_fwd(s, c):
    z = torch.mm(s["x"].double(), s["w"].double().t())
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _exact_act(c["act"], z, False)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "z": z} if c["z"] else {"y": y}


def _exact_linear_bwd(s, c):
    dz = s["dy"].double()
    if c["act"] != "none":
        dz = dz * _exact_act(c["act"], s["z"].double(), True)
    r = {"dx": torch.mm(dz, s["w"].double()), "dw": torch.mm(dz.t(), s["x"].double())}
    if c["bias"]:
        r["dbias"] = dz.sum(0)
    return r


def _exact_layer_norm_fwd(s, c):
    x = s["x"].double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = (var + 1e-5) ** -0.5
    y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double())
    return {"y": y, "mean": mean, "rstd": rstd}


def _exact_layer_norm_bwd(s, c):
    dy, x, r = s["dy"].double(), s["x"].double(), s["rstd"].double()[:, None]
    h = (x - s["mean"].double()[:, None]) * r
    n = x.shape[1]
    a = s["gamma"].double() * dy
    dx = r / n * (n * a - a.sum(1, keepdim=True) - h * (a * h).sum(1, keepdim=True))
    return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, h), "dbeta": dy.sum(0)}


def _exact_logprobs_fwd(s, c):
    x = s["logits"].double()
    rows = torch.arange(x.shape[0], device=x.device)
    lse = torch.logsumexp(x, 1)
    some = lse > -math.inf
    lp = torch.where(some[:, None], x - lse[:, None], torch.full_like(x, -math.inf))
    entropy = -torch.xlogy(lp.exp(), lp.exp()).sum(1)
    tgt = s["targets"].long()
    logp = torch.where(tgt < 0, torch.zeros_like(lse), lp[rows, tgt.clamp(min=0)])
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    return {"logp": logp, "entropy": entropy, "lse": lse, "top_ids": ids.to(torch.int32), "top_logp": lp.gather(1, ids)}


def _exact_logprobs_bwd(s, c):
    x, lse, h = s["logits"].double(), s["lse"].double()[:, None], s["entropy"].double()[:, None]
    p = torch.where(lse > -math.inf, torch.exp(x - lse), torch.zeros_like(x))
    dx = -torch.where(s["targets"] >= 0, s["g_logp"].double(), 0.0)[:, None] * p
    dx -= s["g_entropy"].double()[:, None] * (torch.xlogy(p, p) + p * h)
    hit = ((s["targets"] >= 0) & (lse[:, 0] > -math.inf)).nonzero()[:, 0]
    dx[hit, s["targets"][hit].long()] += s["g_logp"][hit].double()
    return {"dlogits": dx}


def _exact_state(x, block, blocks, rnd, span, signed):
    """x rounded to eighths of a power of two with the given randoms, floored at 2^span below the block's largest."""
    a = x.abs()
    top = torch.zeros(blocks, dtype=torch.float64, device=x.device).scatter_reduce(0, block, a, "amax")
    _, e = torch.frexp(top)                       # top = f 2^e, f in [1/2, 1)
    up = torch.ceil(torch.ldexp(top, 4 - e)) >= 16
    low = e - 1 + up.to(e.dtype) - span
    floor = torch.ldexp(torch.ones_like(top), low)[block]
    _, k = torch.frexp(torch.maximum(a, floor))
    unit = torch.ldexp(torch.ones_like(a), k - 4)
    q = torch.floor(a / unit + rnd.double() / (1 << 20)) * unit
    q = torch.where((a >= floor) & (q > floor), q, torch.zeros_like(q))
    if not signed:
        q = torch.where((a > 0) & (q == 0), floor * 1.125, q)
    return torch.copysign(q, x)


def _exact_adamw(s, c):
    t = s["steps"] + 1
    g, m, v = s["g"].double(), s["m"], s["v"]
    if c["bits"] == 8:
        block, index, tensor = s["where"]
        em, ev = s["m_exp"].double()[block], s["v_exp"].double()[block]
        mi, vi = m.long(), v.long()
        lo = mi & 127
        m = torch.where(lo > 0, 1 + (lo & 7) / 8.0, 0.0).double() * 2.0 ** ((lo >> 3) - 15 + em)
        m = torch.where(mi > 127, -m, m)
        v = torch.where(vi > 0, 1 + (vi & 7) / 8.0, 0.0).double() * 2.0 ** ((vi >> 3) - 31 + ev)
    m = BETA1 * m.double() + (1 - BETA1) * g
    v = BETA2 * v.double() + (1 - BETA2) * g ** 2
    step = LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS)
    w = s["w"].double() * (1 - LR * DECAY) - step
    if c["bits"] == 8:
        rnd_m, rnd_v = _random(index, tensor, t)
        m = _exact_state(m, block, s["m_exp"].numel(), rnd_m, 15, True)
        v = _exact_state(v, block, s["v_exp"].numel(), rnd_v, 31, False)
    return {"w": w, "copy": w, "m": m, "v": v}


EXACT = {"linear_fwd": _exact_linear_fwd, "linear_bwd": _exact_linear_bwd, "layer_norm_fwd": _exact_layer_norm_fwd,
         "layer_norm_bwd": _exact_layer_norm_bwd, "logprobs_fwd": _exact_logprobs_fwd,
         "logprobs_bwd": _exact_logprobs_bwd, "adamw": _exact_adamw}
