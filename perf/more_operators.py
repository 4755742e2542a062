"""More of the float operators' cases: what a token model has at its two ends and in its block.

The operators are the gated feed-forward layer (both projections, the activation and the product;
forward and backward), the cross entropy of a linear layer over a large vocabulary without its
logits in memory (forward and backward) and the embedding lookup with its scale (forward, and the
gradient by sorted tokens).

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, where
`own` is true, through the library's entry points; `exact` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("relu", "gelu", "gelu_tanh", "silu")
LOSS_SCALE = {"bf16": 1.0, "f16": 4096.0}      # float16 gradients are small without one


def listed():
    return [
        # one token's gated layer while answering: latency and both weights' bytes
        dict(name="gated fwd 1 token", op="gated_fwd", b=1, ic=4096, oc=8192, type="bf16", act="silu", bias=False, z=False),
        # a gated layer on a training batch, keeping what the backward pass needs
        dict(name="gated fwd 4096", op="gated_fwd", b=4096, ic=4096, oc=8192, type="bf16", act="silu", bias=False, z=True),
        # a ragged batch through a layer whose rows are no 16-byte multiples, with biases
        dict(name="gated fwd odd", op="gated_fwd", b=333, ic=787, oc=1003, type="f16", act="gelu_tanh", bias=True, z=True),
        # the backward pass of such a layer on half of the batch
        dict(name="gated bwd 2048", op="gated_bwd", b=2048, ic=4096, oc=8192, type="bf16", act="silu", bias=False),
        # the loss of one token over a large vocabulary while scoring: latency and the weights' bytes
        dict(name="cross entropy fwd 1 token", op="ce_fwd", rows=1, d=4096, classes=131072, type="bf16", masked=False),
        # the loss of a training batch, and the gradients of half of it
        dict(name="cross entropy fwd 4096", op="ce_fwd", rows=4096, d=4096, classes=32768, type="bf16", masked=False),
        dict(name="cross entropy bwd 2048", op="ce_bwd", rows=2048, d=4096, classes=32768, type="bf16", masked=False),
        # a ragged batch with rows without a token, an odd vocabulary and width, a loss scale
        dict(name="cross entropy bwd odd", op="ce_bwd", rows=333, d=787, classes=50001, type="f16", masked=True),
        # a few tokens from a float32 table of an odd width: latency
        dict(name="embedding fwd odd", op="emb_fwd", n=7, d=787, classes=50001, type="f32", out="bf16", scale=1.0),
        # the input of a training batch
        dict(name="embedding fwd 16384", op="emb_fwd", n=16384, d=4096, classes=32768, type="bf16", out="bf16", scale=64.0),
        # a small batch's gradient added to that of a tied table
        dict(name="embedding bwd tied", op="emb_bwd", n=2047, d=787, classes=50001, type="bf16", scale=28.0, add=True),
        # a training batch's gradient of the whole table
        dict(name="embedding bwd 16384", op="emb_bwd", n=16384, d=4096, classes=32768, type="bf16", scale=64.0, add=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd ones as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gated_fwd", "gated_bwd", "ce_fwd", "ce_bwd", "emb_fwd", "emb_bwd"))
    if op in ("gated_fwd", "gated_bwd"):
        while True:
            b, ic, oc = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 16384)
            if rng.random() < 0.5:
                ic, oc = ic // 64 * 64, oc // 64 * 64
            if b * ic * oc <= (2048 if op == "gated_bwd" else 4096) * 4096 * 8192:
                break
        case = dict(op=op, b=b, ic=ic, oc=oc, type=rng.choice(("bf16", "f16")), act=rng.choice(ACTS),
                    bias=rng.random() < 0.3)
        if op == "gated_fwd":
            case["z"] = rng.random() < 0.5
        return case
    if op in ("ce_fwd", "ce_bwd"):
        while True:
            rows, d, classes = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 100, 160000)
            if rng.random() < 0.5:
                d, classes = d // 64 * 64, max(128, classes // 64 * 64)
            if rows * d * classes <= (2048 if op == "ce_bwd" else 4096) * 4096 * 32768 and d * classes <= 4096 * 131072:
                return dict(op=op, rows=rows, d=d, classes=classes, type=rng.choice(("bf16", "f16")),
                            masked=rng.random() < 0.3)
    while True:
        n, d, classes = _log(rng, 1, 65536), _log(rng, 16, 8192), _log(rng, 100, 160000)
        if rng.random() < 0.5:
            d = d // 16 * 16
        if n * d <= 16384 * 4096 and classes * d <= 32768 * 4096:
            case = dict(op=op, n=n, d=d, classes=classes, type=rng.choice(("f32", "bf16", "f16")),
                        scale=rng.choice((1.0, 8.0, 28.0)))
            case.update({"out": rng.choice((case["type"], "bf16"))} if op == "emb_fwd" else {"add": rng.random() < 0.4})
            return case


def _frequencies(classes):
    """How often each token comes up in text: about inversely to its rank."""
    p = 1.0 / (np.arange(classes) + 2.7)
    return p / p.sum()


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, t = case["op"], TYPES[case["type"]]

    def normal(shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(dtype)

    s = {"case": case}
    if op in ("gated_fwd", "gated_bwd"):
        b, ic, oc = case["b"], case["ic"], case["oc"]
        s["x"] = normal((b, ic))
        s["wg"], s["wu"] = normal((oc, ic), ic ** -0.5), normal((oc, ic), ic ** -0.5)
        if op == "gated_fwd":
            s["bg"] = normal((oc,), 0.1) if case["bias"] else None
            s["bu"] = normal((oc,), 0.1) if case["bias"] else None
        else:
            s["zg"], s["zu"], s["dh"] = normal((b, oc)), normal((b, oc)), normal((b, oc))
    elif op in ("ce_fwd", "ce_bwd"):
        rows, d, classes = case["rows"], case["d"], case["classes"]
        s["x"] = normal((rows, d))
        s["w"] = normal((classes, d), 2.0 * d ** -0.5)
        tgt = torch.randint(0, classes, (rows,), generator=gen, device=DEVICE, dtype=torch.int32)
        if case["masked"]:       # rows without a token: padding, prompts
            tgt = torch.where(torch.rand((rows,), generator=gen, device=DEVICE) < 0.2, torch.full_like(tgt, -1), tgt)
        s["targets"] = tgt
        if op == "ce_bwd":
            s["lse"] = _lse(s["x"].float() @ s["w"].float().T)
            s["g_loss"] = (0.5 + torch.rand((rows,), generator=gen, device=DEVICE)) * (LOSS_SCALE[case["type"]] / rows)
    else:
        n, d, classes = case["n"], case["d"], case["classes"]
        cdf = torch.from_numpy(np.cumsum(_frequencies(classes))).to(DEVICE)
        u = torch.rand((n,), generator=gen, device=DEVICE, dtype=torch.float64)
        s["ids"] = torch.searchsorted(cdf, u).clamp(max=classes - 1).to(torch.int32)
        if n > 4:
            s["ids"][n // 2] = -1            # a place without a token
        if op == "emb_fwd":
            s["table"] = normal((classes, d), 0.02)
        else:
            s["dy"] = normal((n, d), 1e-2)
            if case["add"]:
                s["grad"] = normal((classes, d), 1e-2, torch.float32)
    return s


# ------------------------------------------------------------ plain forms

def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    q = 1.0 / (1.0 + torch.exp(-z))
    return q * (1.0 + z * (1.0 - q))


def _lse(x):
    top = x.amax(1)
    return top + torch.log(torch.exp(x - top[:, None]).sum(1))


def _plain_gated_fwd(s, c):
    t, x = TYPES[c["type"]], s["x"].float()
    zg, zu = x @ s["wg"].float().T, x @ s["wu"].float().T
    if c["bias"]:
        zg, zu = zg + s["bg"].float(), zu + s["bu"].float()
    h = (_act(c["act"], zg) * zu).to(t)
    return {"h": h, "zg": zg.to(t), "zu": zu.to(t)} if c["z"] else {"h": h}


def _plain_gated_bwd(s, c):
    t, x = TYPES[c["type"]], s["x"].float()
    zg, zu, dh = s["zg"].float(), s["zu"].float(), s["dh"].float()
    dzg, dzu = dh * zu * _act_slope(c["act"], zg), dh * _act(c["act"], zg)
    dx = dzg @ s["wg"].float() + dzu @ s["wu"].float()
    r = {"dx": dx.to(t), "dwg": (dzg.T @ x).to(t), "dwu": (dzu.T @ x).to(t)}
    if c["bias"]:
        r.update(dbg=dzg.sum(0), dbu=dzu.sum(0))
    return r


def _plain_ce_fwd(s, c):
    x, tgt = s["x"].float() @ s["w"].float().T, s["targets"].long()
    lse = _lse(x)
    loss = lse - x.gather(1, tgt.clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(tgt >= 0, loss, torch.zeros_like(loss)), "lse": lse}


def _plain_ce_bwd(s, c):
    t, x, w, tgt = TYPES[c["type"]], s["x"].float(), s["w"].float(), s["targets"].long()
    dl = torch.exp(x @ w.T - s["lse"][:, None])
    g = torch.where(tgt >= 0, s["g_loss"], torch.zeros_like(s["g_loss"]))
    hot = torch.arange(w.shape[0], device=w.device) == tgt[:, None]
    dl = g[:, None] * (dl - hot.float())
    return {"dx": (dl @ w).to(t), "dw": (dl.T @ x).to(t)}


def _plain_emb_fwd(s, c):
    ids = s["ids"].long()
    y = s["table"][ids.clamp(min=0)].float() * c["scale"]
    return {"y": torch.where(ids[:, None] >= 0, y, torch.zeros_like(y)).to(TYPES[c["out"]])}


def _plain_emb_bwd(s, c):
    ids = s["ids"].long()
    dy = torch.where(ids[:, None] >= 0, s["dy"].float() * c["scale"], torch.zeros_like(s["dy"], dtype=torch.float32))
    grad = s["grad"] if c["add"] else torch.zeros((c["classes"], c["d"]), device=dy.device)
    return {"grad": grad.index_add_(0, ids.clamp(min=0), dy)}


PLAIN = {"gated_fwd": _plain_gated_fwd, "gated_bwd": _plain_gated_bwd, "ce_fwd": _plain_ce_fwd, "ce_bwd": _plain_ce_bwd,
         "emb_fwd": _plain_emb_fwd, "emb_bwd": _plain_emb_bwd}


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](state, c)
    import integer_only_nn_gb300 as ito
    if op == "gated_fwd":
        r = ito.ito_fp_gated_linear_fwd(state["x"], state["wg"], state["wu"], bias_g=state["bg"], bias_u=state["bu"],
                                        act=c["act"], save_z=c["z"])
        return {"h": r[0], "zg": r[1], "zu": r[2]} if c["z"] else {"h": r}
    if op == "gated_bwd":
        r = ito.ito_fp_gated_linear_bwd(state["dh"], state["x"], state["wg"], state["wu"], state["zg"], state["zu"],
                                        act=c["act"], need_dbias=c["bias"])
        return dict(zip(("dx", "dwg", "dwu", "dbg", "dbu"), r if c["bias"] else r[:3]))
    if op == "ce_fwd":
        loss, lse = ito.ito_linear_cross_entropy_fwd(state["x"], state["w"], state["targets"])
        return {"loss": loss, "lse": lse}
    if op == "ce_bwd":
        dx, dw = ito.ito_linear_cross_entropy_bwd(state["x"], state["w"], state["targets"], state["lse"], state["g_loss"])
        return {"dx": dx, "dw": dw}
    if op == "emb_fwd":
        return {"y": ito.ito_embedding_fwd(state["ids"], state["table"], scale=c["scale"], out_dtype=TYPES[c["out"]])}
    return {"grad": ito.ito_embedding_bwd(state["dy"], state["ids"], c["classes"], scale=c["scale"],
                                          add_to=state["grad"] if c["add"] else None)}


# ------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    size = 4 if case["type"] == "f32" else 2
    if op in ("gated_fwd", "gated_bwd"):
        b, ic, oc = case["b"], case["ic"], case["oc"]
        if op == "gated_fwd":
            n = b * ic + 2 * oc * ic + b * oc * (3 if case["z"] else 1) + 2 * oc * case["bias"]
            return {"bytes": 2 * n, "flops": 4 * b * ic * oc}
        return {"bytes": 4 * (b * ic + 2 * oc * ic) + 6 * b * oc + 8 * oc * case["bias"], "flops": 8 * b * ic * oc}
    if op in ("ce_fwd", "ce_bwd"):
        rows, d, classes = case["rows"], case["d"], case["classes"]
        n = rows * d + classes * d
        if op == "ce_fwd":
            return {"bytes": 2 * n + 12 * rows, "flops": 2 * rows * d * classes}
        return {"bytes": 4 * n + 12 * rows, "flops": 6 * rows * d * classes}
    n, d, classes = case["n"], case["d"], case["classes"]
    seen = float((1.0 - (1.0 - _frequencies(classes)) ** n).sum())       # distinct tokens to be expected
    if op == "emb_fwd":
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": int(seen * d * size) + n * d * out + 4 * n, "flops": n * d}
    rows = 2 * seen if case["add"] else classes
    return {"bytes": n * d * size + int(rows * d * 4) + 4 * n, "flops": 2 * n * d}


# ----------------------------------------------------------------- exact

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    return EXACT[case["op"]](s, case)


def _exact_act(name, z):
    """act(z) and its slope in 64 bits, from the normal distribution function and the logistic one."""
    if name == "relu":
        gate = (z > 0).double()
        return gate * z, gate
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":          # (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        q = torch.sigmoid(u2)
        return z * q, q + z * q * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    q = torch.sigmoid(z)
    return z * q, q + z * q * torch.sigmoid(-z)


def _exact_gated_fwd(s, c):
    x = s["x"].double()
    zg, zu = torch.mm(x, s["wg"].double().t()), torch.mm(x, s["wu"].double().t())
    if c["bias"]:
        zg += s["bg"].double()
        zu += s["bu"].double()
    h = _exact_act(c["act"], zg)[0] * zu
    return {"h": h, "zg": zg, "zu": zu} if c["z"] else {"h": h}


def _exact_gated_bwd(s, c):
    a, slope = _exact_act(c["act"], s["zg"].double())
    dzu = s["dh"].double() * a
    dzg = s["dh"].double() * s["zu"].double() * slope
    x = s["x"].double()
    dx = torch.addmm(torch.mm(dzg, s["wg"].double()), dzu, s["wu"].double())
    r = {"dx": dx, "dwg": torch.mm(dzg.t(), x), "dwu": torch.mm(dzu.t(), x)}
    if c["bias"]:
        r.update(dbg=dzg.sum(0), dbu=dzu.sum(0))
    return r


def _exact_ce_fwd(s, c):
    x = torch.mm(s["x"].double(), s["w"].double().t())
    lse = torch.logsumexp(x, 1)
    tgt = s["targets"].long()
    hit = x[torch.arange(x.shape[0], device=x.device), tgt.clamp(min=0)]
    return {"loss": torch.where(tgt < 0, torch.zeros_like(lse), lse - hit), "lse": lse}


def _exact_ce_bwd(s, c):
    x, w, tgt = s["x"].double(), s["w"].double(), s["targets"].long()
    g = s["g_loss"].double() * (tgt >= 0)
    dl = torch.mm(x, w.t()).sub_(s["lse"].double()[:, None]).exp_().mul_(g[:, None])
    hit = (tgt >= 0).nonzero()[:, 0]
    dl[hit, tgt[hit]] -= g[hit]
    return {"dx": torch.mm(dl, w), "dw": torch.mm(dl.t(), x)}


def _exact_emb_fwd(s, c):
    ids = s["ids"].long()
    y = torch.index_select(s["table"], 0, ids.clamp(min=0)).double() * c["scale"]
    y[ids < 0] = 0
    return {"y": y}


def _exact_emb_bwd(s, c):
    grad = s["grad"].double() if c["add"] else torch.zeros((c["classes"], c["d"]), dtype=torch.float64, device=DEVICE)
    there = (s["ids"] >= 0).nonzero()[:, 0]
    grad.index_put_((s["ids"][there].long(),), s["dy"][there].double() * c["scale"], accumulate=True)
    return {"grad": grad}


EXACT = {"gated_fwd": _exact_gated_fwd, "gated_bwd": _exact_gated_bwd, "ce_fwd": _exact_ce_fwd, "ce_bwd": _exact_ce_bwd,
         "emb_fwd": _exact_emb_fwd, "emb_bwd": _exact_emb_bwd}
