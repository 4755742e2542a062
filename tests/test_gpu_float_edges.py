"""The float operators where they were wrong once: results written over their inputs, values far
from 0, masks under large factors, rows of many waves of tiles."""
import math

import numpy as np
import pytest

from test_gpu_float_ops import TINY, U, dt, f64, normal, slope64, within, within_rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


# -------------------------------------------------------------- layer norm

@pytest.mark.parametrize("rows,cols,dtype", [
    (50, 520, "bfloat16"), (40000, 24, "float32"), (1300, 768, "bfloat16"), (700, 5001, "bfloat16"),
    (650, 10000, "bfloat16"), (9, 10000, "bfloat16"), (9, 8193, "float32"), (40, 20000, "float32"), (3, 40000, "bfloat16"),
    (2, 16385, "float16")])
def test_layer_norm_backward_in_place(torch, ito, rows, cols, dtype):
    """dx written over dy, with dgamma and dbeta: the bits of the call that writes dx elsewhere."""
    x, dy = normal(torch, (rows, cols), 1, 1.5, dtype), normal(torch, (rows, cols), 2, 1.0, dtype)
    gamma = 1 + normal(torch, (cols,), 3, 0.2)
    _, mean, rstd = ito.ito_layer_norm_fwd(x, gamma)
    dx, dgamma, dbeta = ito.ito_layer_norm_bwd(dy, x, gamma, mean, rstd)
    within(dbeta, f64(dy).sum(0), (rows + 2) * U * np.abs(f64(dy)).sum(0), "dbeta")
    n = ito._lib.ito_layer_norm_bwd_workspace_size(rows, cols)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    dg, db = torch.empty_like(dgamma), torch.empty_like(dbeta)
    ty = {"float32": ito.ITO_F32, "bfloat16": ito.ITO_BF16, "float16": ito.ITO_F16}[dtype]
    assert ito._lib.ito_layer_norm_bwd(dy.data_ptr(), cols, x.data_ptr(), cols, ty, gamma.data_ptr(), ito.ITO_F32,
                                       mean.data_ptr(), rstd.data_ptr(), rows, cols, ito._aligned256(ws), n,
                                       dy.data_ptr(), cols, dg.data_ptr(), db.data_ptr(), ito._stream()) == 0
    assert torch.equal(db, dbeta)
    assert torch.equal(dg, dgamma)
    assert torch.equal(dy, dx)


# --------------------------------------------------------- log probabilities

@pytest.mark.parametrize("factor", [2.0, -3.0, 65536.0, -65536.0])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [16, 1000, 40000])
def test_logprobs_gradient_of_lowest_values_under_large_factors(torch, ito, n, dtype, factor):
    """Classes masked with the type's lowest value have p = 0 and so a gradient of 0, however large
    the entropy's gradient; the others follow the formula, to the bounds of their 32-bit terms."""
    x = normal(torch, (4, n), n, 2.0, dtype)
    low = torch.finfo(x.dtype).min
    x[0, n // 2:] = low
    x[1, 1:] = low
    x[2, ::3] = low
    x[2, 1::3] = -math.inf
    tgt = torch.tensor([0, 0, 2, n - 1], dtype=torch.int32, device="cuda")
    _, ent, lse, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    gl, gh = torch.full((4,), -0.5, device="cuda"), torch.full((4,), factor, device="cuda")
    d = ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl, gh)
    X, L, H = f64(x), f64(lse)[:, None], f64(ent)[:, None]
    lp = np.maximum(X - L, -1e4)
    p = np.exp(lp)
    hot = (np.arange(n) == f64(tgt)[:, None]).astype(np.float64)
    want = -0.5 * (hot - p) - factor * p * (lp + H)
    size = 0.5 * (hot + p) + abs(factor) * p * (np.abs(lp) + np.abs(H))
    e = 8 * U * size + (0.5 + abs(factor) * (np.abs(lp) + np.abs(H) + 1)) * p * (np.abs(lp) + np.abs(L) + 4) * 2 * U
    e = e + 4 * TINY * (1 + abs(factor) * (np.abs(np.where(p > 0, lp, 0)) + np.abs(H)))
    within_rounded(d, want, e, dtype, "dlogits")
    assert bool((d[0, n // 2:] == 0).all()) and bool((d[1, 1:] == 0).all())


@pytest.mark.parametrize("offset", [0.0, 1000.0, 100000.0, -100000.0, 1000000.0])
@pytest.mark.parametrize("n,many", [(500, False), (2048, False), (2048, True), (70000, False)])
def test_logprobs_of_rows_far_from_zero(torch, ito, n, many, offset):
    """Entropy and log p depend on differences of logits alone, so their bounds do not grow with the
    row's offset. A lane adds n / 64 terms to each of its sums, then some ten sums are joined. A term
    2^y errs by y's rounding (|y| u), the exponential (4 u), and the changes of `top` after it: 60 u for
    the products of ten of them, 40 u for their exponents, whose sum is the lane's range of y."""
    rows = 8 * torch.cuda.get_device_properties(0).multi_processor_count + 3 if many else 3
    x = normal(torch, (rows, n), 5, 2.5) + offset
    tgt = torch.arange(rows, device="cuda", dtype=torch.int32) % n
    logp, ent, _, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    X = f64(x)
    d = X - X.max(1, keepdims=True)
    s = np.exp(d).sum(1, keepdims=True)
    p, lp = np.exp(d) / s, d - np.log(s)
    y = np.abs(d) / math.log(2)
    rho = (n / 64 + 10 + y + 4 + 60 + 40) * U
    e_s, mean = (p * rho).sum(1), (p * -d).sum(1)
    want = -(p * lp).sum(1)
    within(ent, want, e_s + math.log(2) * (p * y * (rho + U)).sum(1) + mean * e_s + 8 * U * (1 + want + mean), "entropy")
    at = np.arange(rows) % n
    dt_, lt = np.abs(d[np.arange(rows), at]), lp[np.arange(rows), at]
    within(logp, lt, e_s + U * (2 * dt_ + 4) + 4 * U * (np.log(s[:, 0]) + np.abs(lt)), "logp")


# ------------------------------------------------------------------ linear

@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("B", [1, 200])
def test_activations_of_large_finite_values(torch, ito, act, dtype, B):
    """From |z| = 16 on an activation is z or 0 and its slope 1 or 0, to far below a unit, up to the type's largest
    value; below, the slope's 32-bit evaluation errs by 16 u (1 + |z|) and the activation's by 8 u (1 + |z|)."""
    big = [12.0, 60.0, 1000.0, 65504.0] + [10.0 ** k for k in (10, 13, 13.5, 14, 16, 19, 20, 30, 38)] * (dtype == "bfloat16")
    z = torch.tensor([s * v for v in [0.0, 0.5, 3.0] + big for s in (1, -1)], device="cuda").to(dt(torch, dtype))
    n = z.numel()
    Z = f64(z)
    with np.errstate(over="ignore"):
        slope = slope64(act, Z)
    near = np.minimum(np.abs(Z), 16)
    x, W = torch.zeros((B, 8), dtype=z.dtype, device="cuda"), torch.zeros((n, 8), dtype=z.dtype, device="cuda")
    dy = torch.zeros((B, n), dtype=z.dtype, device="cuda")
    dy[B - 1] = 1.0
    _, _, db = ito.ito_fp_linear_bwd(dy, x, W, z=z.expand(B, n).contiguous(), act=act)
    within(db, slope, 16 * U * (1 + near), "slope")
    y = ito.ito_fp_linear_fwd(x, W, bias=z, act=act, out_dtype=torch.float32)
    want = np.where(np.abs(Z) > 16, np.maximum(Z, 0), Z * slope) if act == "relu" else None
    if want is None:
        cdf = {"gelu": lambda v: 0.5 * math.erfc(-v / math.sqrt(2)),
               "gelu_tanh": lambda v: 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
               "silu": lambda v: 1 / (1 + math.exp(-v))}[act]
        want = np.array([max(v, 0.0) if abs(v) > 60 else v * cdf(v) for v in Z])
    tol = 8 * U * (1 + np.where(Z > 0, Z, near))
    within(y, np.broadcast_to(want, (B, n)), np.broadcast_to(tol, (B, n)), "activation")


# ----------------------------------------------------------------- streams

def test_tensors_may_be_dropped_after_a_call_on_another_stream(torch, ito):
    """A call on a stream that is still busy, its inputs dropped at once and others allocated and
    filled in their place: the results are those of the inputs that were given."""
    side = torch.cuda.Stream()
    x0, W0 = normal(torch, (300, 256), 1, 1.0, "bfloat16"), normal(torch, (512, 256), 2, 0.1, "bfloat16")
    logits0 = normal(torch, (300, 512), 3, 2.0)
    tgt = torch.arange(300, device="cuda", dtype=torch.int32)
    w0, g0 = normal(torch, (5000,), 4), normal(torch, (5000,), 5)
    want_w = w0.clone()
    ito.AdamW([want_w]).step([g0], lr=0.1)
    cases = [(lambda t, s: ito.ito_fp_linear_fwd(t[0], t[1], residual=t[2], stream=s),
              [x0, W0, normal(torch, (300, 512), 6, 1.0, "bfloat16")]),
             (lambda t, s: ito.ito_fp_linear_bwd(t[2], t[0], t[1], stream=s)[0],
              [x0, W0, normal(torch, (300, 512), 6, 1.0, "bfloat16")]),
             (lambda t, s: ito.ito_layer_norm_fwd(t[0], stream=s)[0], [logits0]),
             (lambda t, s: ito.ito_token_logprobs_fwd(t[0], t[1], stream=s)[0], [logits0, tgt])]
    for call, inputs in cases:
        want = call(inputs, None)
        t = [i.clone() for i in inputs]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20000000)
        got = call(t, side)
        del t
        others = [torch.zeros_like(i) for i in inputs for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del others
    w, g = w0.clone(), [g0.clone()]
    opt = ito.AdamW([w])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20000000)
    opt.step(g, lr=0.1, stream=side)
    del g, opt
    others = [torch.full_like(w0, 7.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(w, want_w)
    del others


def test_threads_on_one_stream(torch, ito):
    """Host threads that call on the same stream share no workspace: each gets the bits of a call alone."""
    import threading
    stream = torch.cuda.Stream()
    sets = []
    for i in range(4):
        B, IC, OC = [(40, 251, 264), (333, 787, 1000), (300, 1000, 136), (64, 2048, 72)][i]
        x, W = normal(torch, (B, IC), i, 1.0, "bfloat16"), normal(torch, (OC, IC), i + 10, 0.1, "bfloat16")
        dy, z = normal(torch, (B, OC), i + 20, 1.0, "bfloat16"), normal(torch, (B, OC), i + 30, 1.0, "bfloat16")
        v = normal(torch, (B, OC), i + 40)
        _, mean, rstd = ito.ito_layer_norm_fwd(v)
        sets.append((x, W, dy, z, v, mean, rstd))

    def calls(s):
        x, W, dy, z, v, mean, rstd = s
        return [ito.ito_fp_linear_fwd(x, W, act="silu"), *ito.ito_fp_linear_bwd(dy, x, W, z=z, act="gelu"),
                *ito.ito_layer_norm_bwd(v, v, None, mean, rstd)]

    want = [calls(s) for s in sets]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(sets))

    def work(i):
        try:
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = calls(sets[i])
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:      # (an assertion of a thread would be lost)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ------------------------------------------------------------------- AdamW

@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_steps_tensors_where_they_are(torch, ito, bits):
    """Weights and copies given other memory between two steps: both steps reach them."""
    sizes = [70000, 129, 1]
    start, g = [normal(torch, (n,), n) for n in sizes], [normal(torch, (n,), n + 1) for n in sizes]

    def train(move):
        w = [t.clone() for t in start]
        c = [t.bfloat16() for t in start]
        opt = ito.AdamW(w, bits=bits, copies=c, seed=3)
        for i in range(3):
            opt.step(g, lr=0.01)
            if move:
                for ts in (w, c):
                    for t in ts:
                        t.data = t.data.clone()
        return w + c + [t for ts in opt.states for t in ts] + list(opt.moments())

    assert all(torch.equal(a, b) for a, b in zip(train(False), train(True)))
    w = [t.clone() for t in start]
    opt = ito.AdamW(w, bits=bits)
    w[1].data = w[1].data.half()
    with pytest.raises(ito.ItoError) as e:
        opt.step(g, lr=0.01)
    assert e.value.code == ito.ITO_ERR_ARG and opt.steps == 0


# -------------------------------------------------- beyond 2^31 elements

def _filled(torch, shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=g)


@pytest.mark.parametrize("OC", [4104, 4101])      # rows that TMA stores take, and plain stores
def test_linear_rows_beyond_32_bits(torch, ito, OC):
    """The last rows of more than 2^31 elements, against 64-bit products of those rows."""
    B, IC = (1 << 19) + 5, 72
    x, W, r = _filled(torch, (B, IC), 1), _filled(torch, (OC, IC), 2, IC ** -0.5), _filled(torch, (B, OC), 3)
    y = ito.ito_fp_linear_fwd(x, W, residual=r)
    dx, _, db = ito.ito_fp_linear_bwd(r, x, W, need_dw=False)
    for rows in (slice(0, 130), slice(B - 130, B)):
        X, V, R = f64(x[rows]), f64(W), f64(r[rows])
        within_rounded(y[rows], X @ V.T + R, 2 * (IC + 2) * U * (np.abs(X) @ np.abs(V).T + np.abs(R)), "bfloat16", "y")
        within_rounded(dx[rows], R @ V, 2 * OC * U * (np.abs(R) @ np.abs(V)), "bfloat16", "dx")
    total, size = (sum(f(r[i:i + 65536].double()).sum(0) for i in range(0, B, 65536)) for f in (lambda t: t, torch.abs))
    # a thread adds at most B / (8 * 32) rows of its share, then 32 threads' and 8 blocks' sums are added
    within(db, f64(total), (B / 256 + 48) * U * f64(size), "dbias")


@pytest.mark.parametrize("cols", [4104, 4101])
def test_layer_norm_rows_beyond_32_bits(torch, ito, cols):
    """The last rows of more than 2^31 elements have the bits that a call on them alone gives."""
    rows = (1 << 19) + 5
    x, dy = _filled(torch, (rows, cols), 1, 1.5), _filled(torch, (rows, cols), 2)
    gamma, beta = 1 + normal(torch, (cols,), 3, 0.2), normal(torch, (cols,), 4, 0.5)
    y, mean, rstd = ito.ito_layer_norm_fwd(x, gamma, beta)
    dx, _, _ = ito.ito_layer_norm_bwd(dy, x, gamma, mean, rstd)
    many = 4 * torch.cuda.get_device_properties(0).multi_processor_count + 8       # rows enough for the same kernels
    end = slice(rows - many, rows)
    y2, mean2, rstd2 = ito.ito_layer_norm_fwd(x[end], gamma, beta)
    dx2, _, _ = ito.ito_layer_norm_bwd(dy[end], x[end], gamma, mean2, rstd2)
    assert torch.equal(y[end], y2) and torch.equal(mean[end], mean2) and torch.equal(rstd[end], rstd2)
    assert torch.equal(dx[end], dx2)


@pytest.mark.parametrize("n", [65536, 65533])
def test_logprobs_rows_beyond_32_bits(torch, ito, n):
    """The last rows of more than 2^31 elements have the bits that a call on enough of them alone gives."""
    rows = 33000
    x = _filled(torch, (rows, n), 1, 2.0)
    tgt = torch.arange(rows, device="cuda", dtype=torch.int32)
    gl, gh = normal(torch, (rows,), 2), normal(torch, (rows,), 3)
    got = ito.ito_token_logprobs_fwd(x, tgt, k=3)
    d = ito.ito_token_logprobs_bwd(x, tgt, got[2], got[1], gl, gh)
    end = slice(rows - 8 * torch.cuda.get_device_properties(0).multi_processor_count - 8, rows)
    alone = ito.ito_token_logprobs_fwd(x[end], tgt[end], k=3)
    assert all(torch.equal(a[end], b) for a, b in zip(got, alone))
    assert torch.equal(d[end], ito.ito_token_logprobs_bwd(x[end], tgt[end], alone[2], alone[1], gl[end], gh[end]))
