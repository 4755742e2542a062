"""The linear cross entropy where its sums matter most: rows whose target has nearly all of the probability, so that
p - 1 is what is left of two values next to one another, and rows of many elements.

Tolerances as in test_gpu_token_ops.py: U = 2^-24, a sum of n products with truncation is off by at most 2 n U sum|terms|."""
import math

import pytest

from test_gpu_float_ops import TINY, U, f64, normal, within, within_rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


def confident(torch, rows, d, classes, dtype, seed, targets, logits):
    """x and W of which row r has the logit logits[r] (before x is rounded) for its target, and logits of about a
    normal distribution for the others."""
    W = normal(torch, (classes, d), seed + 1, d ** -0.5, dtype)
    V = W[targets].float()
    n = normal(torch, (rows, d), seed)
    along = (logits - (n * V).sum(1)) / (V * V).sum(1)
    return (n + along[:, None] * V).to(W.dtype), W


HALF = {"bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25)}


def check_confident_bwd(torch, x, W, t, dtype, dx, dw):
    """With l' = l + delta the logits that both passes form (the same sums, |delta| <= eL) and lse' = log sum exp(l')
    off by `ev` where it is evaluated, the target's dl is exp(l'_t - lse') - 1: off by (1 - p) expm1(2 eL) for the
    deltas, because 1 - p is a sum of exp(l'_j - l'_t), and by ev, the exponential and the difference. The other
    classes' are off in proportion. Then the rounding of dl to 16 bits, and the products' sums."""
    rows, d = x.shape
    X, V = x.double(), W.double()
    L = X @ V.T
    lse = torch.logsumexp(L, 1)
    span = L.amax(1) - L.amin(1)
    p = torch.exp(L - lse[:, None])
    eL = torch.expm1(2 * (2 * (d + 1) * U * (X.abs() @ V.abs().T)).amax(1))
    ev = U * (224 + 8 * span) + U * lse.abs()       # (as check_ce_fwd of test_gpu_token_ops.py)
    at = (torch.arange(rows, device="cuda"), t.long())
    rest = p.clone()
    rest[at] = 0
    q = rest.sum(1)
    assert bool((q < 1e-2).all()) and bool((q > 1e-6).all())
    dl = rest
    e = dl * ((eL + ev)[:, None] + 8 * U * (1 + (L - lse[:, None]).abs()))
    dl[at] = -q
    e[at] = q * eL + ev + 8 * U
    half, floor = HALF[dtype]
    e = e + (dl.abs() + e) * half * (1 + 2.0 ** -20) + floor
    m = dl.abs() + e
    if dw is not None:
        within(dw, f64(dl.T @ X), f64(e.T @ X.abs() + 2 * rows * U * (m.T @ X.abs())), "dW")
        # a row's dl add up to 0: their sums, from dW's columns' sums by the rows of x (rows < d: they are independent)
        S = dw.double().sum(0)
        inv = torch.linalg.inv(X @ X.T) @ X
        sums = inv @ S
        tol = e.sum(1) + inv.abs() @ (2 * rows * U * (m.T @ X.abs()).sum(0))
        within(sums, 0 * f64(sums), f64(tol), "sum of dl")
    if dx is not None:
        within_rounded(dx, f64(dl @ V), f64(e @ V.abs() + 2 * W.shape[0] * U * (m @ V.abs())), dtype, "dx")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("rows,d,classes", [(3, 4096, 600), (16, 8192, 640), (20, 4096, 600), (17, 8192, 700),
                                            (24, 2048, 2000), (20, 1024, 4000), (30, 32768, 100), (40, 4096, 600),
                                            (130, 4095, 611), (300, 8192, 600), (300, 4104, 5000)])
def test_gradient_of_confident_rows(torch, ito, rows, d, classes, dtype):
    """1 - p of the targets from 1e-3 to 1e-5."""
    t = torch.randperm(classes, generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda")[:rows].to(torch.int32)
    logits = math.log(classes) + 0.5 + torch.linspace(math.log(1e3), math.log(1e5), rows, device="cuda")
    x, W = confident(torch, rows, d, classes, dtype, rows + d, t.long(), logits)
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = torch.ones(rows, device="cuda")
    dx, dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, dw_dtype=torch.float32)
    check_confident_bwd(torch, x, W, t, dtype, dx, dw)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_gradient_of_confident_rows_in_a_narrow_last_piece(torch, ito, dtype):
    """Targets in the last piece of the vocabulary, of 24 classes: their logits are the sums that the forward pass
    formed, so their gradient is, bit for bit, that of a call of fewer rows, which has the vocabulary in one piece."""
    rows, d, wide, some = 4200, 4096, 31744, 24
    classes = wide + some
    at = torch.arange(some, device="cuda") + wide
    t = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    t[:some] = at.to(torch.int32)
    x = normal(torch, (rows, d), 5, 1.0, dtype)
    logits = math.log(classes) + 0.5 + torch.linspace(math.log(1e3), math.log(1e5), some, device="cuda")
    first, W = confident(torch, some, d, classes, dtype, 7, at, logits)
    x[:some] = first
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = torch.ones(rows, device="cuda")
    dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, need_dx=False, dw_dtype=torch.float32)[1]
    n = 300
    part = ito.ito_linear_cross_entropy_bwd(x[:n], W, t[:n], lse[:n], g[:n], need_dx=False, dw_dtype=torch.float32)[1]
    assert torch.equal(dw[wide:], part[wide:])
    check_confident_bwd(torch, x[:some], W, t[:some], dtype, None, dw)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rows,d,classes", [(1, 16384, 5000), (1, 65536, 64), (9, 65536, 5000), (12, 32776, 3000), (20, 32768, 100),
                                            (40, 65536, 300)])
def test_logits_of_long_rows(torch, ito, rows, d, classes, offset):
    """Positive products, whose sums only grow, so that what each step of 16 k cuts off adds up. A chain of at most
    1024 k loses at most 2^-23 of its sum at each of 64 steps; the chains' sums are added rounded: at most d / 1024 and 16
    (of warps or slices) of them, U each. lse and the logit of the target are off by as much of themselves; what they are
    evaluated with as in check_ce_fwd of test_gpu_token_ops.py."""
    x = normal(torch, (rows, d), 1).abs().to(torch.bfloat16)
    wide = torch.zeros((classes, d + offset), dtype=torch.bfloat16, device="cuda")
    W = wide[:, offset:]
    W.copy_(normal(torch, (classes, d), 2).abs() * (100 / d / 0.64))
    t = (torch.arange(rows, device="cuda") * 7 % classes).to(torch.int32)
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    L = x.double() @ W.double().T
    want = torch.logsumexp(L, 1)
    span = L.amax(1) - L.amin(1)
    s = torch.log(torch.exp(L - L.amax(1, keepdim=True)).sum(1))
    eL = (64 * 2.0 ** -23 + (d / 1024 + 16) * U) * L.amax(1)
    e = eL + U * (224 + 8 * span) + 2 * U * s.abs() + U * want.abs() + TINY
    within(lse, f64(want), f64(e), "lse")
    l = want - L.gather(1, t.long()[:, None])[:, 0]
    within(loss, f64(l), f64(e + eL + U * l.abs()), "loss")


@pytest.mark.parametrize("rows", [5, 60])
@pytest.mark.parametrize("k", [-113, -105, 105, 112, 118, 124])
def test_large_and_small_factors_in_float16(torch, ito, rows, k):
    """Factors at both ends of float32: the gradients scale with them exactly (a power of two), which float32 results show."""
    x, W = normal(torch, (rows, 64), 4, 1.0, "float16"), normal(torch, (2000, 64), 5, 0.25, "float16")
    t = (torch.arange(rows, device="cuda") * 31 - 1).to(torch.int32)
    _, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = normal(torch, (rows,), 6).abs().clamp(0.1, 3.5)
    dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, dw_dtype=torch.float32)[1]
    far = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g * 2.0 ** k, dw_dtype=torch.float32)[1]
    assert bool(torch.isfinite(far).all()) and torch.equal(far, dw * 2.0 ** k)
