"""The float operators against plain computations in 64 bits, their gradients against the
formulas and against differences, and their behaviour on other streams, strides and masks.

Tolerances are bounds of the arithmetic: u = 2^-24 is half a unit of a 32-bit float, a sum of
n terms is off by at most n u sum|terms| in any order (2 n u where the products are
accumulated with truncation). A result's own rounding needs no bound: rounding keeps order, so
a result lies between the roundings of the two ends of what its 32-bit value can be."""
import ctypes
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -149
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


def dt(torch, name):
    return getattr(torch, name)


def normal(torch, shape, seed, scale=1.0, dtype="float32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt(torch, dtype))


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol, what=""):
    got = f64(got) if hasattr(got, "detach") else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %g over its bound at %s" % (
        what, bad.sum(), bad.size, np.nanmax((np.abs(got - want) / np.maximum(tol, 1e-300))), np.argwhere(bad)[:3].tolist())


def rounded(a, dtype):
    """float64 values of a (float64) rounded to a type."""
    import torch
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, dtype)).double().numpy()


def within_rounded(got, want, e, dtype, what=""):
    """got is a value within e of want, rounded to its type."""
    g = f64(got)
    e = e + TINY + 2.0 ** -50 * np.abs(want)
    bad = ~((g >= rounded(want - e, dtype)) & (g <= rounded(want + e, dtype)))
    assert not bad.any(), "%s: %d of %d off at %s, by %g of %g" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[:3].tolist(), np.abs(g - want)[bad].max(), np.abs(want)[bad].max())


def rounding_error(a, dtype):
    """How far a value of magnitude a at most moves when rounded to a type."""
    return np.abs(rounded(np.abs(a) * (1 + 2.0 ** -40), dtype)) * {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}[dtype] + \
        {"bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}[dtype]


# ------------------------------------------------------------------ linear

_erf = np.vectorize(math.erf)


def act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + np.exp(-z))


def slope64(name, z):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    q = 1 / (1 + np.exp(-z))
    return q * (1 + z * (1 - q))


def check_linear_fwd(torch, ito, B, IC, OC, dtype, act, bias, residual, save_z, out_dtype, seed=0, x=None, W=None):
    x = normal(torch, (B, IC), seed + 1, 1.0, dtype) if x is None else x
    W = normal(torch, (OC, IC), seed + 2, IC ** -0.5, dtype) if W is None else W
    b = normal(torch, (OC,), seed + 3, 0.5, bias) if bias else None
    r = normal(torch, (B, OC), seed + 4, 1.0, out_dtype) if residual else None
    got = ito.ito_fp_linear_fwd(x, W, bias=b, act=act, residual=r, save_z=save_z, out_dtype=dt(torch, out_dtype))
    y, z = got if save_z else (got, None)
    X, V = f64(x), f64(W)
    zz = X @ V.T
    sums = np.abs(X) @ np.abs(V).T
    if bias:
        zz = zz + f64(b)
        sums = sums + np.abs(f64(b))
    ez = 2 * (IC + 1) * U * sums
    assert y.shape == (B, OC) and y.dtype == dt(torch, out_dtype)
    # the activations' slopes stay below 1.13; 32-bit evaluations of them err by a few units of 1 + |z|
    yy = act64(act, zz)
    ey = 1.13 * ez + 8 * U * (1 + np.abs(zz)) * (act != "none")
    if residual:
        yy = yy + f64(r)
        ey = ey + U * (np.abs(yy) + np.abs(f64(r)))
    within_rounded(y, yy, ey, out_dtype, "y")
    if save_z:
        assert z.dtype == x.dtype
        within_rounded(z, zz, ez, dtype, "z")


LINEAR_SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 1000), (2, 787, 33), (3, 8, 8), (4, 4096, 512), (5, 100, 1000),
                (8, 1024, 10), (9, 256, 264), (16, 512, 640), (17, 64, 64), (32, 64, 10), (33, 4096, 128),
                (64, 2048, 2048), (127, 129, 130), (128, 128, 128), (129, 65, 257), (256, 256, 256), (257, 264, 511),
                (300, 1000, 520), (512, 640, 768), (700, 72, 1032)]


@pytest.mark.parametrize("i,size", list(enumerate(LINEAR_SIZES)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_fwd(torch, ito, i, size, dtype):
    n = i + (dtype == "float16") * 2
    out = dtype if n % 3 else "float32"
    check_linear_fwd(torch, ito, *size, dtype, ACTS[n % 5], (None, dtype, "float32")[n % 3], n % 2 == 0, n % 4 < 2, out,
                     seed=10 * i)
    check_linear_fwd(torch, ito, *size, dtype, ACTS[(n + 2) % 5], (dtype, "float32", None)[n % 3], n % 2 == 1, n % 4 > 1,
                     "float32" if out == dtype else dtype, seed=10 * i + 5)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 256, 384), (12, 256, 384), (200, 256, 384), (512, 256, 512)])
def test_linear_fwd_every_activation(torch, ito, act, size):
    check_linear_fwd(torch, ito, *size, "bfloat16", act, "bfloat16", True, True, "bfloat16")
    check_linear_fwd(torch, ito, *size, "float16", act, None, False, False, "float32")


def check_linear_bwd(torch, ito, B, IC, OC, dtype, act, dw_dtype, seed=0, x=None, W=None, dy=None, z=None):
    x = normal(torch, (B, IC), seed + 1, 1.0, dtype) if x is None else x
    W = normal(torch, (OC, IC), seed + 2, IC ** -0.5, dtype) if W is None else W
    dy = normal(torch, (B, OC), seed + 3, 1.0, dtype) if dy is None else dy
    z = normal(torch, (B, OC), seed + 4, 2.0, dtype) if z is None else z
    dx, dw, db = ito.ito_fp_linear_bwd(dy, x, W, z=z if act != "none" else None, act=act, dw_dtype=dt(torch, dw_dtype))
    X, V, D, Z = f64(x), f64(W), f64(dy), f64(z)
    dz = D * slope64(act, Z)
    # the slope in 32 bits, the product's rounding, then dz's rounding to the operands' type
    e0 = np.abs(D) * 16 * U * (1 + np.abs(Z)) * (act != "none") + U * np.abs(dz) * (act != "none")
    ez = e0 + (rounding_error(np.abs(dz) + e0, dtype) if act != "none" else 0)
    a = np.abs(dz) + ez
    want = dz @ V
    e = ez @ np.abs(V) + 2 * OC * U * (a @ np.abs(V))
    within_rounded(dx, want, e, dtype, "dx")
    want = dz.T @ X
    e = ez.T @ np.abs(X) + 2 * B * U * (a.T @ np.abs(X))
    within_rounded(dw, want, e, dw_dtype, "dW")
    within(db, dz.sum(0), e0.sum(0) + (B + 1) * U * (np.abs(dz) + e0).sum(0) + TINY, "dbias")


@pytest.mark.parametrize("i,size", list(enumerate(LINEAR_SIZES)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_bwd(torch, ito, i, size, dtype):
    n = i + (dtype == "float16")
    check_linear_bwd(torch, ito, *size, dtype, ACTS[n % 5], dtype if n % 2 else "float32", seed=10 * i)
    check_linear_bwd(torch, ito, *size, dtype, "none", "float32" if n % 2 else dtype, seed=10 * i + 5)


def test_linear_bwd_parts(torch, ito):
    """Each gradient alone is the gradient among the others, bit for bit."""
    x, W = normal(torch, (200, 136), 1, 1.0, "bfloat16"), normal(torch, (264, 136), 2, 0.1, "bfloat16")
    dy, z = normal(torch, (200, 264), 3, 1.0, "bfloat16"), normal(torch, (200, 264), 4, 1.0, "bfloat16")
    for act, zz in (("none", None), ("silu", z)):
        full = ito.ito_fp_linear_bwd(dy, x, W, z=zz, act=act)
        for k in range(3):
            need = dict(need_dx=k == 0, need_dw=k == 1, need_dbias=k == 2)
            part = ito.ito_fp_linear_bwd(dy, x, W, z=zz, act=act, **need)
            assert [p is not None for p in part] == [k == 0, k == 1, k == 2]
            assert torch.equal(part[k], full[k])


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 7), (3, 5), (8, 16), (2, 1)])
@pytest.mark.parametrize("size", [(1, 136, 72), (40, 136, 72), (300, 264, 320)])
def test_linear_strided_and_misaligned(torch, ito, offset, pad, size):
    """Operands inside wider buffers, at odd offsets and odd row strides."""
    B, IC, OC = size

    def inside(rows, cols, seed, scale=1.0):
        wide = normal(torch, (rows, cols + offset + pad), seed, scale, "bfloat16")
        return wide[:, offset:offset + cols]

    x, W, dy, z = inside(B, IC, 1), inside(OC, IC, 2, IC ** -0.5), inside(B, OC, 3), inside(B, OC, 4)
    check_linear_fwd(torch, ito, B, IC, OC, "bfloat16", "silu", "float32", True, True, "bfloat16", x=x, W=W)
    check_linear_bwd(torch, ito, B, IC, OC, "bfloat16", "gelu", "bfloat16", x=x, W=W, dy=dy, z=z)
    check_linear_bwd(torch, ito, B, IC, OC, "bfloat16", "none", "float32", x=x, W=W, dy=dy, z=z)


@pytest.mark.parametrize("offset,ld", [(0, 80), (1, 79), (4, 84), (3, 77)])
@pytest.mark.parametrize("B", [1, 12, 200, 300])
def test_linear_strided_outputs_keep_their_padding(torch, ito, offset, ld, B):
    IC, OC = 64, 72
    x, W = normal(torch, (B, IC), 1, 1.0, "float16"), normal(torch, (OC, IC), 2, 0.1, "float16")
    want, zw = ito.ito_fp_linear_fwd(x, W, act="gelu", save_z=True)
    bufs = [torch.full((B * ld + offset + 8,), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    n = ito._lib.ito_fp_linear_fwd_workspace_size(x.data_ptr(), IC, W.data_ptr(), IC, B, IC, OC)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    y, z = (b.data_ptr() + 2 * offset for b in bufs)
    r = ito._lib.ito_fp_linear_fwd(x.data_ptr(), IC, W.data_ptr(), IC, None, None, 0, ito.ITO_F16, ito.ITO_F16, 0,
                                   ito.ITO_ACT_GELU, B, IC, OC, ito._aligned256(ws), n, z, ld, y, ld, ito._stream())
    assert r == 0
    for b, w in zip(bufs, (want, zw)):
        cells = torch.as_strided(b, (B, OC), (ld, 1), offset)
        assert torch.equal(cells, w)
        cells.fill_(7.0)
        assert bool((b == 7.0).all())


@pytest.mark.parametrize("B", [1, 16, 100, 512])
def test_linear_residual_in_place(torch, ito, B):
    x, W = normal(torch, (B, 256), 1, 1.0, "bfloat16"), normal(torch, (512, 256), 2, 0.1, "bfloat16")
    r = normal(torch, (B, 512), 3, 1.0, "bfloat16")
    want = ito.ito_fp_linear_fwd(x, W, act="silu", residual=r)
    y = r.clone()
    n = ito._lib.ito_fp_linear_fwd_workspace_size(x.data_ptr(), 256, W.data_ptr(), 256, B, 256, 512)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    assert ito._lib.ito_fp_linear_fwd(x.data_ptr(), 256, W.data_ptr(), 256, None, y.data_ptr(), 512, ito.ITO_BF16,
                                      ito.ITO_BF16, 0, ito.ITO_ACT_SILU, B, 256, 512, ito._aligned256(ws), n, None, 0,
                                      y.data_ptr(), 512, ito._stream()) == 0
    assert torch.equal(y, want)


@pytest.mark.parametrize("size", [(1, 70, 40), (20, 300, 136), (150, 300, 136), (300, 300, 264)])
def test_linear_keeps_rows_apart(torch, ito, size):
    """An infinity or a NaN in one row of x, or of W, reaches that row, or column, of y alone."""
    B, IC, OC = size
    x, W = normal(torch, (B, IC), 1, 1.0, "bfloat16"), normal(torch, (OC, IC), 2, 0.1, "bfloat16")
    clean = ito.ito_fp_linear_fwd(x, W)
    x2 = x.clone()
    x2[B // 2, IC - 1] = math.nan
    y = ito.ito_fp_linear_fwd(x2, W)
    assert bool(torch.isnan(y[B // 2]).all())
    keep = torch.arange(B, device="cuda") != B // 2
    assert torch.equal(y[keep], clean[keep])
    W2 = W.clone()
    W2[OC - 1, 0] = math.inf
    y = ito.ito_fp_linear_fwd(x, W2)
    assert not bool(torch.isfinite(y[:, OC - 1]).any())
    assert torch.equal(y[:, :OC - 1], clean[:, :OC - 1])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [3, 40, 256])
def test_linear_gradients_by_differences(torch, ito, act, B):
    """Directional differences of L = sum c y against the gradients, with float32 outputs.
    The products are exact (few-bit operands), so L's error is the activation's, 8 u (1 + |z|)
    an element; central differences of step h are off by h^2/6 |third derivative| (below 3 a unit
    of direction^3)."""
    IC, OC, h = 24, 40, 2.0 ** -8
    g = torch.Generator(device="cuda").manual_seed(B)

    def few(shape, hi):
        return (torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").float() / 16).to(torch.float16)

    x, W, c = few((B, IC), 16), few((OC, IC), 8), few((B, OC), 16)
    bias = few((OC,), 16).float()
    if act == "relu":       # keep away from the corner, where a difference is no derivative
        bias = bias + 2.0 ** -5
    _, z = ito.ito_fp_linear_fwd(x, W, bias=bias, act=act, save_z=True)
    dx, _, db = ito.ito_fp_linear_bwd(c, x, W, z=z, act=act)

    def loss(xx, bb):
        return float((f64(ito.ito_fp_linear_fwd(xx, W, bias=bb, act=act, out_dtype=torch.float32)) * f64(c)).sum())

    C, Z = np.abs(f64(c)), np.abs(f64(z))
    noise = (C * 8 * U * (1.2 + Z)).sum() / h
    i, j = B // 2, 5
    xp, xm = x.clone(), x.clone()
    xp[i, j] += h
    xm[i, j] -= h
    step = np.abs(f64(W)[:, j])
    # relu is linear between its corners, and z's distance from them (1/32 - multiples of 1/256) exceeds h |W|
    third = 0.0 if act in ("none", "relu") else 3 * h * h / 6 * (C[i] * step ** 3).sum()
    slopes = 1.13 * (C[i] * step).sum()
    tol = noise + third + slopes * (2.0 ** -12 * 2 + 2.0 ** -11 * (act != "none"))   # dx's and dz's rounding, z's rounding
    assert abs((loss(xp, bias) - loss(xm, bias)) / (2 * h) - float(dx[i, j])) <= tol
    bp, bm = bias.clone(), bias.clone()
    bp[7] += h
    bm[7] -= h
    third = 0.0 if act in ("none", "relu") else 3 * h * h / 6 * C[:, 7].sum()
    tol = noise + third + (C[:, 7] * (2.0 ** -11 * (1 + Z[:, 7]))).sum()
    assert abs((loss(x, bp) - loss(x, bm)) / (2 * h) - float(db[7])) <= tol


# -------------------------------------------------------------- layer norm

LN_SIZES = [(1, 1), (1, 7), (3, 787), (5, 16), (2, 4096), (33, 64), (40, 1000), (700, 136), (9, 8192), (2, 20000),
            (1, 70001), (1000, 33), (2500, 8), (311, 1024)]


def check_layer_norm(torch, ito, x, gamma, beta, dy, eps, dtype):
    rows, cols = x.shape
    y, mean, rstd = ito.ito_layer_norm_fwd(x, gamma, beta, eps=eps)
    X = f64(x)
    G = np.ones(cols) if gamma is None else f64(gamma)
    Bt = np.zeros(cols) if beta is None else f64(beta)
    mu = X.mean(1, keepdims=True)
    var = ((X - mu) ** 2).mean(1, keepdims=True)
    rs = 1 / np.sqrt(var + eps)
    h = (X - mu) * rs
    n = cols / 32 + 24                 # terms of a thread's own sum at most, and the joining of threads
    e_mu = n * U * np.abs(X).mean(1, keepdims=True) + U * np.abs(mu)
    # centred sums: a wrong mean enters squared; then the sum's, the division's, the root's error
    e_rs = rs * (n * U * 2 + 4 * U + 0.5 * (e_mu * rs) ** 2)
    within(mean[:, None], mu, e_mu, "mean")
    within(rstd[:, None], rs, e_rs, "rstd")
    e_h = rs * (e_mu + U * np.abs(X)) + np.abs(X - mu) * e_rs + 2 * U * np.abs(h)
    want = h * G + Bt
    e = np.abs(G) * e_h + 3 * U * (np.abs(h * G) + np.abs(Bt))
    within_rounded(y, want, e, dtype, "y")
    # the backward pass, from the saved mean and rstd
    dx, dg, db = ito.ito_layer_norm_bwd(dy, x, gamma, mean, rstd)
    D, mu, rs = f64(dy), f64(mean)[:, None], f64(rstd)[:, None]
    h = (X - mu) * rs
    e_h = 3 * U * (np.abs(h) + rs * np.abs(X))
    a = D * G
    ma, mh = a.mean(1, keepdims=True), (a * h).mean(1, keepdims=True)
    want = rs * (a - ma - h * mh)
    e_ma = (n + 1) * U * np.abs(a).mean(1, keepdims=True)
    e_mh = (n + 2) * U * np.abs(a * h).mean(1, keepdims=True) + (np.abs(a) * e_h).mean(1, keepdims=True)
    e = rs * (4 * U * (np.abs(a) + np.abs(ma) + np.abs(h * mh)) + e_ma + np.abs(h) * e_mh + e_h * np.abs(mh))
    within_rounded(dx, want, e, dtype, "dx")
    within(dg, (D * h).sum(0), (np.abs(D) * e_h).sum(0) + (rows + 2) * U * np.abs(D * h).sum(0), "dgamma")
    within(db, D.sum(0), (rows + 2) * U * np.abs(D).sum(0), "dbeta")


@pytest.mark.parametrize("i,size", list(enumerate(LN_SIZES)))
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_layer_norm(torch, ito, i, size, dtype):
    rows, cols = size
    w = "float32" if (i + len(dtype)) % 2 else dtype
    x = (normal(torch, size, i, 1.5) + normal(torch, (rows, 1), i + 50, 1.0)).to(dt(torch, dtype))
    gamma = None if i % 5 == 4 else (1 + normal(torch, (cols,), i + 100, 0.2)).to(dt(torch, w))
    beta = None if i % 4 == 3 else normal(torch, (cols,), i + 200, 0.5, w)
    check_layer_norm(torch, ito, x, gamma, beta, normal(torch, size, i + 300, 1.0, dtype), 1e-5, dtype)


@pytest.mark.parametrize("size", [(1300, 768), (1251, 1000), (700, 2600), (650, 10000), (700, 5001), (2500, 300), (40000, 24)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_layer_norm_of_many_rows(torch, ito, size, dtype):
    """Rows enough for rings and for several to a block, of lengths for each of the block sizes."""
    x = (normal(torch, size, 1, 1.5) + normal(torch, (size[0], 1), 2, 1.0)).to(dt(torch, dtype))
    check_layer_norm(torch, ito, x, 1 + normal(torch, (size[1],), 3, 0.2), normal(torch, (size[1],), 4, 0.5),
                     normal(torch, size, 5, 1.0, dtype), 1e-5, dtype)


@pytest.mark.parametrize("cols", [64, 100, 2048])
def test_layer_norm_of_flat_and_far_rows(torch, ito, cols):
    """Rows of one value (no variance but eps), and rows whose mean is large beside their spread."""
    x = torch.zeros((4, cols), device="cuda")
    x[1] = 3.25
    x[2] = 1000.0 + normal(torch, (cols,), 1, 0.25)
    x[3] = normal(torch, (cols,), 2, 1e-3)
    check_layer_norm(torch, ito, x, normal(torch, (cols,), 3), None, normal(torch, (4, cols), 4), 1e-5, "float32")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 2), (4, 4)])
@pytest.mark.parametrize("size", [(5, 136), (70, 1000)])
def test_layer_norm_strided(torch, ito, dtype, offset, pad, size):
    rows, cols = size
    x, dy = (normal(torch, (rows, cols + offset + pad), s, 1.0, dtype)[:, offset:offset + cols] for s in (1, 2))
    check_layer_norm(torch, ito, x, normal(torch, (cols + 1,), 3)[1:], normal(torch, (cols,), 4), dy, 1e-6, dtype)


def test_layer_norm_in_place(torch, ito):
    x, dy = normal(torch, (50, 520), 1, 1.0, "bfloat16"), normal(torch, (50, 520), 2, 1.0, "bfloat16")
    y, mean, rstd = ito.ito_layer_norm_fwd(x)
    dx, _, _ = ito.ito_layer_norm_bwd(dy, x, None, mean, rstd)
    dy2 = dy.clone()
    assert ito._lib.ito_layer_norm_bwd(dy2.data_ptr(), 520, x.data_ptr(), 520, ito.ITO_BF16, None, 0, mean.data_ptr(),
                                       rstd.data_ptr(), 50, 520, None, 0, dy2.data_ptr(), 520, None, None,
                                       ito._stream()) == 0
    assert torch.equal(dy2, dx)
    assert ito._lib.ito_layer_norm_fwd(x.data_ptr(), 520, ito.ITO_BF16, None, None, 0, 50, 520, 1e-5, x.data_ptr(), 520,
                                       None, None, ito._stream()) == 0
    assert torch.equal(x, y)


def test_layer_norm_nan_stays_in_its_row(torch, ito):
    x = normal(torch, (6, 1000), 1)
    clean, _, _ = ito.ito_layer_norm_fwd(x)
    x[2, 999] = math.nan
    x[4, 0] = math.inf
    y, _, _ = ito.ito_layer_norm_fwd(x)
    for r in range(6):
        if r in (2, 4):
            assert bool(torch.isnan(y[r]).any())
        else:
            assert torch.equal(y[r], clean[r])


def test_layer_norm_gradient_by_differences(torch, ito):
    """d/dt of sum c y along a direction v, against sum dx v. L errs by at most the 32-bit evaluation's
    bound (6 u |c| (1 + |y|) an element, twice a difference, over 2h), the central difference by
    h^2/6 |L'''|, with |L'''| below 24 rstd^3 |v|^3 |c| for rows of unit spread."""
    rows, cols, h = 4, 48, 2.0 ** -7
    x, c, v = (normal(torch, (rows, cols), s) for s in (1, 2, 3))
    v = v / v.norm()
    gamma, beta = 1 + normal(torch, (cols,), 4, 0.2), normal(torch, (cols,), 5, 0.2)
    y, mean, rstd = ito.ito_layer_norm_fwd(x, gamma, beta)
    dx, dg, db = ito.ito_layer_norm_bwd(c, x, gamma, mean, rstd)

    def loss(xx, gg):
        return float((f64(ito.ito_layer_norm_fwd(xx, gg, beta)[0]) * f64(c)).sum())

    noise = (np.abs(f64(c)) * 6 * U * (1 + np.abs(f64(y)))).sum() / h
    rs = float(rstd.max())
    cut = h * h / 6 * 24 * rs ** 3 * float(c.norm()) * float(gamma.abs().max())
    assert abs((loss(x + h * v, gamma) - loss(x - h * v, gamma)) / (2 * h) - float((f64(dx) * f64(v)).sum())) <= noise + cut
    gp, gm = gamma.clone(), gamma.clone()
    gp[3] += h
    gm[3] -= h
    assert abs((loss(x, gp) - loss(x, gm)) / (2 * h) - float(dg[3])) <= noise
    assert db.shape == (cols,)


# --------------------------------------------------------- log probabilities

def logprobs64(X, tgt, k):
    rows, n = X.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = X.max(1, keepdims=True)
        shift = np.where(np.isfinite(top), top, 0)
        e = np.exp(X - shift)
        s = e.sum(1, keepdims=True)
        lse = (shift + np.log(s))[:, 0]
        lp = np.where(s > 0, (X - shift) - np.log(s), -np.inf)   # (not X - lse: a large lse absorbs log s)
        p = np.exp(lp)
        ent = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(1)
    logp = np.where(tgt >= 0, lp[np.arange(rows), np.maximum(tgt, 0)], 0.0)
    ids = np.stack([np.lexsort((np.arange(n), -X[r]))[:k] for r in range(rows)]).reshape(rows, k)
    return logp, ent, lse, ids, np.take_along_axis(lp, ids, 1), p, lp


def finite_within(got, want, tol, what):
    g = f64(got)
    assert np.array_equal(np.isfinite(g), np.isfinite(want)) and np.array_equal(g[~np.isfinite(want)], want[~np.isfinite(want)]), what
    f = np.isfinite(want)
    within(g[f], want[f], np.broadcast_to(tol, want.shape)[f], what)


def check_logprobs(torch, ito, x, tgt, k, dtype, seed=0):
    rows, n = x.shape
    logp, ent, lse, ids, top = ito.ito_token_logprobs_fwd(x, tgt, k=k)
    X, T = f64(x), tgt.cpu().numpy()
    wlogp, went, wlse, wids, wtop, p, lp = logprobs64(X, T, k)
    # exp errs by 2 units and its argument's rounding |x - top| u; the sum by its terms' number
    spread = np.where(np.isfinite(X), np.abs(X - np.where(np.isfinite(wlse), wlse, 0)[:, None]), 0)
    e_s = (n / 32 + 64) * U + (p * (spread + 4) * 4 * U).sum(1)
    mag = 1 + np.where(np.isfinite(wlse), np.abs(wlse), 0)
    e_lse = e_s + 6 * U * mag
    finite_within(lse, wlse, e_lse, "lse")
    xt = np.where(np.isfinite(wlogp), np.abs(wlogp), 0)
    finite_within(logp, wlogp, e_lse + 2 * U * xt, "logp")
    finite_within(ent, went, 2 * e_s + (n / 32 + 64) * U * (1 + (p * spread).sum(1)) + 4 * (p * spread * (spread + 4) * U).sum(1)
                  + 8 * U * (1 + math.log(n + 1)), "entropy")
    assert np.array_equal(ids.cpu().numpy(), wids)
    finite_within(top, wtop, (e_lse + 2 * U * mag)[:, None] + 2 * U * np.where(np.isfinite(wtop), np.abs(wtop), 0), "top_logp")
    # backward, from the saved lse and entropy
    gl, gh = normal(torch, (rows,), seed + 7, 0.5), normal(torch, (rows,), seed + 8, 0.2)
    d = ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl, gh)
    L, H = f64(lse)[:, None], f64(ent)[:, None]
    some = np.isfinite(L)
    with np.errstate(invalid="ignore"):
        lp = np.where(some, X - np.where(some, L, 0), -np.inf)
    p = np.where(np.isfinite(lp), np.exp(np.where(np.isfinite(lp), lp, 0)), 0)
    lp0 = np.where(np.isfinite(lp), lp, 0)
    hot = ((np.arange(n) == T[:, None]) & some).astype(np.float64)
    g, q = np.where(T >= 0, f64(gl), 0)[:, None], f64(gh)[:, None]
    want = g * (hot - p) - q * p * (lp0 + H)
    size = np.abs(g) * (hot + p) + np.abs(q) * p * (np.abs(lp0) + np.abs(H))
    e = 8 * U * size + (np.abs(g) + np.abs(q) * (np.abs(lp0) + np.abs(H) + 1)) * p * (np.abs(lp0) + np.abs(np.where(some, L, 0)) + 4) * 2 * U
    # below 2^-126 exp errs by two units of 2^-149, the products by one each
    e = e + 4 * TINY * (1 + np.abs(g) + np.abs(q) * (np.abs(lp0) + np.abs(H)))
    within_rounded(d, want, e, dtype, "dlogits")


LP_SIZES = [(1, 1, 1), (1, 10, 3), (3, 33, 32), (2, 1000, 8), (1, 131072, 8), (5, 4097, 20), (40, 1000, 5), (700, 257, 2),
            (3, 50001, 32), (2, 65536, 0), (300, 64, 1), (20, 9000, 6)]


@pytest.mark.parametrize("i,size", list(enumerate(LP_SIZES)))
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_logprobs(torch, ito, i, size, dtype):
    rows, n, k = size
    x = normal(torch, (rows, n), i, 2.5, dtype)
    g = torch.Generator(device="cuda").manual_seed(i)
    tgt = torch.randint(-1, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    check_logprobs(torch, ito, x, tgt, k, dtype, i)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n", [16, 1000, 40000])
def test_logprobs_masks(torch, ito, dtype, n):
    """Masked classes at either end, everywhere, everywhere but one, and the type's lowest value as a mask."""
    x = normal(torch, (9, n), n, 2.0, dtype)
    x[1, n // 2:] = -math.inf
    x[2, :n // 2] = -math.inf
    x[3] = -math.inf
    x[4] = -math.inf
    x[4, n - 3] = 1.5
    x[5, ::2] = -math.inf
    x[6] = torch.finfo(x.dtype).min
    x[7, 1:] = torch.finfo(x.dtype).min
    x[8] = 0.0
    tgt = torch.tensor([0, 1, n - 1, 2, n - 3, 1, 3, 0, -1], dtype=torch.int32, device="cuda")
    check_logprobs(torch, ito, x, tgt, min(n, 12), dtype)
    tgt = torch.tensor([0, n - 1, 0, -1, 0, 0, 0, 5, 2], dtype=torch.int32, device="cuda")   # masked targets
    check_logprobs(torch, ito, x, tgt, 1, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [10, 4000, 50000])
def test_logprobs_gradient_of_rows_at_the_lowest_value(torch, ito, dtype, n):
    """A row masked with the type's lowest value throughout is a uniform distribution, whatever its lse
    absorbs: p = 1 / n to the accuracy of n's logarithm in 32 bits, 16 u (1 + log n)."""
    low = torch.finfo(dt(torch, dtype)).min
    x = torch.full((3, n), low, dtype=dt(torch, dtype), device="cuda")
    x[1] = 100000.0
    x[2] = normal(torch, (n,), 1, 1.0, dtype)
    tgt = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    logp, ent, lse, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    gl = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    d = ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl)
    for r in (0, 1):
        want = np.full(n, -float(gl[r]) / n)
        want[r + 1] += float(gl[r])
        within_rounded(d[r], want, np.abs(float(gl[r])) * 16 * U * (1 + math.log(n)) * (1.0 / n + (want * float(gl[r]) > 0)), dtype)
        assert abs(float(logp[r]) + math.log(n)) <= 16 * U * (1 + math.log(n)) + n / 32 * U


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "saw"])
@pytest.mark.parametrize("n", [100, 5000, 70000])
def test_logprobs_alternatives_in_any_order(torch, ito, order, n):
    i = torch.arange(n, device="cuda", dtype=torch.float32)
    row = {"rising": i, "falling": -i, "equal": 0 * i, "saw": (i % 37)}[order] / 64
    x = torch.stack([row, row.flip(0)])
    check_logprobs(torch, ito, x, torch.tensor([0, n - 1], dtype=torch.int32, device="cuda"), 32, "float32")


@pytest.mark.parametrize("n", [50, 33000])
def test_logprobs_of_nan_and_infinity(torch, ito, n):
    x = normal(torch, (4, n), 1)
    clean = ito.ito_token_logprobs_fwd(x, torch.zeros(4, dtype=torch.int32, device="cuda"), k=3)
    x[1, 7] = math.nan
    x[3, n - 1] = math.inf
    logp, ent, lse, ids, top = ito.ito_token_logprobs_fwd(x, torch.zeros(4, dtype=torch.int32, device="cuda"), k=3)
    for r in (1, 3):
        assert all(bool(torch.isnan(t[r]).all()) for t in (logp, ent, lse, top))
    assert int(ids[1, 0]) == 7 and int(ids[3, 0]) == n - 1
    for r in (0, 2):
        assert all(torch.equal(a[r], b[r]) for a, b in zip((logp, ent, lse, ids, top), clean))


@pytest.mark.parametrize("dtype,n,pad,k", [("float32", 1537, 3, 3), ("bfloat16", 2500, 4, 9), ("float16", 1031, 1, 32),
                                           ("bfloat16", 2049, 0, 4), ("bfloat16", 3000, 0, 0),
                                           ("bfloat16", 1, 0, 1), ("float16", 5, 2, 3)])
def test_logprobs_of_many_rows(torch, ito, dtype, n, pad, k):
    """Rows enough for several to a warp, on 16 bytes or not, with rows in order, masked ends and whole masks."""
    rows = 30 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    x = normal(torch, (rows, n + pad), 3, 2.0, dtype)[:, :n]
    x[0::7] = x[0::7].sort(dim=1)[0]
    x[1::7] = x[1::7].sort(dim=1, descending=True)[0]
    x[2::7, n // 3:] = -math.inf
    x[3::70] = -math.inf
    x[4::70] = torch.finfo(x.dtype).min
    check_logprobs(torch, ito, x, torch.arange(rows, device="cuda", dtype=torch.int32) % n, k, dtype)


def test_logprobs_of_nan_among_many_rows(torch, ito):
    rows, n = 30 * torch.cuda.get_device_properties(0).multi_processor_count, 1500
    x = normal(torch, (rows, n), 1, 1.0, "bfloat16")
    clean = ito.ito_token_logprobs_fwd(x, None, k=4)[3:]
    x[1::2, 1234] = math.nan
    x[rows - 1] = math.nan
    ids, top = ito.ito_token_logprobs_fwd(x, None, k=4)[3:]
    assert all(torch.equal(a[0::2], b[0::2]) for a, b in zip((ids, top), clean))
    assert bool(torch.isnan(top[1::2]).all()) and bool((ids[1:-1:2, 0] == 1234).all())
    assert torch.equal(ids[1:-2:2, 1:], x[1:-2:2].nan_to_num(nan=-math.inf).float().sort(dim=1, descending=True, stable=True)[1][:, :3].int())
    assert ids[rows - 1].cpu().tolist() == [0, 1, 2, 3]


def test_logprobs_negative_zero_ties_with_zero(torch, ito):
    x = torch.full((1, 64), -1.0, device="cuda")
    x[0, 9], x[0, 4], x[0, 30] = 0.0, -0.0, 0.0
    ids = ito.ito_token_logprobs_fwd(x, None, k=3)[3]
    assert ids.cpu().tolist() == [[4, 9, 30]]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 6), (5, 2)])
@pytest.mark.parametrize("size", [(3, 1000), (1, 40000), (200, 130)])
def test_logprobs_strided(torch, ito, dtype, offset, pad, size):
    rows, n = size
    x = normal(torch, (rows, n + offset + pad), 1, 2.0, dtype)[:, offset:offset + n]
    check_logprobs(torch, ito, x, torch.arange(rows, device="cuda", dtype=torch.int32) % n, 4, dtype)


def test_logprobs_strided_gradient_keeps_its_padding(torch, ito):
    x = normal(torch, (6, 100), 1, 1.0, "bfloat16")
    tgt = torch.arange(6, device="cuda", dtype=torch.int32)
    _, ent, lse, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    gl = normal(torch, (6,), 2)
    want = ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl)
    buf = torch.full((6, 107), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl, out=buf[:, 3:103]), want)
    buf[:, 3:103] = 7.0
    assert bool((buf == 7.0).all())
    same = x.clone()
    assert torch.equal(ito.ito_token_logprobs_bwd(same, tgt, lse, ent, gl, out=same), want)


def test_logprobs_gradient_terms(torch, ito):
    """Either term alone; a target outside the classes is no token and is reported."""
    x = normal(torch, (5, 300), 1)
    tgt = torch.tensor([3, -1, 299, 0, 7], dtype=torch.int32, device="cuda")
    _, ent, lse, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    gl, gh = normal(torch, (5,), 2), normal(torch, (5,), 3)
    zero = torch.zeros_like(gl)
    assert torch.equal(ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl), ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl, zero))
    assert torch.equal(ito.ito_token_logprobs_bwd(x, None, lse, ent, None, gh),
                       ito.ito_token_logprobs_bwd(x, tgt, lse, ent, zero, gh))
    torch.cuda.synchronize()
    assert ito.ito_get_error() == ito.ITO_OK
    bad = tgt.clone()
    bad[0], bad[4] = 300, -2
    logp = ito.ito_token_logprobs_fwd(x, bad)[0]
    assert ito.ito_get_error() == ito.ITO_ERR_ARG
    assert float(logp[0]) == 0.0 and float(logp[4]) == 0.0
    none = tgt.clone()
    none[0], none[4] = -1, -1
    d = ito.ito_token_logprobs_bwd(x, bad, lse, ent, gl, gh)
    assert ito.ito_get_error() == ito.ITO_ERR_ARG
    assert torch.equal(d, ito.ito_token_logprobs_bwd(x, none, lse, ent, gl, gh))


def test_logprobs_gradient_by_differences(torch, ito):
    """Central differences along a unit direction: values err by 16 u (1 + |lse|) a row and the
    difference by h^2/6 of a third derivative below 2 a row for logp, 12 for the entropy."""
    rows, n, h = 3, 40, 2.0 ** -6
    x, v = normal(torch, (rows, n), 1), normal(torch, (rows, n), 2)
    v = v / v.norm()
    tgt = torch.tensor([5, 0, 39], dtype=torch.int32, device="cuda")
    gl, gh = normal(torch, (rows,), 3), normal(torch, (rows,), 4)
    _, ent, lse, _, _ = ito.ito_token_logprobs_fwd(x, tgt)
    d = ito.ito_token_logprobs_bwd(x, tgt, lse, ent, gl, gh)

    def value(xx):
        logp, e, _, _, _ = ito.ito_token_logprobs_fwd(xx, tgt)
        return float((f64(gl) * f64(logp) + f64(gh) * f64(e)).sum())

    noise = (16 * U * (1 + np.abs(f64(lse))) * (np.abs(f64(gl)) + np.abs(f64(gh)))).sum() / h
    cut = h * h / 6 * (2 * np.abs(f64(gl)) + 12 * np.abs(f64(gh))).sum()
    assert abs((value(x + h * v) - value(x - h * v)) / (2 * h) - float((f64(d) * f64(v)).sum())) <= noise + cut


# ------------------------------------------------------------------- AdamW

def mix(seed, step, tensor, n):
    """The rounding's random words, as include/ito.h's hash is defined in the kernel's comment."""
    m = np.uint64(0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64)
    key = (seed + step * 0x9E3779B1 + tensor * 0x510E527F) & 0xFFFFFFFF
    h = (i * np.uint64(0x6A09E667) + np.uint64(key)) & m
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0xBB67AE85)) & m
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0x6A09E667)) & m
    h ^= h >> np.uint64(16)
    return h & np.uint64(0xFFFFF), ((h * np.uint64(0x510E527F)) & m) >> np.uint64(12)


def decode(code, exp, first):
    """float64 values of 8-bit moments, by the header's formula."""
    n = code.size
    e = np.repeat(exp.astype(np.float64), 128)[:n]
    c = code.astype(np.int64)
    mag = c & 127 if first else c
    v = np.where(mag > 0, 2.0 ** (e - (15 if first else 31) + (mag >> 3)) * (1 + (mag & 7) / 8), 0.0)
    if first:
        v = np.where(c >= 128, -v, v)
    return np.where(e == -128, np.nan, v)


def encode(x, rnd, first):
    """Codes and exponents of float32 values: E from the block's largest value rounded up to four
    bits; a code is the value's bits, counted from the lowest binade, rounded up by chance."""
    n = x.size
    low, bias = (-111, 112) if first else (-95, 96)
    mag = np.abs(x).view(np.uint32).astype(np.int64)
    blocks = -(-n // 128)
    codes, exps = np.zeros(n, np.uint8), np.zeros(blocks, np.int8)
    for b in range(blocks):
        s = slice(128 * b, min(n, 128 * b + 128))
        top = mag[s].max()
        if top >= 0x7F800000:
            exps[b] = -128
            continue
        e = max(low, ((min(top, 0x7F700000) + 0xFFFFF) >> 23) - 127)
        t = np.minimum(mag[s], 0x7F700000) - ((e + bias) << 23)
        c = np.where(t >= 0, (t + rnd[s].astype(np.int64)) >> 20, 0)
        if first:
            c = np.where((x[s] < 0) & (c > 0), c + 128, c)
        else:
            c = np.where(mag[s] > 0, np.maximum(c, 1), c)
        exps[b] = e
        codes[s] = c
    return codes, exps


def adamw32(w, g, m, v, k, wd):
    """One step, every operation rounded to 32 bits in the documented order."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = g.astype(f) * f(k["grad_scale"])
        m = m * f(k["b1"]) + g * f(1 - k["b1"])
        v = v * f(k["b2"]) + (g * g) * f(1 - k["b2"])
        den = np.sqrt(v) * f(1 / math.sqrt(1 - k["b2"] ** k["t"])) + f(k["eps"])
        w = w * f(1 - k["lr"] * wd) - (m * f(k["lr"] / (1 - k["b1"] ** k["t"]))) / den
    return w, m, v


def same_bits(torch, got, want):
    g = got.cpu().numpy().reshape(-1)
    return np.array_equal(g.view(np.uint32 if g.dtype == np.float32 else g.dtype),
                          want.view(np.uint32 if want.dtype == np.float32 else want.dtype)) or \
        (g.dtype == np.float32 and np.array_equal(g, want, equal_nan=True))


def bf16_of(torch, w, dtype):
    return torch.from_numpy(w).to(dtype)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("copies", [None, "bfloat16", "float16"])
def test_adamw_steps(torch, ito, bits, grad, copies):
    """Five steps over tensors of odd and even sizes at odd and even offsets of one buffer: weights,
    copies, moments (codes and exponents) equal a program that rounds after every operation."""
    sizes = [1, 10, 127, 128, 129, 640, 0, 4096, 8192, 8193, 20000, 33]
    n = sum(sizes)
    rng = np.random.default_rng(bits)
    w = rng.normal(0, 0.1, n).astype(np.float32)
    flat = torch.from_numpy(w.copy()).cuda()
    ws = list(torch.split(flat, sizes))
    cf = None if copies is None else torch.zeros(n, dtype=dt(torch, copies), device="cuda")
    decays = [0.0 if i % 3 == 0 else 0.1 for i in range(len(sizes))]
    opt = ito.AdamW(ws, bits=bits, betas=(0.9, 0.99), eps=1e-8, weight_decay=decays,
                    copies=None if cf is None else list(torch.split(cf, sizes)), seed=77)
    at = np.concatenate([[0], np.cumsum(sizes)])
    ms, vs = ([np.zeros(s, np.float32) for s in sizes] for _ in range(2))
    codes = [None] * len(sizes)
    for t in range(1, 6):
        g = torch.from_numpy((rng.normal(0, 1, n) * 10.0 ** rng.integers(-6, 1, n)).astype(np.float32)).cuda().to(dt(torch, grad))
        opt.step(list(torch.split(g, sizes)), lr=1e-2, grad_scale=0.5)
        G = g.float().cpu().numpy()
        k = dict(b1=0.9, b2=0.99, eps=1e-8, lr=1e-2, grad_scale=0.5, t=t)
        for i, s in enumerate(sizes):
            sl = slice(at[i], at[i + 1])
            w[sl], ms[i], vs[i] = adamw32(w[sl], G[sl], ms[i], vs[i], k, decays[i])
            if bits == 8 and s:
                um, uv = mix(77, t, i, s)
                (mc, me), (vc, ve) = encode(ms[i], um, True), encode(vs[i], uv, False)
                codes[i] = (mc, vc, me, ve)
                ms[i], vs[i] = decode(mc, me, True).astype(np.float32), decode(vc, ve, False).astype(np.float32)
    assert same_bits(torch, flat, w)
    if cf is not None:
        assert torch.equal(cf.cpu(), bf16_of(torch, w, dt(torch, copies)))
    for i, s in enumerate(sizes):
        if not s:
            continue
        if bits == 32:
            assert same_bits(torch, opt.states[0][i], ms[i]) and same_bits(torch, opt.states[1][i], vs[i])
        else:
            for got, want in zip((st[i] for st in opt.states), codes[i]):
                assert np.array_equal(got.cpu().numpy(), want)
    m, v = opt.moments()
    assert np.array_equal(m.float().cpu().numpy(), np.concatenate(ms)) and np.array_equal(v.float().cpu().numpy(), np.concatenate(vs))
    if bits == 8:
        m, v = opt.moments(torch.float32)
        assert np.array_equal(m.cpu().numpy(), np.concatenate(ms)) and np.array_equal(v.cpu().numpy(), np.concatenate(vs))


def encode_whole(x, rnd, first):
    """encode() for whole blocks, all at once."""
    low, bias = (-111, 112) if first else (-95, 96)
    mag = np.abs(x).view(np.uint32).astype(np.int64).reshape(-1, 128)
    top = mag.max(1)
    e = np.maximum(low, ((np.minimum(top, 0x7F700000) + 0xFFFFF) >> 23) - 127)
    t = np.minimum(mag, 0x7F700000) - ((e[:, None] + bias) << 23)
    c = np.where(t >= 0, (t + rnd.astype(np.int64).reshape(-1, 128)) >> 20, 0)
    if first:
        c = np.where((x.reshape(-1, 128) < 0) & (c > 0), c + 128, c)
    else:
        c = np.where(mag > 0, np.maximum(c, 1), c)
    bad = top >= 0x7F800000
    return np.where(bad[:, None], 0, c).reshape(-1).astype(np.uint8), np.where(bad, -128, e).astype(np.int8)


@pytest.mark.parametrize("grad,copies", [("bfloat16", "bfloat16"), ("float32", None), ("float16", "float16")])
def test_adamw_large_tensors_in_8_bits(torch, ito, grad, copies):
    """Tensors of many chunks, their ends and odd neighbours: three steps equal the program that
    rounds after every operation; a NaN and an infinity stay in their blocks."""
    sizes = [1 << 20, 128, 65536 + 4096 + 256, 1 << 21, 640, 65536]
    n = sum(sizes)
    at = np.concatenate([[0], np.cumsum(sizes)])
    rng = np.random.default_rng(3)
    w = rng.normal(0, 0.1, n).astype(np.float32)
    flat = torch.from_numpy(w.copy()).cuda()
    cf = None if copies is None else torch.zeros(n, dtype=dt(torch, copies), device="cuda")
    opt = ito.AdamW(list(torch.split(flat, sizes)), bits=8, weight_decay=0.1, seed=9,
                    copies=None if cf is None else list(torch.split(cf, sizes)))
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    for t in range(1, 4):
        g = (rng.normal(0, 1, n) * 10.0 ** rng.integers(-4, 1, n)).astype(np.float32)
        if t == 2:
            g[5000], g[(1 << 20) + 200 + 70000] = np.nan, np.inf
        g = torch.from_numpy(g).cuda().to(dt(torch, grad))
        opt.step(list(torch.split(g, sizes)), lr=1e-2)
        k = dict(b1=0.9, b2=0.999, eps=1e-8, lr=1e-2, grad_scale=1.0, t=t)
        w, m, v = adamw32(w, g.float().cpu().numpy(), m, v, k, 0.1)
        codes = []
        for i, s in enumerate(sizes):
            sl = slice(at[i], at[i + 1])
            um, uv = mix(9, t, i, s)
            (mc, me), (vc, ve) = encode_whole(m[sl], um, True), encode_whole(v[sl], uv, False)
            codes.append((mc, vc, me, ve))
            m[sl], v[sl] = decode(mc, me, True).astype(np.float32), decode(vc, ve, False).astype(np.float32)
    for i in range(len(sizes)):
        for got, want in zip((st[i] for st in opt.states), codes[i]):
            assert np.array_equal(got.cpu().numpy(), want), i
    assert same_bits(torch, flat, w)
    if cf is not None:
        ok = torch.from_numpy(np.isfinite(w))
        assert torch.equal(cf.cpu()[ok], bf16_of(torch, w, dt(torch, copies))[ok])
    bad = np.isnan(m)
    assert bad.sum() == 256 and bad[4992:5120].all()


def test_adamw_against_64_bits(torch, ito):
    """One step's formula in 64 bits. Each moment is two rounded products and a rounded sum; the step
    is a root, two products, a sum, a product and a quotient of them: 12 units of its size."""
    n = 5000
    w, g = normal(torch, (n,), 1, 0.1), normal(torch, (n,), 2, 0.01)
    m, v = normal(torch, (n,), 3, 0.01), normal(torch, (n,), 4, 0.01).square()
    W, G, M, V = f64(w), f64(g), f64(m), f64(v)
    opt = ito.AdamW([w], states=[[m], [v]], step=9, weight_decay=0.02)
    opt.step([g], lr=1e-3)
    M1, V1 = 0.9 * M + 0.1 * G, 0.999 * V + 0.001 * G * G
    within(m, M1, 4 * U * (0.9 * np.abs(M) + 0.1 * np.abs(G)))
    within(v, V1, 5 * U * V1)
    step = 1e-3 / (1 - 0.9 ** 10) * M1 / (np.sqrt(V1 / (1 - 0.999 ** 10)) + 1e-8)
    size = 1e-3 / (1 - 0.9 ** 10) * (0.9 * np.abs(M) + 0.1 * np.abs(G)) / (np.sqrt(V1 / (1 - 0.999 ** 10)) + 1e-8)
    want = W * (1 - 1e-3 * 0.02) - step
    within(w, want, 3 * U * np.abs(W) + 16 * U * size)


def test_adamw_many_tensors(torch, ito):
    """More tensors than one launch's table holds, as one tensor at a time."""
    sizes = [(37 * i) % 900 + 1 for i in range(130)]
    flat, g = normal(torch, (sum(sizes),), 1), normal(torch, (sum(sizes),), 2)
    alone = flat.clone()
    opt = ito.AdamW(list(torch.split(flat, sizes)))
    for _ in range(2):
        opt.step(list(torch.split(g, sizes)), lr=0.01)
    for w, gr in zip(torch.split(alone, sizes), torch.split(g, sizes)):
        one = ito.AdamW([w])
        for _ in range(2):
            one.step([gr], lr=0.01)
    assert torch.equal(flat, alone)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_nonfinite_and_extreme_gradients(torch, ito, bits):
    """A NaN or an infinity reaches its element's (8 bits: its block's) state and no other; the
    smallest and largest gradients neither hang, wrap nor turn a positive v into zero."""
    n = 1024
    w = torch.ones(n, device="cuda")
    g = normal(torch, (n,), 1, 1e-3)
    g[200], g[700] = math.nan, math.inf
    g[300:310] = 0.0
    g[400:420] = 1e-30
    g[900] = 3e18
    opt = ito.AdamW([w], bits=bits, weight_decay=0.0)
    opt.step([g], lr=1e-3)
    m, v = (t.float().cpu().numpy() for t in opt.moments())
    G = g.cpu().numpy()
    if bits == 32:
        assert np.isnan(m[200]) and np.isinf(m[700])
        assert np.isfinite(np.delete(m, [200, 700])).all()
    else:
        assert np.isnan(m[128:256]).all() and np.isnan(m[640:768]).all()
        assert np.isfinite(np.concatenate([m[:128], m[256:640], m[768:]])).all()
        f = np.isfinite(v)
        assert (v[f & (np.float32(0.001) * (G * G) > 0)] > 0).all()
    out = w.cpu().numpy()
    assert np.isnan(out[200]) and (out[300:310] == 1.0).all()
    assert np.isfinite(np.delete(out, [200, 700])).all()


def test_adamw_rounding_is_unbiased(torch, ito):
    """The second moment of a constant gradient follows its course although each step's change is
    far below a code's step: the mean of 16384 elements after 200 steps. A code's relative
    step is at most 1/8, so a step's rounding has a relative deviation of at most 1/16, decaying
    with b2; their sum's deviation is below sqrt(200) / 16 = 0.89 of the value, an average of
    16384 elements' 0.0069, and six of those 0.042."""
    n, b2 = 16384, 0.999
    w = torch.zeros(n, device="cuda")
    opt = ito.AdamW([w], bits=8, betas=(0.9, b2), weight_decay=0.0, seed=5)
    g = torch.full((n,), 0.01, device="cuda")
    big = torch.full((n,), 0.1, device="cuda")
    opt.step([big], lr=0.0)
    v = float(opt.moments()[1].double().mean())
    want = (1 - b2) * 0.01
    assert abs(v / want - 1) <= 0.042
    for _ in range(199):
        opt.step([g], lr=0.0)
    want = want * b2 ** 199 + (1 - b2 ** 199) * 1e-4
    assert abs(float(opt.moments()[1].double().mean()) / want - 1) <= 0.042


# ------------------------------------------------- streams, graphs, refusals

def _calls(torch, ito):
    """One call of each operator, as closures over their inputs: -> list of (call(stream), outputs)."""
    x, W = normal(torch, (40, 256), 1, 1.0, "bfloat16"), normal(torch, (264, 256), 2, 0.1, "bfloat16")
    x1 = normal(torch, (1, 256), 9, 1.0, "bfloat16")
    odd, wodd = normal(torch, (40, 251), 1, 1.0, "bfloat16"), normal(torch, (264, 251), 2, 0.1, "bfloat16")
    big, wbig = normal(torch, (512, 512), 3, 1.0, "float16"), normal(torch, (768, 512), 4, 0.1, "float16")
    dy, z = normal(torch, (40, 264), 5, 1.0, "bfloat16"), normal(torch, (40, 264), 6, 1.0, "bfloat16")
    logits = normal(torch, (9, 20000), 7, 2.0)
    tgt = torch.arange(9, device="cuda", dtype=torch.int32)
    _, ent, lse, _, _ = ito.ito_token_logprobs_fwd(logits, tgt)
    _, mean, rstd = ito.ito_layer_norm_fwd(x)
    gl = normal(torch, (9,), 8)
    return [lambda s: ito.ito_fp_linear_fwd(x, W, act="gelu", stream=s),
            lambda s: ito.ito_fp_linear_fwd(x1, W, act="gelu", stream=s),
            lambda s: ito.ito_fp_linear_fwd(odd, wodd, act="silu", stream=s),
            lambda s: ito.ito_fp_linear_fwd(big, wbig, stream=s),
            lambda s: ito.ito_fp_linear_bwd(dy, x, W, z=z, act="silu", stream=s),
            lambda s: ito.ito_layer_norm_fwd(x, stream=s),
            lambda s: ito.ito_layer_norm_bwd(x, x, None, mean, rstd, stream=s),
            lambda s: ito.ito_token_logprobs_fwd(logits, tgt, k=4, stream=s),
            lambda s: ito.ito_token_logprobs_bwd(logits, tgt, lse, ent, gl, stream=s)]


def _flat(r):
    return [r] if hasattr(r, "detach") else list(r)


def test_float_ops_on_another_stream_and_twice(torch, ito):
    """The same bits on the default stream, on another stream, and on two streams at once."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for call in _calls(torch, ito):
        want = _flat(call(None))
        torch.cuda.synchronize()
        got = [_flat(call(s)) for s in (a, b, a, b)]
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(p, q) for p, q in zip(g, want))


def test_float_ops_in_a_graph(torch, ito):
    for call in _calls(torch, ito):
        want = [t.clone() for t in _flat(call(None))]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(None)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = _flat(call(None))
        for t in got:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_float_ops_leave_no_error(torch, ito):
    torch.cuda.synchronize()
    assert ito.ito_get_error() == ito.ITO_OK


def test_wrapper_refusals(torch, ito):
    x, W = normal(torch, (4, 16), 1, 1.0, "bfloat16"), normal(torch, (8, 16), 2, 1.0, "bfloat16")

    def refuses(code, f):
        with pytest.raises(ito.ItoError) as e:
            f()
        assert e.value.code == code

    arg, shape = ito.ITO_ERR_ARG, ito.ITO_ERR_SHAPE
    refuses(shape, lambda: ito.ito_fp_linear_fwd(x, W[:, :8]))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x, W.half()))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x.float(), W.float()))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x.t().contiguous().t(), W))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x, W, act="selu"))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x, W, act=7))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x, W, out_dtype=torch.float16))
    refuses(shape, lambda: ito.ito_fp_linear_fwd(x, W, bias=torch.zeros(9, device="cuda")))
    refuses(arg, lambda: ito.ito_fp_linear_fwd(x.cpu(), W))
    refuses(shape, lambda: ito.ito_fp_linear_fwd(x[:0], W))
    refuses(arg, lambda: ito.ito_fp_linear_bwd(normal(torch, (4, 8), 3, 1.0, "bfloat16"), x, W, act="gelu"))
    refuses(arg, lambda: ito.ito_layer_norm_fwd(x, gamma=torch.zeros(16, dtype=torch.float16, device="cuda")))
    refuses(arg, lambda: ito.ito_layer_norm_fwd(x, eps=-1.0))
    refuses(shape, lambda: ito.ito_layer_norm_fwd(x[:, :0]))
    refuses(arg, lambda: ito.ito_layer_norm_fwd(x.double()))
    tgt = torch.zeros(4, dtype=torch.int32, device="cuda")
    refuses(arg, lambda: ito.ito_token_logprobs_fwd(x, tgt.long()))
    refuses(arg, lambda: ito.ito_token_logprobs_fwd(x, tgt, k=33))
    refuses(shape, lambda: ito.ito_token_logprobs_fwd(x, tgt, k=17))
    refuses(shape, lambda: ito.ito_token_logprobs_fwd(x[:0], tgt[:0]))
    w = torch.zeros(10, device="cuda")
    refuses(arg, lambda: ito.AdamW([w], bits=16))
    refuses(arg, lambda: ito.AdamW([w.half()]))
    refuses(shape, lambda: ito.AdamW([]))
    refuses(shape, lambda: ito.AdamW([w], copies=[torch.zeros(9, dtype=torch.bfloat16, device="cuda")]))
    opt = ito.AdamW([w])
    refuses(shape, lambda: opt.step([], lr=0.1))
    refuses(shape, lambda: opt.step([torch.zeros(9, device="cuda")], lr=0.1))
    assert opt.steps == 0
