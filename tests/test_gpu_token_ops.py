"""The gated layer, the linear cross entropy and the embedding against plain computations in 64 bits,
their gradients against the formulas and against differences, and their behaviour on other streams, in
graphs, on strides, masks and the smallest sizes.

Tolerances are bounds of the arithmetic, as in test_gpu_float_ops.py: U = 2^-24, a sum of n products is
off by at most 2 n U sum|terms|, and a result's own rounding needs none."""
import math

import numpy as np
import pytest

from test_gpu_float_ops import ACTS, LINEAR_SIZES, TINY, U, act64, dt, f64, normal, rounding_error, slope64, within, \
    within_rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


# --------------------------------------------------------------- embedding

def tokens(torch, kind, n, classes, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        ids = torch.full((n,), classes - 1, dtype=torch.int64, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    elif kind == "even":
        ids = torch.randint(0, classes, (n,), generator=g, device="cuda")
    elif kind == "up":
        ids = torch.arange(n, device="cuda") % classes
    elif kind == "down":
        ids = classes - 1 - torch.arange(n, device="cuda") % classes
    else:       # few frequent tokens, many rare ones, some places without one
        u = torch.rand((n,), generator=g, device="cuda", dtype=torch.float64)
        ids = (classes ** u - 1).long().clamp(0, classes - 1)
        ids[torch.rand((n,), generator=g, device="cuda") < 0.1] = -1
    return ids.to(torch.int32)


EMB_SIZES = [(1, 1, 1), (1, 5, 787), (2, 2, 3), (7, 50001, 787), (31, 100, 8), (32, 3, 16), (33, 255, 256), (65, 256, 250),
             (300, 257, 264), (1000, 17, 1), (2047, 65535, 40), (2049, 65536, 24), (5000, 70000, 8), (4096, 300, 1024),
             (20000, 1000, 72), (9000, 40, 520), (4097, 257, 16), (8192, 70000, 8), (8193, 300, 24), (50000, 3000, 40),
             (65537, 66000, 8)]
KINDS = ("text", "one", "even", "up", "down", "none")
TYPES = ("float32", "bfloat16", "float16")


@pytest.mark.parametrize("i,size", list(enumerate(EMB_SIZES)))
@pytest.mark.parametrize("dtype", TYPES)
def test_embedding_fwd(torch, ito, i, size, dtype):
    n, classes, d = size
    ids = tokens(torch, KINDS[i % 6], n, classes, i)
    table = normal(torch, (classes, d), i + 1, 0.5, dtype)
    for out in TYPES:
        y = ito.ito_embedding_fwd(ids, table, scale=3.7, out_dtype=dt(torch, out))
        want = table[ids.long().clamp(min=0)].float() * np.float32(3.7).item()
        want[ids < 0] = 0
        assert y.dtype == dt(torch, out) and torch.equal(y, want.to(y.dtype))
    y = ito.ito_embedding_fwd(ids, table)          # a scale of 1 copies
    want = table[ids.long().clamp(min=0)]
    want[ids < 0] = 0
    assert torch.equal(y, want)


def check_embedding_bwd(torch, ito, dy, ids, classes, scale, out, add=None):
    n, d = dy.shape
    before = None if add is None else f64(add)
    keep = None if add is None else add.clone()
    got = ito.ito_embedding_bwd(dy, ids, classes, scale=scale, dtype=dt(torch, out), add_to=add)
    assert got.shape == (classes, d) and got.dtype == dt(torch, out) and (add is None or got is add)
    I, D = ids.cpu().numpy(), f64(dy)
    s = float(np.float32(scale))
    want, mags, count = np.zeros((classes, d)), np.zeros((classes, d)), np.zeros((classes, 1))
    there = I >= 0
    np.add.at(want, I[there], D[there])
    np.add.at(mags, I[there], np.abs(D[there]))
    np.add.at(count, I[there], 1)
    e = (count + 1) * U * mags * abs(s)
    want = want * s
    if add is not None:
        e = e + U * (np.abs(want) + np.abs(before) + e) * (count > 0)
        want = want + before
    within_rounded(got, want, e, out, "dtable")
    absent = torch.from_numpy(count[:, 0] == 0).cuda()
    if add is None:
        assert bool((got[absent] == 0).all())
    else:
        assert torch.equal(got[absent], keep[absent])


@pytest.mark.parametrize("i,size", list(enumerate(EMB_SIZES)))
@pytest.mark.parametrize("dtype", TYPES)
def test_embedding_bwd(torch, ito, i, size, dtype):
    n, classes, d = size
    k = i + TYPES.index(dtype)
    dy = normal(torch, (n, d), i, 1.0, dtype)
    for j in range(2):
        ids = tokens(torch, KINDS[(k + 3 * j) % 6], n, classes, i + 7)
        out = "float32" if (k + j) % 2 else dtype
        check_embedding_bwd(torch, ito, dy, ids, classes, (1.0, 0.25, 28.3)[k % 3], out)
        check_embedding_bwd(torch, ito, dy, ids, classes, 2.5, out, add=normal(torch, (classes, d), i + 9, 1.0, out))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 8, 9, 31, 32, 33, 64, 100, 256, 257, 2000, 70000])
def test_embedding_bwd_chunks(torch, ito, kind, n):
    """Runs of equal tokens that fill chunks, end with them, go on through many, and all at once."""
    for classes, d in ((3, 40), (500, 300)):
        check_embedding_bwd(torch, ito, normal(torch, (n, d), n, 1.0, "bfloat16"), tokens(torch, kind, n, classes, n),
                            classes, 1.0, "float32")


def test_embedding_bwd_long_rows_in_large_chunks(torch, ito):
    """Places enough for chunks of 32, with a token that fills most of them."""
    n, classes, d = 12000, 1000, 1032
    ids = tokens(torch, "text", n, classes, 5)
    ids[1000:9000] = 17
    check_embedding_bwd(torch, ito, normal(torch, (n, d), 6, 1.0, "float16"), ids, classes, 0.5, "float32")
    check_embedding_bwd(torch, ito, normal(torch, (n, d), 6, 1.0, "float16"), ids, classes, 0.5, "float16",
                        add=normal(torch, (classes, d), 7, 1.0, "float16"))


@pytest.mark.parametrize("classes", [1, 40000, 3000000])
def test_embedding_of_many_classes(torch, ito, classes):
    """Tables of one row and of more than 2^21 (keys of three digits; presence noted in several rounds)."""
    ids = tokens(torch, "even", 700, classes, 3)
    dy = normal(torch, (700, 9), 4)
    got = ito.ito_embedding_bwd(dy, ids, classes)
    want = torch.zeros((classes, 9), dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dy.double())
    within(got, f64(want), f64(torch.zeros_like(want).index_add_(0, ids.long(), dy.double().abs())) * 702 * U, "dtable")


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (8, 16)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_embedding_strided(torch, ito, offset, pad, dtype):
    n, classes, d = 70, 33, 136
    ids = tokens(torch, "text", n, classes, 1)
    wide = normal(torch, (classes, d + offset + pad), 2, 1.0, dtype)
    table = wide[:, offset:offset + d]
    want = table[ids.long().clamp(min=0)].clone()
    want[ids < 0] = 0
    assert torch.equal(ito.ito_embedding_fwd(ids, table), want)
    dy = normal(torch, (n, d + offset + pad), 3, 1.0, dtype)[:, offset:offset + d]
    check_embedding_bwd(torch, ito, dy, ids, classes, 1.5, dtype)
    keep = wide.clone()
    check_embedding_bwd(torch, ito, dy, ids, classes, 1.5, dtype, add=table)
    wide[:, offset:offset + d] = keep[:, offset:offset + d]
    assert torch.equal(wide, keep)                 # what lies beside the rows is left alone


def test_embedding_ids_out_of_range(torch, ito):
    """They stand for no token and leave an error to be read; the rest of the call is as without them."""
    ids = torch.tensor([3, 9, -2, 0, -1, 1 << 30, -(1 << 31), 3], dtype=torch.int32, device="cuda")
    clean = torch.tensor([3, -1, -1, 0, -1, -1, -1, 3], dtype=torch.int32, device="cuda")
    table, dy = normal(torch, (9, 40), 1), normal(torch, (8, 40), 2)
    assert ito._lib.ito_get_error() == 0
    want = ito.ito_embedding_fwd(clean, table), ito.ito_embedding_bwd(dy, clean, 9)
    assert ito._lib.ito_get_error() == 0
    got = ito.ito_embedding_fwd(ids, table)
    assert ito._lib.ito_get_error() == ito.ITO_ERR_ARG and torch.equal(got, want[0])
    got = ito.ito_embedding_bwd(dy, ids, 9)
    assert ito._lib.ito_get_error() == ito.ITO_ERR_ARG and torch.equal(got, want[1])
    assert ito._lib.ito_get_error() == 0


def test_embedding_keeps_nan_in_its_row(torch, ito):
    ids = tokens(torch, "even", 400, 50, 1)
    dy = normal(torch, (400, 72), 2, 1.0, "bfloat16")
    clean = ito.ito_embedding_bwd(dy, ids, 50)
    dy[200, 5] = math.nan
    dy[300] = math.inf
    ids[100] = -1
    dy[100] = math.nan                              # a place without a token
    base = dy.clone()
    base[200, 5], base[300] = 0, 0
    got = ito.ito_embedding_bwd(dy, ids, 50)
    a, b = int(ids[200]), int(ids[300])
    bad = torch.zeros((50, 72), dtype=torch.bool, device="cuda")
    bad[a, 5], bad[b] = True, True
    assert torch.equal(~torch.isfinite(got), bad) and clean.shape == got.shape


def test_embedding_beyond_32_bits(torch, ito):
    """Offsets into the table and the rows that pass 2^31 elements."""
    classes, d = 600000, 4096                       # 2.5e9 elements of 16 bits
    table = torch.empty((classes, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([classes - 1, 0, 530000, classes - 1], dtype=torch.int32, device="cuda")
    rows = normal(torch, (4, d), 1, 1.0, "bfloat16")
    table[ids[:3].long()] = rows[:3]
    assert torch.equal(ito.ito_embedding_fwd(ids, table)[:3], rows[:3])
    table.fill_(1.0)
    got = ito.ito_embedding_bwd(rows, ids, classes, add_to=table)
    # (a sum of two, one more with 1, rounded once)
    assert torch.equal(got[530000], (rows[2].float() + 1).bfloat16())
    assert torch.equal(got[classes - 1], (rows[0].float() + rows[3].float() + 1).bfloat16())
    assert bool((got[classes - 2] == 1).all())


# ------------------------------------------------------------- gated layer

def check_gated_fwd(torch, ito, B, IC, OC, dtype, act, bias, save_z, seed=0, x=None, Wg=None, Wu=None):
    x = normal(torch, (B, IC), seed + 1, 1.0, dtype) if x is None else x
    Wg = normal(torch, (OC, IC), seed + 2, IC ** -0.5, dtype) if Wg is None else Wg
    Wu = normal(torch, (OC, IC), seed + 3, IC ** -0.5, dtype) if Wu is None else Wu
    bg = normal(torch, (OC,), seed + 4, 0.5, bias) if bias else None
    bu = normal(torch, (OC,), seed + 5, 0.5, bias) if bias else None
    got = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, bias_g=bg, bias_u=bu, act=act, save_z=save_z)
    h, zg, zu = got if save_z else (got, None, None)
    X = f64(x)
    z, e = [], []
    for W, b in ((Wg, bg), (Wu, bu)):
        s, m = X @ f64(W).T, np.abs(X) @ np.abs(f64(W)).T
        if b is not None:
            s, m = s + f64(b), m + np.abs(f64(b))
        z.append(s)
        e.append(2 * (IC + 1) * U * m)
    a = act64(act, z[0])
    # as the linear layer's activation, then a product of two values that are each off
    ea = 1.13 * e[0] + 8 * U * (1 + np.abs(z[0])) * (act != "none")
    want = a * z[1]
    eh = ea * (np.abs(z[1]) + e[1]) + np.abs(a) * e[1]
    eh = eh + U * (np.abs(want) + eh)
    assert h.shape == (B, OC) and h.dtype == x.dtype
    within_rounded(h, want, eh, dtype, "h")
    if save_z:
        within_rounded(zg, z[0], e[0], dtype, "zg")
        within_rounded(zu, z[1], e[1], dtype, "zu")


def check_gated_bwd(torch, ito, B, IC, OC, dtype, act, dw_dtype, seed=0, x=None, Wg=None, Wu=None, dh=None, zg=None, zu=None):
    x = normal(torch, (B, IC), seed + 1, 1.0, dtype) if x is None else x
    Wg = normal(torch, (OC, IC), seed + 2, IC ** -0.5, dtype) if Wg is None else Wg
    Wu = normal(torch, (OC, IC), seed + 3, IC ** -0.5, dtype) if Wu is None else Wu
    dh = normal(torch, (B, OC), seed + 4, 1.0, dtype) if dh is None else dh
    zg = normal(torch, (B, OC), seed + 5, 2.0, dtype) if zg is None else zg
    zu = normal(torch, (B, OC), seed + 6, 1.0, dtype) if zu is None else zu
    got = ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, act=act, need_dbias=True, dw_dtype=dt(torch, dw_dtype))
    X, D, G, Z = f64(x), f64(dh), f64(zg), f64(zu)
    some = act != "none"
    dzg, dzu = D * Z * slope64(act, G), D * act64(act, G)
    # the slope's and the activation's evaluation in 32 bits, the products' roundings
    e0g = np.abs(D * Z) * 16 * U * (1 + np.abs(G)) * some + 2 * U * np.abs(dzg)
    e0u = np.abs(D) * 8 * U * (1 + np.abs(G)) * some + U * np.abs(dzu)
    want_x, e_x, a_x = 0, 0, 0
    for k, (dz, e0, W) in enumerate(((dzg, e0g, Wg), (dzu, e0u, Wu))):
        ez = e0 + rounding_error(np.abs(dz) + e0, dtype)
        a = np.abs(dz) + ez
        want_x, e_x, a_x = want_x + dz @ f64(W), e_x + ez @ np.abs(f64(W)), a_x + a @ np.abs(f64(W))
        within_rounded(got[1 + k], dz.T @ X, ez.T @ np.abs(X) + 2 * B * U * (a.T @ np.abs(X)), dw_dtype, "dW %d" % k)
        within(got[3 + k], dz.sum(0), e0.sum(0) + (B + 1) * U * (np.abs(dz) + e0).sum(0) + TINY, "dbias %d" % k)
    within_rounded(got[0], want_x, e_x + 2 * 2 * OC * U * a_x, dtype, "dx")


GATED_SIZES = LINEAR_SIZES + [(12, 520, 1000), (24, 136, 72), (200, 64, 4000), (256, 4096, 160), (400, 776, 700),
                              (1100, 200, 1000)]


@pytest.mark.parametrize("i,size", list(enumerate(GATED_SIZES)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_gated_fwd(torch, ito, i, size, dtype):
    n = i + (dtype == "float16") * 2
    check_gated_fwd(torch, ito, *size, dtype, ACTS[n % 5], (None, dtype, "float32")[n % 3], n % 2 == 0, seed=10 * i)
    check_gated_fwd(torch, ito, *size, dtype, ACTS[(n + 2) % 5], (dtype, "float32", None)[n % 3], n % 2 == 1, seed=10 * i + 5)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 256, 384), (12, 256, 384), (100, 256, 384), (512, 256, 512), (300, 4096, 128)])
def test_gated_every_activation(torch, ito, act, size):
    check_gated_fwd(torch, ito, *size, "bfloat16", act, "bfloat16", True)
    check_gated_bwd(torch, ito, *size, "float16", act, "float32")


@pytest.mark.parametrize("i,size", list(enumerate(GATED_SIZES)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_gated_bwd(torch, ito, i, size, dtype):
    n = i + (dtype == "float16")
    check_gated_bwd(torch, ito, *size, dtype, ACTS[n % 5], dtype if n % 2 else "float32", seed=10 * i)


def test_gated_bwd_parts(torch, ito):
    """Each gradient alone is the gradient among the others, bit for bit."""
    for B, IC, OC in ((200, 136, 264), (5, 136, 72), (600, 520, 1000)):
        x, dh = normal(torch, (B, IC), 1, 1.0, "bfloat16"), normal(torch, (B, OC), 2, 1.0, "bfloat16")
        Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "bfloat16") for s in (3, 4))
        zg, zu = (normal(torch, (B, OC), s, 1.0, "bfloat16") for s in (5, 6))
        full = ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, need_dbias=True)
        for k, mine in (("need_dx", (0,)), ("need_dw", (1, 2)), ("need_dbias", (3, 4))):
            need = {n: n == k for n in ("need_dx", "need_dw", "need_dbias")}
            part = ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, **need)
            assert [p is not None for p in part] == [j in mine for j in range(5)]
            for j in mine:
                assert torch.equal(part[j], full[j])


# (columns, rows of a weight): fewer than a tile's, one more, ragged ends; the last two give each warp many chunks
FEW_SIZES = [(1, 1), (2, 16), (3, 40), (7, 17), (8, 15), (63, 33), (64, 16), (65, 1000), (130, 257), (264, 5000), (520, 70),
             (4096, 4000), (2051, 7511)]


@pytest.mark.parametrize("B", [1, 7, 8, 9, 16, 17])
@pytest.mark.parametrize("i,size", list(enumerate(FEW_SIZES)))
def test_gradients_of_few_rows(torch, ito, i, size, B):
    n = i + B
    dtype = ("bfloat16", "float16")[n % 2]
    check_gated_bwd(torch, ito, B, *size, dtype, ACTS[n % 5], "float32" if n % 3 else dtype, seed=n)
    x, W, t = make_ce(torch, B, *size, dtype, n, masked=n % 4 > 0)
    _, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = normal(torch, (B,), n + 3).abs() + 0.1
    check_ce_bwd(torch, ito, x, W, t, lse, g, None, dtype, dtype if n % 3 else "float32")


@pytest.mark.parametrize("offset,pad", [(0, 0), (0, 8), (1, 0), (2, 3), (5, 2), (7, 1)])
@pytest.mark.parametrize("size", [(1, 1, 3), (3, 5, 40), (9, 65, 33), (16, 130, 257), (8, 72, 1000)])
def test_gradients_of_few_rows_amid_nan(torch, ito, offset, pad, size):
    """Neither what lies between and around the rows of x and the weights nor the workspace's old contents come into the
    results, and what lies between the results' rows is left as it was."""
    B, IC, OC = size
    lib = ito._lib

    def amid(rows, cols, seed, scale):
        t = normal(torch, (rows, cols), seed, scale, "bfloat16")
        wide = torch.full((rows * (cols + offset + pad) + 16,), math.nan, dtype=torch.bfloat16, device="cuda")
        v = torch.as_strided(wide, (rows, cols), (cols + offset + pad, 1), offset)
        v.copy_(t)
        return t, v

    (x, xv), (Wg, gv), (Wu, uv) = (amid(r, IC, s, sc) for r, s, sc in ((B, 1, 1.0), (OC, 2, 0.2), (OC, 3, 0.2)))
    dh, zg, zu = (normal(torch, (B, OC), s, 1.0, "bfloat16") for s in (4, 5, 6))
    t = torch.randint(0, OC, (B,), device="cuda", dtype=torch.int32)
    _, lse = ito.ito_linear_cross_entropy_fwd(x, Wg, t)
    g = torch.ones(B, device="cuda")
    # Logits of rows at other alignments are added in another order: dl may be rounded to the other side, half a step or
    # 2^-8 of it each, and so the results (the 32-bit sums' own errors: the last factor).
    dl = torch.exp(x.double() @ Wg.double().T - lse.double()[:, None])
    dl[torch.arange(B, device="cuda"), t.long()] -= 1.0
    apart = [4 * 2.0 ** -8 * 1.01 * m for m in (dl.abs() @ Wg.double().abs(), dl.abs().T @ x.double().abs())]
    ld = IC + offset + pad
    xs, gs, us = (xv.data_ptr(), ld), (gv.data_ptr(), ld), (uv.data_ptr(), ld)
    for dw in (torch.bfloat16, torch.float32):
        ty = ito.ITO_BF16 if dw is torch.bfloat16 else ito.ITO_F32
        wants = (ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, dw_dtype=dw)[:3],
                 ito.ito_linear_cross_entropy_bwd(x, Wg, t, lse, g, dw_dtype=dw))
        for k, want in enumerate(wants):
            bufs = [torch.full((w.shape[0] * ld + 16,), 7.0, dtype=w.dtype, device="cuda") for w in want]
            out = [v for b in bufs for v in (b.data_ptr() + offset * b.element_size(), ld)]
            n = (lib.ito_linear_cross_entropy_bwd_workspace_size(*xs, *gs, B, IC, OC) if k else
                 lib.ito_fp_gated_linear_bwd_workspace_size(*xs, *gs, *us, B, IC, OC))
            ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
            if k:
                r = lib.ito_linear_cross_entropy_bwd(*xs, *gs, ito.ITO_BF16, t.data_ptr(), lse.data_ptr(), g.data_ptr(), None,
                                                     ty, B, IC, OC, ito._aligned256(ws), n, *out, ito._stream())
            else:
                r = lib.ito_fp_gated_linear_bwd(dh.data_ptr(), OC, zg.data_ptr(), OC, zu.data_ptr(), OC, *xs, *gs, *us,
                                                ito.ITO_BF16, ty, ito.ITO_ACT_SILU, B, IC, OC, ito._aligned256(ws), n, *out,
                                                None, None, ito._stream())
            assert r == 0
            for b, w, e in zip(bufs, want, apart if k else want):
                cells = torch.as_strided(b, tuple(w.shape), (ld, 1), offset)
                if k:
                    assert bool(((cells.double() - w.double()).abs() <= e).all())
                else:                    # the same products in the same order
                    assert torch.equal(cells, w)
                cells.fill_(7.0)
                assert bool((b == 7.0).all())


@pytest.mark.parametrize("B", [4, 13, 40])
def test_gated_bwd_without_what_it_does_not_read(torch, ito, B):
    """x may be missing where no dW is asked for, the weights where no dx is."""
    IC, OC = 133, 77
    x, dh = normal(torch, (B, IC), 1, 1.0, "float16"), normal(torch, (B, OC), 2, 1.0, "float16")
    Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "float16") for s in (3, 4))
    zg, zu = (normal(torch, (B, OC), s, 1.0, "float16") for s in (5, 6))
    want = ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu)
    got = [torch.full_like(w, 7.0) for w in want[:3]]
    dz = [v for t in (dh, zg, zu) for v in (t.data_ptr(), OC)]
    for dx in (True, False):
        xs = (None, IC) if dx else (x.data_ptr(), IC)
        ws = (Wg.data_ptr(), IC, Wu.data_ptr(), IC) if dx else (None, IC, None, IC)
        outs = [v for k, t in enumerate(got) for v in (t.data_ptr() if (k == 0) == dx else None, IC)]
        n = ito._lib.ito_fp_gated_linear_bwd_workspace_size(*xs, *ws, B, IC, OC)
        buf = torch.empty(n + 512, dtype=torch.uint8, device="cuda")
        assert ito._lib.ito_fp_gated_linear_bwd(*dz, *xs, *ws, ito.ITO_F16, ito.ITO_F16, ito.ITO_ACT_SILU, B, IC, OC,
                                                ito._aligned256(buf), n, *outs, None, None, ito._stream()) == 0
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_gated_one_bias(torch, ito):
    x = normal(torch, (150, 72), 1, 1.0, "bfloat16")
    Wg, Wu = (normal(torch, (136, 72), s, 0.1, "bfloat16") for s in (2, 3))
    b, zero = normal(torch, (136,), 4), torch.zeros(136, device="cuda")
    for rows in (150, 3):
        for g, u in ((b, None), (None, b)):
            full = ito.ito_fp_gated_linear_fwd(x[:rows], Wg, Wu, bias_g=zero if g is None else g,
                                               bias_u=zero if u is None else u, save_z=True)
            part = ito.ito_fp_gated_linear_fwd(x[:rows], Wg, Wu, bias_g=g, bias_u=u, save_z=True)
            assert all(torch.equal(p, q) for p, q in zip(part, full))


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 7), (3, 5), (8, 16), (2, 1)])
@pytest.mark.parametrize("size", [(1, 136, 72), (40, 136, 72), (300, 264, 320)])
def test_gated_strided_and_misaligned(torch, ito, offset, pad, size):
    B, IC, OC = size

    def inside(rows, cols, seed, scale=1.0):
        wide = normal(torch, (rows, cols + offset + pad), seed, scale, "bfloat16")
        return wide[:, offset:offset + cols]

    x, Wg, Wu = inside(B, IC, 1), inside(OC, IC, 2, IC ** -0.5), inside(OC, IC, 3, IC ** -0.5)
    dh, zg, zu = (inside(B, OC, s) for s in (4, 5, 6))
    aligned = normal(torch, (OC, IC), 7, IC ** -0.5, "bfloat16")
    check_gated_fwd(torch, ito, B, IC, OC, "bfloat16", "silu", "float32", True, x=x, Wg=Wg, Wu=Wu)
    check_gated_fwd(torch, ito, B, IC, OC, "bfloat16", "gelu", None, True, x=x, Wg=aligned, Wu=Wu)
    check_gated_bwd(torch, ito, B, IC, OC, "bfloat16", "gelu", "bfloat16", x=x, Wg=Wg, Wu=Wu, dh=dh, zg=zg, zu=zu)
    check_gated_bwd(torch, ito, B, IC, OC, "bfloat16", "silu", "float32", x=x, Wg=Wg, Wu=aligned, dh=dh, zg=zg, zu=zu)


@pytest.mark.parametrize("offset,ld", [(0, 80), (1, 79), (4, 84), (3, 77)])
@pytest.mark.parametrize("B", [1, 12, 100, 300])
def test_gated_strided_outputs_keep_their_padding(torch, ito, offset, ld, B):
    IC, OC = 64, 72
    x = normal(torch, (B, IC), 1, 1.0, "float16")
    Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "float16") for s in (2, 3))
    want = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, act="gelu", save_z=True)
    bufs = [torch.full((B * ld + offset + 8,), 7.0, dtype=torch.float16, device="cuda") for _ in range(3)]
    a = (x.data_ptr(), IC, Wg.data_ptr(), IC, Wu.data_ptr(), IC)
    n = ito._lib.ito_fp_gated_linear_fwd_workspace_size(*a, B, IC, OC)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    h, zg, zu = (b.data_ptr() + 2 * offset for b in bufs)
    assert ito._lib.ito_fp_gated_linear_fwd(*a, None, None, ito.ITO_F16, 0, ito.ITO_ACT_GELU, B, IC, OC,
                                            ito._aligned256(ws), n, zg, ld, zu, ld, h, ld, ito._stream()) == 0
    for b, w in zip(bufs, want):
        cells = torch.as_strided(b, (B, OC), (ld, 1), offset)
        assert torch.equal(cells, w)
        cells.fill_(7.0)
        assert bool((b == 7.0).all())


@pytest.mark.parametrize("size", [(1, 70, 40), (20, 300, 136), (150, 300, 136), (300, 300, 264)])
def test_gated_keeps_rows_apart(torch, ito, size):
    """A NaN in one row of x, or of one weight, reaches that row, or column, of h alone; in the saved zg only
    where it is zg's."""
    B, IC, OC = size
    x = normal(torch, (B, IC), 1, 1.0, "bfloat16")
    Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "bfloat16") for s in (2, 3))
    clean = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, save_z=True)
    x2 = x.clone()
    x2[B // 2, IC - 1] = math.nan
    keep = torch.arange(B, device="cuda") != B // 2
    for got, c in zip(ito.ito_fp_gated_linear_fwd(x2, Wg, Wu, save_z=True), clean):
        assert bool(torch.isnan(got[B // 2]).all()) and torch.equal(got[keep], c[keep])
    W2 = Wu.clone()
    W2[OC - 1, 0] = math.nan
    h, zg, zu = ito.ito_fp_gated_linear_fwd(x, Wg, W2, save_z=True)
    assert torch.equal(zg, clean[1]) and bool(torch.isnan(zu[:, OC - 1]).all()) and bool(torch.isnan(h[:, OC - 1]).all())
    assert torch.equal(h[:, :OC - 1], clean[0][:, :OC - 1])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [3, 40, 256])
def test_gated_gradients_by_differences(torch, ito, act, B):
    """Differences of L = sum c h against the gradients, for an element of a bias of each side (float32, so a
    step is exact). h is rounded to float16: off by 2^-11 |h| an element; the product is linear in u, and
    the activations' third derivatives stay below 3."""
    IC, OC, h = 24, 40, 2.0 ** -4
    g = torch.Generator(device="cuda").manual_seed(B)

    def few(shape, hi):
        return (torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").float() / 16).to(torch.float16)

    x, Wg, Wu, c = few((B, IC), 16), few((OC, IC), 8), few((OC, IC), 8), few((B, OC), 16)
    bg, bu = few((OC,), 16).float(), few((OC,), 16).float()
    if act == "relu":
        bg = bg.round() + 2.0 ** -9      # (z is a multiple of 1/256 off it: no corner within h only for the column below)
    _, zg, zu = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, bias_g=bg, bias_u=bu, act=act, save_z=True)
    dbg, dbu = ito.ito_fp_gated_linear_bwd(c, x, Wg, Wu, zg, zu, act=act, need_dbias=True)[3:]

    def column(b_g, b_u, j):
        return f64(ito.ito_fp_gated_linear_fwd(x, Wg, Wu, bias_g=b_g, bias_u=b_u, act=act))[:, j]

    C, G, Z = np.abs(f64(c)), np.abs(f64(zg)), np.abs(f64(zu))
    for j in (7, 33):
        for which, (b, d) in enumerate(((bg, dbg), (bu, dbu))):
            if act == "relu" and which == 0 and float(G[:, j].min()) < 2 * h:
                continue                 # a corner inside the step: a difference is no derivative there
            up, down = b.clone(), b.clone()
            up[j] += h
            down[j] -= h
            args = [(up, bu), (down, bu)] if which == 0 else [(bg, up), (bg, down)]
            lp, lm = column(*args[0], j), column(*args[1], j)
            got = ((lp - lm) * f64(c)[:, j]).sum() / (2 * h)
            rounding = (C[:, j] * 2.0 ** -11 * (np.abs(lp) + np.abs(lm) + 2.0 ** -13)).sum() / (2 * h)
            third = 0.0 if which or act in ("none", "relu") else 3 * h * h / 6 * (C[:, j] * Z[:, j]).sum()
            saved = (C[:, j] * 2.0 ** -11 * (1.13 * G[:, j] + (1 + G[:, j]) * Z[:, j] * 2)).sum()    # z's own roundings
            assert abs(got - float(d[j])) <= rounding + third + saved + 1e-4 * C[:, j].sum() * (1 + G + Z)[:, j].max()


# ------------------------------------------------------ linear cross entropy

def make_ce(torch, rows, d, classes, dtype, seed, masked=True, scale=2.0):
    x = normal(torch, (rows, d), seed, 1.0, dtype)
    W = normal(torch, (classes, d), seed + 1, scale * d ** -0.5, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    t = torch.randint(0, classes, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if masked:
        t[torch.rand((rows,), generator=g, device="cuda") < 0.25] = -1
    return x, W, t


def check_ce_fwd(torch, ito, x, W, t):
    """Each logit is off by eL; a row's sum of exponentials passes through at most 40 changes of its largest
    value and 64 additions, each exponential off by 4 U (1 + its exponent), the exponents' sum at most the
    logits' range twice."""
    rows, d = x.shape
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    X, V = x.double(), W.double()
    L = X @ V.T
    eL = (2 * (d + 1) * U * (X.abs() @ V.abs().T)).amax(1)
    want = torch.logsumexp(L, 1)
    span = L.amax(1) - L.amin(1)
    s = torch.log(torch.exp(L - L.amax(1, keepdim=True)).sum(1))
    e = eL + U * (224 + 8 * span) + 2 * U * s.abs() + U * want.abs() + TINY
    within(lse, f64(want), f64(e), "lse")
    tt = t.long()
    hit = L.gather(1, tt.clamp(min=0)[:, None])[:, 0]
    l = torch.where(tt >= 0, want - hit, torch.zeros_like(hit))
    within(loss, f64(l), f64(e + eL + U * l.abs()) * (f64(t) >= 0), "loss")
    return loss, lse


def check_ce_bwd(torch, ito, x, W, t, lse, g, g_lse, dtype, dw_dtype, pieces=1):
    rows, d = x.shape
    classes = W.shape[0]
    dx, dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, g_lse, dw_dtype=dt(torch, dw_dtype))
    X, V = x.double(), W.double()
    D = X @ V.T
    eL = 2 * (d + 1) * U * (X.abs() @ V.abs().T)
    far = (D - lse.double()[:, None])
    eL = torch.expm1(eL + 6 * U * (1 + far.abs()))           # relative, of p
    p = torch.exp(far)
    del D, far
    tt = t.long()
    gg = torch.where(tt >= 0, g, torch.zeros_like(g)).double()
    a = gg + (0 if g_lse is None else g_lse.double())
    dl = a[:, None] * p
    e = dl.abs() * (eL + 2 * U) + a.abs()[:, None] * 2.0 ** -126     # (an exponential below 2^-126 comes as 0)
    del p, eL
    rows_hit = (tt >= 0).nonzero()[:, 0]
    dl[rows_hit, tt[rows_hit]] -= gg[rows_hit]
    e = e + U * dl.abs()
    S = 1.0
    if dtype == "float16":
        most = float((g.abs() + (0 if g_lse is None else g_lse.abs())).max())
        S = 2.0 ** min(max(13 - math.frexp(most)[1], -100), 100) if most > 0 else 1.0
    half, floor = {"bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25)}[dtype]
    e = e + (dl.abs() + e) * half * (1 + 2.0 ** -20) + floor / S
    m = dl.abs() + e
    want = dl @ V
    ex = e @ V.abs() + (2 * classes + pieces) * U * (m @ V.abs())
    within_rounded(dx, f64(want), f64(ex), dtype, "dx")
    want = dl.T @ X
    ew = e.T @ X.abs() + 2 * rows * U * (m.T @ X.abs())
    within_rounded(dw, f64(want), f64(ew), dw_dtype, "dW")


CE_SIZES = [(1, 1, 1), (1, 64, 1000), (1, 4096, 777), (2, 787, 50001), (3, 8, 2), (5, 100, 16), (9, 264, 4097), (16, 512, 640),
            (17, 64, 64), (31, 128, 1031), (32, 64, 10), (33, 4096, 128), (64, 72, 9000), (100, 1000, 333), (128, 128, 128),
            (129, 65, 257), (257, 264, 1511), (300, 2048, 1000), (512, 64, 5000), (700, 72, 2032)]


@pytest.mark.parametrize("i,size", list(enumerate(CE_SIZES)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_cross_entropy(torch, ito, i, size, dtype):
    rows, d, classes = size
    n = i + (dtype == "float16")
    x, W, t = make_ce(torch, rows, d, classes, dtype, 10 * i, masked=i % 3 > 0)
    loss, lse = check_ce_fwd(torch, ito, x, W, t)
    g = (normal(torch, (rows,), i + 3).abs() + 0.1) * (1.0 if n % 3 else 1.0 / rows)
    g_lse = normal(torch, (rows,), i + 4, 0.1) if n % 2 else None
    check_ce_bwd(torch, ito, x, W, t, lse, g, g_lse, dtype, "float32" if n % 2 else dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_cross_entropy_in_pieces(torch, ito, dtype):
    """Rows enough for three pieces of the vocabulary, the last one narrower; targets in each."""
    rows, d, classes = 70000, 24, 4200
    x, W, t = make_ce(torch, rows, d, classes, dtype, 5)
    loss, lse = check_ce_fwd(torch, ito, x, W, t)
    check_ce_bwd(torch, ito, x, W, t, lse, torch.full((rows,), 1.0 / rows, device="cuda"), None, dtype, "float32", pieces=3)


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (8, 16)])
@pytest.mark.parametrize("size", [(1, 136, 72), (40, 136, 720), (300, 264, 520)])
def test_cross_entropy_strided_and_misaligned(torch, ito, offset, pad, size):
    rows, d, classes = size

    def inside(n, cols, seed, scale):
        return normal(torch, (n, cols + offset + pad), seed, scale, "bfloat16")[:, offset:offset + cols]

    x, W = inside(rows, d, 1, 1.0), inside(classes, d, 2, d ** -0.5)
    t = make_ce(torch, rows, 1, classes, "bfloat16", 3)[2]
    loss, lse = check_ce_fwd(torch, ito, x, W, t)
    check_ce_bwd(torch, ito, x, W, t, lse, normal(torch, (rows,), 4), None, "bfloat16", "bfloat16")


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_cross_entropy_of_far_logits(torch, ito, rows):
    """Logits in the thousands: the largest class takes nearly all, and classes far below it add nothing."""
    x, W, t = make_ce(torch, rows, 64, 500, "bfloat16", 8, scale=300.0)
    loss, lse = check_ce_fwd(torch, ito, x, W, t)
    check_ce_bwd(torch, ito, x, W, t, lse, torch.ones(rows, device="cuda"), None, "bfloat16", "float32")


@pytest.mark.parametrize("rows", [2, 20, 130, 300])
def test_cross_entropy_of_infinities_and_nan(torch, ito, rows):
    """Classes whose every logit is -inf take no part; a row of them only; a NaN and a +inf stay in their row.
    Every row has a first element of 1, which W's column picks up."""
    d, classes = 72, 300
    x, W, t = make_ce(torch, rows, d, classes, "bfloat16", 9, masked=False)
    x[:, 0] = 1.0
    W[:, 0] = 0.0
    t[:] = torch.arange(rows, device="cuda", dtype=torch.int32) % 100
    part = ito.ito_linear_cross_entropy_fwd(x, W[:200].contiguous(), t)
    W[200:, 0] = -math.inf
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    within(lse, f64(part[1]), U * 64 * (1 + np.abs(f64(lse))), "lse")
    within(loss, f64(part[0]), U * 64 * (1 + np.abs(f64(lse))), "loss")
    # (a class of -inf has p = 0, but its row of W is an operand of dx: 0 times -inf is a NaN there, as in any product)
    dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.ones(rows, device="cuda"), need_dx=False)[1]
    assert bool((dw[200:] == 0).all()) and bool(torch.isfinite(dw[:200]).all())
    W[:, 0] = -math.inf
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    assert bool((lse == -math.inf).all()) and bool((loss == math.inf).all())
    dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.ones(rows, device="cuda"), need_dx=False)[1]
    assert bool((dw == 0).all())
    W[:, 0] = 0.0
    clean = ito.ito_linear_cross_entropy_fwd(x, W, t)
    for bad in (math.nan, math.inf):
        y = x.clone()
        y[1, 5] = bad
        for got, c in zip(ito.ito_linear_cross_entropy_fwd(y, W, t), clean):
            assert bool(torch.isnan(got[1])) and torch.equal(got[2:], c[2:]) and torch.equal(got[:1], c[:1])


@pytest.mark.parametrize("rows", [3, 50, 300])
def test_cross_entropy_targets(torch, ito, rows):
    """-1 has no loss and no gradient; other targets outside the classes the same, with an error to be read."""
    x, W, t = make_ce(torch, rows, 40, 700, "bfloat16", 3, masked=False)
    none = torch.full_like(t, -1)
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, none)
    assert bool((loss == 0).all()) and torch.equal(lse, ito.ito_linear_cross_entropy_fwd(x, W, t)[1])
    one = torch.ones(rows, device="cuda")
    assert all(bool((g == 0).all()) for g in ito.ito_linear_cross_entropy_bwd(x, W, none, lse, one))
    # with lse's factor the rows without a token have its term alone, like rows whose loss has the factor 0
    for got, want in zip(ito.ito_linear_cross_entropy_bwd(x, W, none, lse, one, one),
                         ito.ito_linear_cross_entropy_bwd(x, W, t, lse, 0 * one, one)):
        assert torch.equal(got, want)
    assert ito._lib.ito_get_error() == 0
    bad, clean = t.clone(), t.clone()
    bad[0], bad[1], clean[0], clean[1] = 700, -5, -1, -1
    want = ito.ito_linear_cross_entropy_fwd(x, W, clean)
    got = ito.ito_linear_cross_entropy_fwd(x, W, bad)
    assert ito._lib.ito_get_error() == ito.ITO_ERR_ARG and all(torch.equal(a, b) for a, b in zip(got, want))
    want = ito.ito_linear_cross_entropy_bwd(x, W, clean, lse, one)
    got = ito.ito_linear_cross_entropy_bwd(x, W, bad, lse, one)
    assert ito._lib.ito_get_error() == ito.ITO_ERR_ARG and all(torch.equal(a, b) for a, b in zip(got, want))


def test_cross_entropy_padding_rows_with_nan(torch, ito):
    """Rows without a token that hold NaN: the loss of the others, and their dx, are as without them. (x of such a
    row is an operand of dW, so its values have to be finite for dW; 0 of them is what a padded batch holds.)"""
    x, W, t = make_ce(torch, 200, 64, 300, "bfloat16", 6, masked=False)
    t[100:] = -1
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    dx, _ = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.ones(200, device="cuda"))
    x[100:] = math.nan
    loss2, lse2 = ito.ito_linear_cross_entropy_fwd(x, W, t)
    dx2, _ = ito.ito_linear_cross_entropy_bwd(x, W, t, lse2, torch.ones(200, device="cuda"))
    assert torch.equal(loss, loss2) and torch.equal(lse[:100], lse2[:100]) and torch.equal(dx, dx2)


def test_cross_entropy_small_factors_in_float16(torch, ito):
    """Factors far below float16's range: the gradients scale with them exactly (a power of two), down to
    float16's own range of the results, so float32 ones show it."""
    x, W, t = make_ce(torch, 60, 64, 2000, "float16", 4)
    _, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = normal(torch, (60,), 5).abs() + 0.1
    dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, dw_dtype=torch.float32)[1]
    tiny = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g * 2.0 ** -40, dw_dtype=torch.float32)[1]
    assert torch.equal(dw * 2.0 ** -40, tiny)
    zero = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, 0 * g)
    assert all(bool((z == 0).all()) for z in zero)


@pytest.mark.parametrize("junk", [1e30, -1e30, math.inf, math.nan])
@pytest.mark.parametrize("rows", [5, 90])
def test_cross_entropy_factors_of_rows_without_a_token(torch, ito, junk, rows):
    """What they hold is not looked at: not for the gradient, and not for float16's factor."""
    x, W, t = make_ce(torch, rows, 64, 300, "float16", 14)
    t[::3] = -1
    _, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    g = normal(torch, (rows,), 5).abs() * 2.0 ** -20
    want = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.where(t < 0, torch.zeros_like(g), g), dw_dtype=torch.float32)
    got = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.where(t < 0, torch.full_like(g, junk), g), dw_dtype=torch.float32)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((want[1] != 0).any())


def test_cross_entropy_parts(torch, ito):
    for rows, d, classes in ((300, 136, 1000), (7, 64, 333)):
        x, W, t = make_ce(torch, rows, d, classes, "bfloat16", 4)
        _, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
        g = normal(torch, (rows,), 5)
        full = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g)
        dx, none = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, need_dw=False)
        assert none is None and torch.equal(dx, full[0])
        none, dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, need_dx=False)
        assert none is None and torch.equal(dw, full[1])


@pytest.mark.parametrize("rows", [4, 200])
def test_cross_entropy_gradient_by_differences(torch, ito, rows):
    """Differences of L = sum g loss for an element of x and one of W, against dx and dW. The loss is in 32 bits,
    off by at most 64 U (1 + |lse|) a row; |third derivative| along a logit's direction stays below |w|^3."""
    d, classes, h = 32, 90, 2.0 ** -4
    gen = torch.Generator(device="cuda").manual_seed(rows)
    few = lambda shape: (torch.randint(-16, 17, shape, generator=gen, device="cuda").float() / 32).to(torch.float16)  # noqa: E731
    x, W = few((rows, d)), few((classes, d))
    t = torch.randint(0, classes, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    g = torch.rand((rows,), generator=gen, device="cuda") + 0.5
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    dx, dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, g, dw_dtype=torch.float32)

    def total(xx, ww):
        return (f64(ito.ito_linear_cross_entropy_fwd(xx, ww, t)[0]) * f64(g)).sum()

    noise = (64 * U * (1 + np.abs(f64(lse))) * f64(g)).sum() / h
    i, j = rows // 2, 7
    xp, xm = x.clone(), x.clone()
    xp[i, j] += h
    xm[i, j] -= h
    top = np.abs(f64(W)[:, j]).max()
    tol = noise + h * h / 6 * float(g[i]) * 8 * top ** 3 + float(g[i]) * top * 2 * 2.0 ** -10
    assert abs((total(xp, W) - total(xm, W)) / (2 * h) - float(dx[i, j])) <= tol
    c = int(t[i])
    wp, wm = W.clone(), W.clone()
    wp[c, j] += h
    wm[c, j] -= h
    X = np.abs(f64(x)[:, j])
    tol = noise + (f64(g) * (h * h / 6 * X ** 3 + X * 2.0 ** -10)).sum()
    assert abs((total(x, wp) - total(x, wm)) / (2 * h) - float(dw[c, j])) <= tol


# ------------------------------------------------- streams, graphs, refusals

def _calls(torch, ito, seed=0):
    """Calls of every entry point over its paths (few rows, tensor cores, K slices, pieces), as thunks."""
    out = []
    for B, IC, OC in ((1, 264, 136), (40, 2048, 128), (300, 264, 520), (300, 133, 77)):
        x, dh = normal(torch, (B, IC), seed + 1, 1.0, "bfloat16"), normal(torch, (B, OC), seed + 2, 1.0, "bfloat16")
        Wg, Wu = (normal(torch, (OC, IC), seed + s, 0.1, "bfloat16") for s in (3, 4))
        zg, zu = (normal(torch, (B, OC), seed + s, 1.0, "bfloat16") for s in (5, 6))
        out.append(lambda s=None, a=(x, Wg, Wu): ito.ito_fp_gated_linear_fwd(*a, save_z=True, stream=s))
        out.append(lambda s=None, a=(dh, x, Wg, Wu, zg, zu): ito.ito_fp_gated_linear_bwd(*a, need_dbias=True, stream=s))
        for dtype in ("bfloat16", "float16"):
            x, W, t = make_ce(torch, B, IC, 3 * OC + 1, dtype, seed + 7)
            lse, g = normal(torch, (B,), seed + 8).abs() + 8, normal(torch, (B,), seed + 9)
            out.append(lambda s=None, a=(x, W, t): ito.ito_linear_cross_entropy_fwd(*a, stream=s))
            out.append(lambda s=None, a=(x, W, t, lse, g): ito.ito_linear_cross_entropy_bwd(*a, stream=s))
        ids, table = tokens(torch, "text", 10 * B, OC, seed + 10), normal(torch, (OC, IC), seed + 11)
        dy = normal(torch, (10 * B, IC), seed + 12, 1.0, "float16")
        out.append(lambda s=None, a=(ids, table): ito.ito_embedding_fwd(*a, scale=2.0, stream=s))
        out.append(lambda s=None, a=(dy, ids, OC): ito.ito_embedding_bwd(*a, scale=2.0, stream=s))
        out.append(lambda s=None, a=(dy, ids, OC), t=table: ito.ito_embedding_bwd(*a, add_to=t.clone(), stream=s))
    return out


def _flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def same(torch, a, b):
    return all(torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8)) for p, q in zip(_flat(a), _flat(b)))


def test_token_ops_on_another_stream_and_twice(torch, ito):
    calls = _calls(torch, ito)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [c() for c in calls]
    s.synchronize()
    assert all(same(torch, a, b) for a, b in zip(got, want))
    assert all(same(torch, c(), w) for c, w in zip(calls, want))
    s.wait_stream(torch.cuda.current_stream())      # (what a call clones is made on the current stream)
    got = []
    for c in calls:
        torch.cuda.current_stream().synchronize()
        got.append(c(s))
    s.synchronize()
    assert all(same(torch, a, b) for a, b in zip(got, want))


def test_token_ops_on_two_streams_at_once(torch, ito):
    """The same calls on two streams beside one another, on different values: neither disturbs the other."""
    first, second = _calls(torch, ito, 0), _calls(torch, ito, 500)
    want = [[c() for c in calls] for calls in (first, second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for a, b in zip(first, second):
        for k, c in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(c())
    torch.cuda.synchronize()
    for k in range(2):
        assert all(same(torch, a, b) for a, b in zip(got[k], want[k]))


def test_token_ops_in_a_graph(torch, ito):
    """Captured once, replayed on other values: the values of eager calls; two graphs hold memory of their own."""
    calls = _calls(torch, ito)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([c() for c in calls])
        graphs.append(g)
    for r in outs[0] + outs[1]:
        for t in _flat(r):
            t.fill_(-3)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(same(torch, a, b) for a, b in zip(o, want))


def test_token_ops_leave_no_error(torch, ito):
    for c in _calls(torch, ito):
        c()
    assert ito._lib.ito_get_error() == 0


def test_token_wrapper_refusals(torch, ito):
    h = torch.bfloat16
    x, W, y = normal(torch, (4, 16), 1, 1.0, "bfloat16"), normal(torch, (8, 16), 2, 1.0, "bfloat16"), normal(torch, (4, 8), 3, 1.0, "bfloat16")
    t, f = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    bad = [lambda: ito.ito_fp_gated_linear_fwd(x, W, W[:7]), lambda: ito.ito_fp_gated_linear_fwd(x, W, W.half()),
           lambda: ito.ito_fp_gated_linear_fwd(x.float(), W.float(), W.float()),
           lambda: ito.ito_fp_gated_linear_fwd(x, W, W, act="tanh"), lambda: ito.ito_fp_gated_linear_fwd(x, W.cpu(), W),
           lambda: ito.ito_fp_gated_linear_fwd(x, W, W, bias_g=torch.zeros(8, device="cuda"), bias_u=torch.zeros(8, device="cuda", dtype=h)),
           lambda: ito.ito_fp_gated_linear_fwd(x[:0], W, W), lambda: ito.ito_fp_gated_linear_fwd(x, W, W.t()),
           lambda: ito.ito_fp_gated_linear_bwd(y, x, W, W, y, y[:, :7]),
           lambda: ito.ito_fp_gated_linear_bwd(y, x, W, W, y, y, need_dx=False, need_dw=False),
           lambda: ito.ito_fp_gated_linear_bwd(y, x, W, W, y, y, dw_dtype=torch.float16),
           lambda: ito.ito_linear_cross_entropy_fwd(x, W, t[:3]), lambda: ito.ito_linear_cross_entropy_fwd(x, W, t.long()),
           lambda: ito.ito_linear_cross_entropy_fwd(x, W, None),
           lambda: ito.ito_linear_cross_entropy_fwd(x.float(), W.float(), t),
           lambda: ito.ito_linear_cross_entropy_bwd(x, W, t, f, None), lambda: ito.ito_linear_cross_entropy_bwd(x, W, t, f.half(), f),
           lambda: ito.ito_linear_cross_entropy_bwd(x, W, t, f, f, need_dx=False, need_dw=False),
           lambda: ito.ito_embedding_fwd(t.long(), x), lambda: ito.ito_embedding_fwd(t[:0], x),
           lambda: ito.ito_embedding_fwd(t.view(2, 2), x), lambda: ito.ito_embedding_fwd(t, x.int()),
           lambda: ito.ito_embedding_fwd(t[::2], x), lambda: ito.ito_embedding_fwd(t, x, out_dtype=torch.int32),
           lambda: ito.ito_embedding_bwd(x, t[:3], 5), lambda: ito.ito_embedding_bwd(x, t, 0),
           lambda: ito.ito_embedding_bwd(x, t, 5, dtype=torch.float16),
           lambda: ito.ito_embedding_bwd(x, t, 5, add_to=torch.zeros((4, 16), device="cuda")),
           lambda: ito.ito_embedding_bwd(x, t, 4, dtype=h, add_to=torch.zeros((4, 16), device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ito.ItoError):
            call()
            pytest.fail("call %d was not refused" % i)
    assert ito._lib.ito_get_error() == 0


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("n", [3, 150])
def test_a_token_model_step(torch, ito, n):
    """Embedding, gated block with a residual, tied head, and back, as a training step runs them: each gradient
    of the whole against 64-bit autograd of the same 16-bit weights. Each stage rounds its results to bf16
    (2^-8 of the value at most, its sums' errors far below), so along four stages forward and six back a
    gradient's norm is off by at most about 20 of those."""
    V, D, H = 331, 136, 200
    gen = torch.Generator(device="cuda").manual_seed(n)
    ids = tokens(torch, "text", n, V, 1)
    tgt = torch.randint(0, V, (n,), generator=gen, device="cuda", dtype=torch.int32)
    E = normal(torch, (V, D), 2, 0.3, "bfloat16")
    Wg, Wu, Wd = (normal(torch, s, k, s[1] ** -0.5, "bfloat16") for k, s in ((3, (H, D)), (4, (H, D)), (5, (D, H))))
    scale = 2.0
    x = ito.ito_embedding_fwd(ids, E, scale=scale)
    h, zg, zu = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, act="silu", save_z=True)
    y = ito.ito_fp_linear_fwd(h, Wd, residual=x)
    loss, lse = ito.ito_linear_cross_entropy_fwd(y, E, tgt)
    g = torch.full((n,), 1.0 / n, device="cuda")
    dy, dE = ito.ito_linear_cross_entropy_bwd(y, E, tgt, lse, g, dw_dtype=torch.float32)
    dh, dWd, _ = ito.ito_fp_linear_bwd(dy, h, Wd, need_dbias=False)
    dx, dWg, dWu, _, _ = ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, act="silu")
    dx = dx + dy
    dE = ito.ito_embedding_bwd(dx, ids, V, scale=scale, add_to=dE)

    leaves = [w.double().requires_grad_() for w in (E, Wg, Wu, Wd)]
    e, wg, wu, wd = leaves
    X = e[ids.long().clamp(min=0)] * scale * (ids >= 0)[:, None]
    G = X @ wg.T
    Y = (G * torch.sigmoid(G) * (X @ wu.T)) @ wd.T + X
    L = Y @ e.T
    each = torch.logsumexp(L, 1) - L.gather(1, tgt.long()[:, None])[:, 0]
    each.mean().backward()
    assert float((loss.double() - each.detach()).norm() / each.detach().norm()) <= 4 * 2.0 ** -8
    for got, leaf in zip((dE, dWg, dWu, dWd), leaves):
        assert float((got.double() - leaf.grad).norm() / leaf.grad.norm()) <= 20 * 2.0 ** -8
    assert ito._lib.ito_get_error() == 0
