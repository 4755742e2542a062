"""The token operators at edges that their other tests leave out."""
import math

import pytest

from test_gpu_float_ops import normal

pytestmark = pytest.mark.gpu

TYPES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d", [3, 16, 40, 41, 1000])
@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_without_a_token_at_a_scale_that_is_not_finite(torch, ito, dtype, d, scale):
    """0 without a token whatever the scale; table[id] scale as elsewhere (elements of the table are not 0)."""
    table = normal(torch, (7, d), 1).abs().clamp(min=0.1).to(getattr(torch, dtype))
    ids = torch.tensor([0, -1, 6, -1, 3], dtype=torch.int32, device="cuda")
    for out in TYPES:
        y = ito.ito_embedding_fwd(ids, table, scale=scale, out_dtype=getattr(torch, out))
        assert bool((y[1] == 0).all()) and bool((y[3] == 0).all())
        there = y[[0, 2, 4]].float()
        assert bool(torch.isnan(there).all() if math.isnan(scale) else (there == scale).all())


# ------------------------------------------------------------ strided results (C callers have them)

def strided(torch, shape, offset, pad, dtype):
    """A buffer of sevens, and a view of it whose rows are apart."""
    rows, cols = shape
    ld = cols + offset + pad
    b = torch.full((rows * ld + offset + 16,), 7.0, dtype=dtype, device="cuda")
    return b, torch.as_strided(b, shape, (ld, 1), offset), ld


def only(torch, b, view, want):
    """The view holds `want`, and what lies between its rows is as it was."""
    assert torch.equal(view, want)
    view.fill_(7.0)
    assert bool((b == 7.0).all())


STRIDES = [(0, 8), (1, 0), (3, 2), (8, 16), (7, 1)]


@pytest.mark.parametrize("offset,pad", STRIDES)
@pytest.mark.parametrize("n,classes,d", [(1, 1, 5), (300, 20000, 40), (3000, 5000, 41), (9000, 300, 520), (5, 40000, 8)])
@pytest.mark.parametrize("out", ["bfloat16", "float32"])
def test_embedding_gradient_of_strided_tables(torch, ito, n, classes, d, offset, pad, out):
    """A new table gradient in rows that are apart: sums and zeros in them, nothing between."""
    dy = normal(torch, (n, d), 1, 1.0, "bfloat16")
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, classes, (n,), generator=g, device="cuda", dtype=torch.int32)
    ids[n // 2:] //= 3
    want = ito.ito_embedding_bwd(dy, ids, classes, scale=1.5, dtype=getattr(torch, out))
    b, v, ld = strided(torch, (classes, d), offset, pad, getattr(torch, out))
    m = ito._lib.ito_embedding_bwd_workspace_size(n, classes, d)
    ws = torch.full((m + 256,), 255, dtype=torch.uint8, device="cuda")
    assert ito._lib.ito_embedding_bwd(dy.data_ptr(), d, ito.ITO_BF16, ids.data_ptr(), n, classes, d, 1.5, 0,
                                      ito.ITO_BF16 if out == "bfloat16" else ito.ITO_F32, ito._aligned256(ws), m,
                                      v.data_ptr(), ld, ito._stream()) == 0
    only(torch, b, v, want)


@pytest.mark.parametrize("offset,pad", STRIDES)
@pytest.mark.parametrize("n,d", [(1, 5), (40, 16), (70, 41), (3000, 520), (100, 1001)])
@pytest.mark.parametrize("dtype,out", [("float32", "bfloat16"), ("bfloat16", "bfloat16"), ("float16", "float32"),
                                       ("bfloat16", "float16")])
@pytest.mark.parametrize("scale", [1.0, 3.5, math.inf])
def test_lookup_into_strided_rows(torch, ito, n, d, dtype, out, offset, pad, scale):
    table = normal(torch, (50, d), 1).abs().clamp(min=0.1).to(getattr(torch, dtype))
    ids = (torch.arange(n, device="cuda") * 7 % 51 - 1).to(torch.int32)
    want = ito.ito_embedding_fwd(ids, table, scale=scale, out_dtype=getattr(torch, out))
    b, v, ld = strided(torch, (n, d), offset, pad, getattr(torch, out))
    ids_of = {"float32": ito.ITO_F32, "bfloat16": ito.ITO_BF16, "float16": ito.ITO_F16}
    assert ito._lib.ito_embedding_fwd(ids.data_ptr(), n, table.data_ptr(), d, ids_of[dtype], 50, d, scale, ids_of[out],
                                      v.data_ptr(), ld, ito._stream()) == 0
    only(torch, b, v, want)


@pytest.mark.parametrize("offset,pad", STRIDES)
@pytest.mark.parametrize("B,IC,OC", [(17, 72, 40), (40, 136, 264), (300, 133, 520), (200, 2048, 96)])
@pytest.mark.parametrize("dw", ["bfloat16", "float32"])
def test_gradients_into_strided_results(torch, ito, B, IC, OC, offset, pad, dw):
    """Of more rows than stream the weights: dx and dW of both layers in rows that are apart."""
    lib, ty, dwt = ito._lib, ito.ITO_BF16 if dw == "bfloat16" else ito.ITO_F32, getattr(torch, dw)
    x, dh = normal(torch, (B, IC), 1, 1.0, "bfloat16"), normal(torch, (B, OC), 2, 1.0, "bfloat16")
    Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "bfloat16") for s in (3, 4))
    zg, zu = (normal(torch, (B, OC), s, 1.0, "bfloat16") for s in (5, 6))
    t = (torch.arange(B, device="cuda") * 5 % OC).to(torch.int32)
    _, lse = ito.ito_linear_cross_entropy_fwd(x, Wg, t)
    g = torch.ones(B, device="cuda")
    xs, gs, us = (x.data_ptr(), IC), (Wg.data_ptr(), IC), (Wu.data_ptr(), IC)
    for k, want in enumerate((ito.ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, dw_dtype=dwt)[:3],
                              ito.ito_linear_cross_entropy_bwd(x, Wg, t, lse, g, dw_dtype=dwt))):
        outs = [strided(torch, tuple(w.shape), offset, pad, w.dtype) for w in want]
        to = [v for _, view, ld in outs for v in (view.data_ptr(), ld)]
        n = (lib.ito_linear_cross_entropy_bwd_workspace_size(*xs, *gs, B, IC, OC) if k else
             lib.ito_fp_gated_linear_bwd_workspace_size(*xs, *gs, *us, B, IC, OC))
        ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
        if k:
            r = lib.ito_linear_cross_entropy_bwd(*xs, *gs, ito.ITO_BF16, t.data_ptr(), lse.data_ptr(), g.data_ptr(), None, ty,
                                                 B, IC, OC, ito._aligned256(ws), n, *to, ito._stream())
        else:
            r = lib.ito_fp_gated_linear_bwd(dh.data_ptr(), OC, zg.data_ptr(), OC, zu.data_ptr(), OC, *xs, *gs, *us,
                                            ito.ITO_BF16, ty, ito.ITO_ACT_SILU, B, IC, OC, ito._aligned256(ws), n, *to, None,
                                            None, ito._stream())
        assert r == 0
        for (b, view, _), w in zip(outs, want):
            only(torch, b, view, w)


# ------------------------------------------------------------ offsets beyond 2^31 elements

def test_gated_layer_beyond_32_bits(torch, ito):
    """Results of more than 2^31 elements each: rows at the end, against calls that have these rows alone (one K block, so
    the same sums), and their gradients."""
    B, IC, OC = 131400, 64, 16416
    x = normal(torch, (B, IC), 1, 1.0, "bfloat16")
    Wg, Wu = (normal(torch, (OC, IC), s, 0.1, "bfloat16") for s in (2, 3))
    assert B * OC > 1 << 31
    all_ = ito.ito_fp_gated_linear_fwd(x, Wg, Wu, save_z=True)
    for lo in (0, 65536, B - 600):
        part = ito.ito_fp_gated_linear_fwd(x[lo:lo + 600], Wg, Wu, save_z=True)
        assert all(torch.equal(a[lo:lo + 600], p) for a, p in zip(all_, part))
    h, zg, zu = all_
    del all_
    h.zero_()
    h[B - 600:] = normal(torch, (600, OC), 5, 1.0, "bfloat16")     # dh: only the last rows have any
    dx, dwg, dwu, dbg, dbu = ito.ito_fp_gated_linear_bwd(h, x, Wg, Wu, zg, zu, need_dbias=True, dw_dtype=torch.float32)
    part = ito.ito_fp_gated_linear_bwd(h[B - 600:], x[B - 600:], Wg, Wu, zg[B - 600:], zu[B - 600:], need_dbias=True,
                                       dw_dtype=torch.float32)
    assert bool((dx[:B - 600] == 0).all())
    # dx: 600 rows alone have their 2 x 16448 terms in slices. Each sum is off by 2 n 2^-24 of its terms' magnitudes, n = 2 OC,
    # and rounded by 2^-8 of itself.
    mags = (h[B - 600:].double() * zu[B - 600:].double()).abs() * 1.2 @ Wg.double().abs()
    mags += h[B - 600:].double().abs() * (zg[B - 600:].double().abs() + 1) @ Wu.double().abs()
    apart = 2 * 2 * 2 * OC * 2.0 ** -24 * mags
    a, b = dx[B - 600:].double(), part[0].double()
    assert bool(((a - b).abs() <= apart + 2.0 ** -8 * (a.abs() + b.abs() + apart)).all())
    # sums over the batch: the same terms among zeros, in other places of the order (2 x 600 x 2^-24 of their magnitudes)
    X, D = x[B - 600:].double().abs(), h[B - 600:].double().abs()
    G, Z = zg[B - 600:].double(), zu[B - 600:].double().abs()
    for got, want, m in ((dwg, part[1], D * Z * 1.2), (dwu, part[2], D * (G.abs() + 1))):
        assert bool(((got - want).abs() <= 2 * 2 * 600 * 2.0 ** -24 * (m.T @ X)).all())
    for got, want, m in ((dbg, part[3], D * Z * 1.2), (dbu, part[4], D * (G.abs() + 1))):
        assert bool(((got - want).abs() <= 2 * 2 * 600 * 2.0 ** -24 * m.sum(0)).all())


@pytest.mark.parametrize("rows", [2, 40])
def test_cross_entropy_beyond_32_bits(torch, ito, rows):
    """A vocabulary of more than 2^31 elements, whose rows repeat every 1009: lse from those 1009, dW's rows alike where
    no target is."""
    d, period, classes = 4096, 1009, 600000
    base = normal(torch, (period, d), 1, d ** -0.5, "bfloat16")
    W = base.repeat(-(-classes // period), 1)[:classes]
    assert W.numel() > 1 << 31
    x = normal(torch, (rows, d), 2, 1.0, "bfloat16")
    t = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    t[0], t[1] = classes - 1, 3
    loss, lse = ito.ito_linear_cross_entropy_fwd(x, W, t)
    L = x.double() @ base.double().T
    count = torch.full((period,), classes // period, device="cuda", dtype=torch.float64)
    count[:classes % period] += 1
    want = torch.log((torch.exp(L) * count).sum(1))
    # (l is off by less than 1e-4 here: 2 x 4097 x 2^-24 sum|x||w|, sum|x||w| about 41, is 0.02 at worst)
    assert bool(((lse.double() - want).abs() <= 0.02 + 1e-4).all())
    hit = torch.stack([L[0, (classes - 1) % period], L[1, 3]])
    assert bool(((loss[:2].double() - (want[:2] - hit)).abs() <= 0.04 + 1e-4).all()) and bool((loss[2:] == 0).all())
    dx, dw = ito.ito_linear_cross_entropy_bwd(x, W, t, lse, torch.ones(rows, device="cuda"))
    hits = torch.zeros((classes,), dtype=torch.bool, device="cuda")
    hits[t[:2].long()] = True
    first = dw[period:2 * period]
    for lo in (0, 100 * period, 524288 // period * period, classes // period * period - period):
        same = (dw[lo:lo + period] == first).all(1) | hits[lo:lo + period]
        assert bool(same.all())
    tail = classes // period * period
    assert bool(((dw[tail:] == first[:classes - tail]).all(1) | hits[tail:]).all())
    # the targets' own rows: dl = p - 1, rounded (2^-8), and p x
    for r in range(2):
        row = -x[r].double()
        p = torch.exp(L[:, int(t[r]) % period] - want)[:2, None]
        e = (2.0 ** -8 + 0.03 * p.sum()) * x[:2].double().abs().sum(0) + 2.0 ** -7 * row.abs()
        assert bool(((dw[int(t[r])].double() - row).abs() <= e + (p * x[:2].double().abs()).sum(0)).all())
    assert bool(torch.isfinite(dx).all())
