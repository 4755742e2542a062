"""Linear products whose CTAs, or CTA pairs, have several items each: the rings' and accumulators' phases
across tiles, every tile width, K slices in both kernels, two products in a launch with and without a gap.
The sizes' paths are asserted from the plan; results are checked in full against 64-bit products on the
GPU, with the bounds of the small sizes' tests, and between calls bit by bit."""
import pytest

from float_plan import items, plan, two_products
from test_gpu_float_ops import TINY, U, dt, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


def within_rounded(got, want, e, dtype, what):
    """got is a value within e of want (both float64), rounded to its type."""
    e = e + TINY + 2.0 ** -50 * want.abs()
    g = got.double()
    ok = (g >= (want - e).to(dtype).double()) & (g <= (want + e).to(dtype).double())
    assert bool(ok.all()), "%s: %d of %d off at %s" % (what, int((~ok).sum()), ok.numel(), (~ok).nonzero()[:3].tolist())


def silu(z):
    import torch
    return z * torch.sigmoid(z)


def silu_slope(z):
    import torch
    q = torch.sigmoid(z)
    return q * (1 + z * (1 - q))


def check_forward(torch, ito, B, IC, OC, dtype, act, bias, residual, out):
    x, W = normal(torch, (B, IC), 1, 1.0, dtype), normal(torch, (OC, IC), 2, IC ** -0.5, dtype)
    b = normal(torch, (OC,), 3, 0.5, "float32") if bias else None
    r = normal(torch, (B, OC), 4, 1.0, out) if residual else None

    def call():
        return ito.ito_fp_linear_fwd(x, W, bias=b, act=act, residual=r, save_z=True, out_dtype=dt(torch, out))

    y, z = call()
    y2, z2 = call()
    assert torch.equal(y, y2) and torch.equal(z, z2)
    zz = x.double() @ W.double().T
    sums = x.double().abs() @ W.double().abs().T
    if bias:
        zz, sums = zz + b.double(), sums + b.double().abs()
    ez = 2 * (IC + 1) * U * sums
    within_rounded(z, zz, ez, x.dtype, "z")
    yy, ey = (silu(zz), 1.13 * ez + 8 * U * (1 + zz.abs())) if act == "silu" else (zz, ez)
    if residual:
        yy = yy + r.double()
        ey = ey + U * (yy.abs() + r.double().abs())
    within_rounded(y, yy, ey, y.dtype, "y")


# sizes, and what the plan of 152 SMs has to be: pairs, columns of a tile, more than one slice, and at least
# how many items a CTA or pair
FORWARD = [((40001, 200, 50), False, 64, False, 2), ((100, 128, 40000), False, 128, False, 2),
           ((8192, 136, 2600), True, 256, False, 4), ((2048, 512, 4096), True, 224, False, 2),
           ((2051, 520, 4100), True, 192, False, 2.5), ((3000, 512, 1900), True, 160, False, 1.5),
           ((700, 16384, 130), True, 160, True, 0.5), ((256, 8192, 256), True, 128, True, 0.4)]


@pytest.mark.parametrize("i,case", list(enumerate(FORWARD)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_fwd_in_several_waves(torch, ito, i, case, dtype):
    (B, IC, OC), pair, width, sliced, rounds = case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        p = plan(B, OC, IC, False, sms)
        assert (p[0], p[1], p[2] > 1) == (pair, width, sliced)
        assert items(B, OC, p) >= rounds * (sms // 2 if pair else sms)
    check_forward(torch, ito, B, IC, OC, dtype, "silu", True, True, dtype)
    check_forward(torch, ito, B, IC, OC, dtype, "none", i % 2 == 0, i % 2 == 1, "float32")


# sizes, gap and rest of the shared launch's first round, and which product comes first (longer K)
BACKWARD = [((2048, 4096, 4096), 2, True, "dx"), ((300, 2048, 4096), 3, True, "dx"), ((600, 3000, 5000), 7, True, "dx"),
            ((4096, 2100, 300), 3, True, "dW"), ((2300, 2000, 520), 4, True, "dW"), ((2051, 520, 4100), 1, True, "dx"),
            ((8192, 1024, 4864), 0, False, "dW")]


@pytest.mark.parametrize("i,case", list(enumerate(BACKWARD)))
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_linear_bwd_in_several_waves(torch, ito, i, case, dtype):
    (B, IC, OC), gap, rest, first = case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        (dx, dw), n0, n1, pairs, r, g = two_products(B, IC, OC, sms)
        assert (g, r > 0) == (gap, rest) and n0 + n1 > pairs
        assert (dx[3] >= dw[3]) == (first == "dx")
    x, W = normal(torch, (B, IC), 1, 1.0, dtype), normal(torch, (OC, IC), 2, IC ** -0.5, dtype)
    dy, z = normal(torch, (B, OC), 3, 1.0, dtype), normal(torch, (B, OC), 4, 2.0, dtype)
    act, out = ("silu", dtype) if i % 2 else ("none", "float32")

    def call():
        return ito.ito_fp_linear_bwd(dy, x, W, z=z if act != "none" else None, act=act, dw_dtype=dt(torch, out))

    got = call()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))
    X, V, D = x.double(), W.double(), dy.double()
    dz, e0, ez = D, torch.zeros_like(D), torch.zeros_like(D)
    if act != "none":
        dz = D * silu_slope(z.double())
        e0 = D.abs() * 16 * U * (1 + z.double().abs()) + U * dz.abs()
        half, least = {"bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25)}[dtype]
        ez = e0 + (dz.abs() + e0) * (1 + half) * half + least
    a = dz.abs() + ez
    within_rounded(got[0], dz @ V, ez @ V.abs() + 2 * OC * U * (a @ V.abs()), x.dtype, "dx")
    within_rounded(got[1], dz.T @ X, ez.T @ X.abs() + 2 * B * U * (a.T @ X.abs()), dt(torch, out), "dW")
    bound = e0.sum(0) + (B + 1) * U * (dz.abs() + e0).sum(0) + TINY
    assert bool(((got[2].double() - dz.sum(0)).abs() <= bound).all())
