"""The gated layer's, the linear cross entropy's and the embedding's C entry points refuse bad arguments on the
host, their wrappers tensors on other devices and in other shapes (no GPU needed); and their index arithmetic."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
from test_abi import _lib_path
from test_float_devices import Stand, Stream
from test_float_devices import ito as stand_ito  # noqa: F401  (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "integer_only_nn_gb300", "csrc")
NVCC = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
BIG = 1 << 40


@pytest.fixture(scope="module")
def ito():
    _lib_path()
    import integer_only_nn_gb300 as m
    return m


def gated_fwd(ito, **kw):
    a = dict(x=P, ldx=64, Wg=P, ldwg=64, Wu=P, ldwu=64, bg=P, bu=P, type=ito.ITO_BF16, bias_type=ito.ITO_F32,
             act=ito.ITO_ACT_SILU, B=40, IC=64, OC=64, ws=P, n=BIG, zg=P, ldzg=64, zu=P, ldzu=64, h=P, ldh=64, stream=None)
    a.update(kw)
    return ito._lib.ito_fp_gated_linear_fwd(*a.values())


def gated_bwd(ito, **kw):
    a = dict(dh=P, lddh=64, zg=P, ldzg=64, zu=P, ldzu=64, x=P, ldx=64, Wg=P, ldwg=64, Wu=P, ldwu=64, type=ito.ITO_F16,
             out=ito.ITO_F32, act=ito.ITO_ACT_GELU, B=4, IC=64, OC=64, ws=P, n=BIG, dx=P, lddx=64, dWg=P, lddwg=64, dWu=P,
             lddwu=64, dbg=P, dbu=P, stream=None)
    a.update(kw)
    return ito._lib.ito_fp_gated_linear_bwd(*a.values())


def ce_fwd(ito, **kw):
    a = dict(x=P, ldx=64, W=P, ldw=64, type=ito.ITO_BF16, t=P, rows=4, d=64, classes=64, ws=P, n=BIG, loss=P, lse=P,
             stream=None)
    a.update(kw)
    return ito._lib.ito_linear_cross_entropy_fwd(*a.values())


def ce_bwd(ito, **kw):
    a = dict(x=P, ldx=64, W=P, ldw=64, type=ito.ITO_BF16, t=P, lse=P, g=P, gl=P, out=ito.ITO_F32, rows=4, d=64, classes=64,
             ws=P, n=BIG, dx=P, lddx=64, dW=P, lddw=64, stream=None)
    a.update(kw)
    return ito._lib.ito_linear_cross_entropy_bwd(*a.values())


def emb_fwd(ito, **kw):
    a = dict(ids=P, n=4, table=P, ldt=64, type=ito.ITO_BF16, classes=10, d=64, scale=1.0, out=ito.ITO_F32, y=P, ldy=64,
             stream=None)
    a.update(kw)
    return ito._lib.ito_embedding_fwd(*a.values())


def emb_bwd(ito, **kw):
    a = dict(dy=P, lddy=64, type=ito.ITO_BF16, ids=P, n=4, classes=10, d=64, scale=1.0, add=0, out=ito.ITO_F32, ws=P, bytes=BIG,
             dt=P, ldt=64, stream=None)
    a.update(kw)
    return ito._lib.ito_embedding_bwd(*a.values())


WS = [dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 128)), dict(n=0)]


@pytest.mark.parametrize("kw", [dict(x=None), dict(Wg=None), dict(Wu=None), dict(h=None), dict(zg=None), dict(zu=None),
                                dict(type=0), dict(type=3), dict(act=5), dict(act=-1), dict(bias_type=2), dict(x=ODD),
                                dict(Wu=ODD), dict(bg=ODD), dict(bu=ctypes.c_void_p(4098)), dict(zu=ODD), dict(h=ODD),
                                dict(ldx=60, IC=60, ws=None)])
def test_gated_fwd_arguments(ito, kw):
    assert gated_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(IC=-1), dict(OC=(1 << 20) + 1), dict(ldx=63), dict(ldwg=63), dict(ldwu=63),
                                dict(ldzg=63), dict(ldzu=63), dict(ldh=63)])
def test_gated_fwd_shapes(ito, kw):
    assert gated_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dh=None), dict(zg=None), dict(zu=None), dict(x=None), dict(Wg=None), dict(Wu=None),
                                dict(dWg=None), dict(dWu=None), dict(dx=None, dWg=None, dWu=None, dbg=None, dbu=None),
                                dict(type=0), dict(out=1), dict(act=9), dict(dh=ODD), dict(dbg=ODD),
                                dict(dWu=ctypes.c_void_p(4098))] + WS)
def test_gated_bwd_arguments(ito, kw):
    assert gated_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(IC=0), dict(OC=0), dict(lddh=63), dict(ldzg=63), dict(ldzu=63), dict(ldx=63),
                                dict(ldwg=63), dict(ldwu=63), dict(lddx=63), dict(lddwg=63), dict(lddwu=63)])
def test_gated_bwd_shapes(ito, kw):
    assert gated_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(x=None), dict(W=None), dict(t=None), dict(loss=None, lse=None), dict(type=0), dict(type=5),
                                dict(x=ODD), dict(W=ODD), dict(t=ODD), dict(loss=ODD), dict(lse=ODD)] + WS)
def test_cross_entropy_fwd_arguments(ito, kw):
    assert ce_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=0), dict(d=0), dict(classes=0), dict(classes=(1 << 20) + 1), dict(ldx=63),
                                dict(ldw=63)])
def test_cross_entropy_fwd_shapes(ito, kw):
    assert ce_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(x=None), dict(W=None), dict(t=None), dict(lse=None), dict(g=None), dict(dx=None, dW=None),
                                dict(type=0), dict(out=2), dict(lse=ODD), dict(g=ODD), dict(gl=ODD), dict(dx=ODD),
                                dict(dW=ctypes.c_void_p(4098))] + WS)
def test_cross_entropy_bwd_arguments(ito, kw):
    assert ce_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=0), dict(d=-4), dict(classes=0), dict(ldx=63), dict(ldw=63), dict(lddx=63),
                                dict(lddw=63)])
def test_cross_entropy_bwd_shapes(ito, kw):
    assert ce_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(ids=None), dict(table=None), dict(y=None), dict(type=3), dict(out=-1), dict(ids=ODD),
                                dict(table=ODD), dict(y=ctypes.c_void_p(4098))])
def test_embedding_fwd_arguments(ito, kw):
    assert emb_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(n=0), dict(n=(1 << 30) + 1), dict(classes=0), dict(d=0), dict(d=(1 << 24) + 1),
                                dict(ldt=63), dict(ldy=63)])
def test_embedding_fwd_shapes(ito, kw):
    assert emb_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dy=None), dict(ids=None), dict(dt=None), dict(type=3), dict(out=2), dict(ids=ODD),
                                dict(dy=ODD), dict(dt=ODD), dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 64)), dict(bytes=16)])
def test_embedding_bwd_arguments(ito, kw):
    assert emb_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(n=0), dict(classes=-1), dict(d=0), dict(lddy=63), dict(ldt=63)])
def test_embedding_bwd_shapes(ito, kw):
    assert emb_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


def test_workspaces_of_invalid_sizes_are_none(ito):
    lib = ito._lib
    assert lib.ito_fp_gated_linear_fwd_workspace_size(P, 64, P, 64, P, 64, 0, 64, 64) == 0
    assert lib.ito_fp_gated_linear_bwd_workspace_size(P, 64, P, 64, P, 64, 4, 64, 1 << 21) == 0
    assert lib.ito_linear_cross_entropy_fwd_workspace_size(P, 64, P, 64, 4, 0, 64) == 0
    assert lib.ito_linear_cross_entropy_bwd_workspace_size(P, 64, P, 64, 4, 64, -1) == 0
    assert lib.ito_embedding_bwd_workspace_size(0, 10, 64) == 0
    # a piece of dl takes 256 MB at most (and 256 classes at least), whatever the vocabulary
    for rows in (1, 64, 8192, 1 << 20):
        small, large = (lib.ito_linear_cross_entropy_bwd_workspace_size(P, 64, P, 64, rows, 64, v) for v in (1000, 1 << 20))
        assert large < small + (600 << 20) + rows * 64 * 4 + (64 << 20)


# --------------------------------------------------------------- wrappers

def calls(m):
    import torch
    h, f, i32 = torch.bfloat16, torch.float32, torch.int32
    return {
        "gated_fwd": (dict(x=((40, 16), h), Wg=((8, 16), h), Wu=((8, 16), h), bg=((8,), f), bu=((8,), f)),
                      lambda t, **k: m.ito_fp_gated_linear_fwd(t["x"], t["Wg"], t["Wu"], t["bg"], t["bu"], **k)),
        "gated_bwd": (dict(x=((40, 16), h), dh=((40, 8), h), Wg=((8, 16), h), Wu=((8, 16), h), zg=((40, 8), h), zu=((40, 8), h)),
                      lambda t, **k: m.ito_fp_gated_linear_bwd(t["dh"], t["x"], t["Wg"], t["Wu"], t["zg"], t["zu"], **k)),
        "ce_fwd": (dict(x=((4, 16), h), W=((8, 16), h), t=((4,), i32)),
                   lambda t, **k: m.ito_linear_cross_entropy_fwd(t["x"], t["W"], t["t"], **k)),
        "ce_bwd": (dict(x=((4, 16), h), W=((8, 16), h), t=((4,), i32), lse=((4,), f), g=((4,), f), g_lse=((4,), f)),
                   lambda t, **k: m.ito_linear_cross_entropy_bwd(t["x"], t["W"], t["t"], t["lse"], t["g"], t["g_lse"], **k)),
        "emb_fwd": (dict(table=((9, 16), h), ids=((4,), i32)), lambda t, **k: m.ito_embedding_fwd(t["ids"], t["table"], **k)),
        "emb_bwd": (dict(dy=((4, 16), h), ids=((4,), i32), add=((9, 16), f)),
                    lambda t, **k: m.ito_embedding_bwd(t["dy"], t["ids"], 9, add_to=t["add"], **k)),
    }


NAMES = ["gated_fwd", "gated_bwd", "ce_fwd", "ce_bwd", "emb_fwd", "emb_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_on_one_device(stand_ito, name):  # noqa: F811
    tensors, call = calls(stand_ito)[name]
    for other in tensors:
        for index in (1, -1):
            t = {k: Stand(shape, dtype, index if k == other else 0) for k, (shape, dtype) in tensors.items()}
            with pytest.raises(stand_ito.ItoError) as e:
                call(t)
            assert e.value.code == stand_ito.ITO_ERR_ARG, other


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device(stand_ito, name):  # noqa: F811
    tensors, call = calls(stand_ito)[name]
    with pytest.raises(stand_ito.ItoError) as e:
        call({k: Stand(shape, dtype, 1) for k, (shape, dtype) in tensors.items()})
    assert e.value.code == stand_ito.ITO_ERR_ARG and "current" in str(e.value)


@pytest.mark.parametrize("name", NAMES)
def test_shapes_and_types_are_refused_before_anything_is_allocated(stand_ito, name):  # noqa: F811
    """Each tensor in turn with one element, row or dimension more, or in a type that it cannot have."""
    import torch
    tensors, call = calls(stand_ito)[name]
    for other, (shape, dtype) in tensors.items():
        bad = [Stand(shape + (2,), dtype), Stand(shape, torch.int64)]
        if name != "emb_fwd":            # (a lookup's two tensors share no size)
            bad.append(Stand(shape[:-1] + (shape[-1] + 1,), dtype))
        for b in bad:
            t = {k: Stand(s, d) for k, (s, d) in tensors.items()}
            t[other] = b
            with pytest.raises(stand_ito.ItoError):
                call(t)


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_a_stream_keep_their_tensors(stand_ito, monkeypatch, name):  # noqa: F811
    given = []
    monkeypatch.setattr(stand_ito, "_on_stream", lambda call, stream, *tensors: given.append((stream, tensors)))
    tensors, call = calls(stand_ito)[name]
    t = {k: Stand(shape, dtype) for k, (shape, dtype) in tensors.items()}
    for i, each in enumerate(t.values()):
        each.at = 4096 * (i + 1)
    s = Stream()
    call(t, stream=s)
    (stream, got), = given
    assert stream is s and sorted(a.at for a in got) == sorted(a.at for a in t.values())


# -------------------------------------------------------- index arithmetic

PLAY = r"""
#include <cstdio>
#include <cstdlib>
#include "ito_fp.h"

// Reads lines: "div d n" -> n / d; "span rows cols ld first last" -> whether the rows' words are in the span
int main()
{
    char what[8];
    long long a, b, c, d, e;
    while (scanf("%7s %lld %lld", what, &a, &b) == 3) {
        if (what[0] == 'd') {
            printf("%u\n", ito::Divider((uint32_t)a)((uint32_t)b));
        } else {
            if (scanf("%lld %lld %lld", &c, &d, &e) != 3) return 1;
            printf("%d\n", (int)ito::fp_copy_inner(d, e, (int)a, (int)b, c));
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def play(tmp_path_factory):
    if not os.path.exists(NVCC):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("play")
    src, exe = d / "play.cu", d / "play"
    src.write_text(PLAY)
    subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr", "-I" + CSRC,
                    "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True, capture_output=True)
    return lambda lines: subprocess.run([str(exe)], input="\n".join(lines), text=True, capture_output=True,
                                        check=True).stdout.split()


def test_division_by_multiplication(play):
    rng = random.Random(1)
    pairs = []
    for _ in range(20000):
        d = rng.choice((rng.randint(1, 40), rng.randint(1, 1 << 18), 1 << rng.randint(0, 18), (1 << rng.randint(1, 18)) - 1))
        q = rng.randint(0, ((1 << 31) - 1) // d)
        pairs += [(d, min((1 << 31) - 1, d * q + r)) for r in (0, d - 1)] + [(d, rng.randint(0, (1 << 31) - 1))]
    assert play(["div %d %d" % p for p in pairs]) == [str(n // d) for d, n in pairs]


def test_copied_words_stay_in_the_tensor(play):
    """Where rows count as inner, no word of their eights reaches before the tensor's first element or behind
    its last, at either of a word's halves."""
    rng = random.Random(2)
    cases = []
    for _ in range(4000):
        rows, cols = rng.randint(1, 30), rng.randint(1, 40)
        ld = cols + rng.choice((0, 0, 1, 3, 8))
        first = rng.randint(0, rows - 1)
        cases.append((rows, cols, ld, first, rng.randint(first, rows - 1)))
    got = play(["span %d %d %d %d %d" % c for c in cases])
    inner = 0
    for (rows, cols, ld, first, last), g in zip(cases, got):
        low = first * ld - 1                                  # a word's other half before the first eight
        high = last * ld + (cols - 1) // 8 * 8 + 8            # and behind the last
        fits = low >= 0 and high <= (rows - 1) * ld + cols - 1
        assert g == "01"[fits] or (g == "0" and not fits), (rows, cols, ld, first, last)
        inner += g == "1"
    assert inner > 500
