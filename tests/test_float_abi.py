"""The float operators' C entry points refuse bad arguments on the host (no GPU needed)."""
import ctypes

import pytest
from test_abi import _lib_path

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
BIG = 1 << 40


@pytest.fixture(scope="module")
def ito():
    _lib_path()
    import integer_only_nn_gb300 as m
    return m


def linear_fwd(ito, **kw):
    a = dict(x=P, ldx=64, W=P, ldw=64, bias=P, residual=P, ldr=64, type=ito.ITO_BF16, out=ito.ITO_BF16,
             bias_type=ito.ITO_F32, act=ito.ITO_ACT_GELU, B=4, IC=64, OC=64, ws=P, n=BIG, z=P, ldz=64, y=P, ldy=64,
             stream=None)
    a.update(kw)
    return ito._lib.ito_fp_linear_fwd(*a.values())


def linear_bwd(ito, **kw):
    a = dict(dy=P, lddy=64, z=P, ldz=64, x=P, ldx=64, W=P, ldw=64, type=ito.ITO_F16, out=ito.ITO_F32,
             act=ito.ITO_ACT_SILU, B=4, IC=64, OC=64, ws=P, n=BIG, dx=P, lddx=64, dW=P, lddw=64, db=P, stream=None)
    a.update(kw)
    return ito._lib.ito_fp_linear_bwd(*a.values())


def ln_fwd(ito, **kw):
    a = dict(x=P, ldx=64, type=ito.ITO_BF16, gamma=P, beta=P, w=ito.ITO_F32, rows=4, cols=64, eps=1e-5, y=P, ldy=64,
             mean=P, rstd=P, stream=None)
    a.update(kw)
    return ito._lib.ito_layer_norm_fwd(*a.values())


def ln_bwd(ito, **kw):
    a = dict(dy=P, lddy=64, x=P, ldx=64, type=ito.ITO_BF16, gamma=P, w=ito.ITO_F32, mean=P, rstd=P, rows=4, cols=64,
             ws=P, n=BIG, dx=P, lddx=64, dg=P, db=P, stream=None)
    a.update(kw)
    return ito._lib.ito_layer_norm_bwd(*a.values())


def lp_fwd(ito, **kw):
    a = dict(x=P, ld=64, type=ito.ITO_F32, t=P, rows=4, classes=64, k=2, logp=P, ent=P, lse=P, ids=P, top=P, stream=None)
    a.update(kw)
    return ito._lib.ito_token_logprobs_fwd(*a.values())


def lp_bwd(ito, **kw):
    a = dict(x=P, ld=64, type=ito.ITO_F32, t=P, lse=P, ent=P, rows=4, classes=64, gl=P, gh=P, d=P, ldd=64, stream=None)
    a.update(kw)
    return ito._lib.ito_token_logprobs_bwd(*a.values())


@pytest.mark.parametrize("kw", [dict(x=None), dict(W=None), dict(y=None), dict(type=0), dict(type=3), dict(out=2),
                                dict(act=5), dict(act=-1), dict(bias_type=2), dict(x=ODD), dict(y=ODD), dict(bias=ODD),
                                dict(residual=ODD), dict(z=ODD)])
def test_linear_fwd_arguments(ito, kw):
    assert linear_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(IC=-1), dict(OC=(1 << 20) + 1), dict(ldx=63), dict(ldw=63), dict(ldy=63),
                                dict(ldz=63), dict(ldr=63)])
def test_linear_fwd_shapes(ito, kw):
    assert linear_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dy=None), dict(x=None), dict(W=None), dict(z=None), dict(dx=None, dW=None, db=None),
                                dict(type=0), dict(out=1), dict(act=9), dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 64)),
                                dict(n=0), dict(dy=ODD), dict(db=ODD), dict(dW=ctypes.c_void_p(4098))])
def test_linear_bwd_arguments(ito, kw):
    assert linear_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(B=0), dict(IC=0), dict(OC=0), dict(lddy=63), dict(ldz=63), dict(ldx=63), dict(ldw=63),
                                dict(lddx=63), dict(lddw=63)])
def test_linear_bwd_shapes(ito, kw):
    assert linear_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(type=3), dict(w=2), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(x=ODD), dict(gamma=ctypes.c_void_p(4098)), dict(mean=ODD)])
def test_layer_norm_fwd_arguments(ito, kw):
    assert ln_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0), dict(rows=(1 << 40) + 1), dict(cols=(1 << 24) + 1), dict(ldx=63),
                                dict(ldy=63)])
def test_layer_norm_fwd_shapes(ito, kw):
    assert ln_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None, dg=None, db=None),
                                dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 128)), dict(n=16), dict(dy=ODD), dict(dg=ODD)])
def test_layer_norm_bwd_arguments(ito, kw):
    assert ln_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0), dict(lddy=63), dict(ldx=63), dict(lddx=63)])
def test_layer_norm_bwd_shapes(ito, kw):
    assert ln_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(x=None), dict(t=None), dict(type=-1), dict(k=-1), dict(k=33), dict(ids=None),
                                dict(top=None), dict(x=ctypes.c_void_p(4098)), dict(t=ODD), dict(ids=ODD),
                                dict(k=0, logp=None, ent=None, lse=None)])
def test_logprobs_fwd_arguments(ito, kw):
    assert lp_fwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=0), dict(classes=0), dict(classes=1, k=2), dict(ld=63), dict(classes=(1 << 30) + 1)])
def test_logprobs_fwd_shapes(ito, kw):
    assert lp_fwd(ito, **kw) == ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(x=None), dict(t=None), dict(lse=None), dict(ent=None), dict(d=None), dict(gl=None, gh=None),
                                dict(type=7), dict(d=ODD), dict(lse=ODD)])
def test_logprobs_bwd_arguments(ito, kw):
    assert lp_bwd(ito, **kw) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(classes=0), dict(ld=63), dict(ldd=63)])
def test_logprobs_bwd_shapes(ito, kw):
    assert lp_bwd(ito, **kw) == ito.ITO_ERR_SHAPE


def adamw(ito, tensor=None, n_tensors=1, **kw):
    t = dict(w=4096, g=4096, copy=4096, m=4096, v=4096, m_exp=4096, v_exp=4096, n=10, weight_decay=0.0)
    t.update(tensor or {})
    p = dict(lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0, step=1, state_bits=8, grad_type=ito.ITO_F32,
             copy_type=ito.ITO_BF16, seed=0)
    p.update(kw)
    arr = (ito.AdamwTensor * 1)(ito.AdamwTensor(*t.values()))
    return ito._lib.ito_adamw_step(arr, n_tensors, ctypes.byref(ito.AdamwParams(*p.values())), None)


@pytest.mark.parametrize("tensor", [dict(w=None), dict(g=None), dict(m=None), dict(v=None), dict(m_exp=None),
                                    dict(v_exp=None), dict(w=4098), dict(g=4098), dict(copy=4097)])
def test_adamw_tensors(ito, tensor):
    assert adamw(ito, tensor) == ito.ITO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=-1.0),
                                dict(state_bits=16), dict(grad_type=3), dict(copy_type=0)])
def test_adamw_arguments(ito, kw):
    assert adamw(ito, **kw) == ito.ITO_ERR_ARG


def test_adamw_shapes(ito):
    assert adamw(ito, n_tensors=0) == ito.ITO_ERR_SHAPE
    assert adamw(ito, dict(n=-1)) == ito.ITO_ERR_SHAPE
    assert adamw(ito, dict(n=(1 << 40) + 1)) == ito.ITO_ERR_SHAPE
    assert adamw(ito, dict(m=4098), state_bits=32) == ito.ITO_ERR_ARG
    assert ito._lib.ito_adamw_step(None, 1, None, None) == ito.ITO_ERR_ARG


def test_adamw_moments_arguments(ito):
    arr = (ito.AdamwTensor * 1)(ito.AdamwTensor(None, None, None, 4096, 4096, 4096, 4096, 10, 0.0))
    f = ito._lib.ito_adamw_moments
    assert f(None, 1, ito.ITO_F32, P, P, None) == ito.ITO_ERR_ARG
    assert f(arr, 1, ito.ITO_F32, None, None, None) == ito.ITO_ERR_ARG
    assert f(arr, 1, ito.ITO_F16, P, P, None) == ito.ITO_ERR_ARG
    assert f(arr, 0, ito.ITO_F32, P, P, None) == ito.ITO_ERR_SHAPE
    assert f(arr, 1, ito.ITO_F32, ODD, P, None) == ito.ITO_ERR_ARG


def test_structs_match_the_header(ito):
    import os
    import re
    from test_abi import ROOT
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ito.h")).read(), flags=re.S)
    for name, cls in (("ito_adamw_tensor", ito.AdamwTensor), ("ito_adamw_params", ito.AdamwParams)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        fields = [f.strip(" *\n") for d in re.findall(r"\w+\s+([^;]+);", body) for f in d.split(",")]
        assert [f.split()[-1].strip("*") for f in fields] == [f for f, _ in cls._fields_]


def test_workspace_sizes_of_bad_shapes(ito):
    assert ito._lib.ito_fp_linear_fwd_workspace_size(P, 64, P, 64, 0, 64, 64) == 0
    assert ito._lib.ito_fp_linear_bwd_workspace_size(P, 64, P, 64, P, 64, 1, 4, 64, 0) == 0
    assert ito._lib.ito_layer_norm_bwd_workspace_size(0, 4) == 0
