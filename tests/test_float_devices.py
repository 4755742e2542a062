"""The float operators' wrappers refuse tensors that are not on the current device, or not all on one
(stand-ins for tensors: no GPU needed)."""
import pytest
from test_abi import _lib_path


class Stand:
    """What the wrappers look at before a launch."""

    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = shape, dtype, index
        self.device = "cuda:%d" % index

    def get_device(self):
        return self.index

    def stride(self, dim=None):
        s = [1] * len(self.shape)
        for i in range(len(s) - 2, -1, -1):
            s[i] = s[i + 1] * self.shape[i + 1]
        return tuple(s) if dim is None else s[dim]

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def is_contiguous(self):
        return True

    at = 4096

    def data_ptr(self):
        return self.at

    def detach(self):
        t = Stand(self.shape, self.dtype, self.index)
        t.at = self.at
        return t


@pytest.fixture
def ito(monkeypatch):
    torch = pytest.importorskip("torch")
    _lib_path()
    import integer_only_nn_gb300 as m
    m._float_setup()
    monkeypatch.setattr(m, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(m, "_address", lambda t: t.data_ptr(), raising=False)
    monkeypatch.setattr(m, "_float_setup", lambda: torch)

    def no_more(*a, **kw):
        raise AssertionError("the call went past its checks")

    monkeypatch.setattr(torch, "empty", no_more)
    return m


def calls(ito):
    """Each wrapper with the names of its tensors, and a call with any of them on another device."""
    import torch
    h, f, i32 = torch.bfloat16, torch.float32, torch.int32
    spec = {
        "linear_fwd": (dict(x=((4, 16), h), W=((8, 16), h), bias=((8,), h), residual=((4, 8), h)),
                       lambda t: ito.ito_fp_linear_fwd(t["x"], t["W"], bias=t["bias"], residual=t["residual"])),
        "linear_bwd": (dict(x=((4, 16), h), dy=((4, 8), h), W=((8, 16), h), z=((4, 8), h)),
                       lambda t: ito.ito_fp_linear_bwd(t["dy"], t["x"], t["W"], z=t["z"], act="gelu")),
        "layer_norm_fwd": (dict(x=((4, 16), h), gamma=((16,), f), beta=((16,), f)),
                           lambda t: ito.ito_layer_norm_fwd(t["x"], t["gamma"], t["beta"])),
        "layer_norm_bwd": (dict(x=((4, 16), h), dy=((4, 16), h), gamma=((16,), f), mean=((4,), f), rstd=((4,), f)),
                           lambda t: ito.ito_layer_norm_bwd(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"])),
        "logprobs_fwd": (dict(logits=((4, 16), h), targets=((4,), i32)),
                         lambda t: ito.ito_token_logprobs_fwd(t["logits"], t["targets"])),
        "logprobs_bwd": (dict(logits=((4, 16), h), targets=((4,), i32), lse=((4,), f), entropy=((4,), f), g_logp=((4,), f),
                              g_entropy=((4,), f), out=((4, 16), h)),
                         lambda t: ito.ito_token_logprobs_bwd(t["logits"], t["targets"], t["lse"], t["entropy"], t["g_logp"],
                                                              t["g_entropy"], out=t["out"])),
        "adamw": (dict(w=((10,), f), copy=((10,), h), m=((10,), f), v=((10,), f)),
                  lambda t: ito.AdamW([t["w"]], copies=[t["copy"]], states=[[t["m"]], [t["v"]]])),
    }
    return spec


NAMES = ["linear_fwd", "linear_bwd", "layer_norm_fwd", "layer_norm_bwd", "logprobs_fwd", "logprobs_bwd", "adamw"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_on_one_device(ito, name):
    tensors, call = calls(ito)[name]
    for other in tensors:
        for index in (1, -1):
            t = {k: Stand(shape, dtype, index if k == other else 0) for k, (shape, dtype) in tensors.items()}
            with pytest.raises(ito.ItoError) as e:
                call(t)
            assert e.value.code == ito.ITO_ERR_ARG, other


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device(ito, name):
    """All tensors on one device which is not the current one."""
    tensors, call = calls(ito)[name]
    with pytest.raises(ito.ItoError) as e:
        call({k: Stand(shape, dtype, 1) for k, (shape, dtype) in tensors.items()})
    assert e.value.code == ito.ITO_ERR_ARG and "current" in str(e.value)


def test_a_step_on_one_device(ito):
    import torch
    opt = ito.AdamW([Stand((10,), torch.float32) for _ in range(2)],
                    states=[[Stand((10,), torch.float32) for _ in range(2)] for _ in range(2)])
    with pytest.raises(ito.ItoError) as e:
        opt.step([Stand((10,), torch.bfloat16), Stand((10,), torch.bfloat16, 1)], lr=0.1)
    assert e.value.code == ito.ITO_ERR_ARG
    opt.weights[0].index = 1
    with pytest.raises(ito.ItoError) as e:
        opt.step([Stand((10,), torch.bfloat16) for _ in range(2)], lr=0.1)
    assert e.value.code == ito.ITO_ERR_ARG and opt.steps == 0


class Stream:
    cuda_stream = 77


def test_calls_on_a_stream_keep_their_tensors(ito, monkeypatch):
    """Each wrapper names all its tensors to the stream it is given, whether or not they outlive the call."""
    given = []
    monkeypatch.setattr(ito, "_on_stream", lambda call, stream, *tensors: given.append((stream, tensors)))
    import torch
    h, f, i32 = torch.bfloat16, torch.float32, torch.int32
    x, W, dy, b = Stand((4, 16), h), Stand((8, 16), h), Stand((4, 8), h), Stand((8,), h)
    v, t, r = [Stand((4,), f) for _ in range(4)], Stand((4,), i32), Stand((4, 8), h)
    s = Stream()
    calls = [(lambda: ito.ito_fp_linear_fwd(x, W, bias=b, residual=r, stream=s), [x, W, b, r]),
             (lambda: ito.ito_fp_linear_bwd(dy, x, W, z=r, act="gelu", stream=s), [dy, x, W, r]),
             (lambda: ito.ito_layer_norm_fwd(x, b, dy, stream=s), [x, b, dy]),
             (lambda: ito.ito_layer_norm_bwd(dy, x, b, v[0], v[1], stream=s), [dy, x, b, v[0], v[1]]),
             (lambda: ito.ito_token_logprobs_fwd(x, t, stream=s), [x, t]),
             (lambda: ito.ito_token_logprobs_bwd(x, t, v[0], v[1], v[2], v[3], out=W, stream=s), [x, t, *v, W])]
    w, c, m, n, g = [Stand((10,), k) for k in (f, h, f, f, h)]
    calls += [(lambda: opt.step([g], lr=0.1, stream=s), [g, w, c, m, n]), (lambda: opt.step([g], lr=0.1, stream=s), [g])]
    for i, each in enumerate([x, W, dy, b, t, r, w, c, m, n, g] + v):
        each.at = 4096 * (i + 1)
    opt = ito.AdamW([w], copies=[c], states=[[m], [n]])
    for call, tensors in calls:
        call()
        stream, got = given.pop()
        assert stream is s and not given
        assert sorted(a.at for a in got) == sorted(a.at for a in tensors)


def test_a_stream_is_recorded_for_each_tensor(ito, monkeypatch):
    import contextlib
    import types
    seen = []

    class Recorded:
        def record_stream(self, stream):
            seen.append((self, stream))

    monkeypatch.setattr(ito, "_torch", lambda: types.SimpleNamespace(
        cuda=types.SimpleNamespace(stream=lambda s: contextlib.nullcontext())))
    a, b, s = Recorded(), Recorded(), Stream()
    assert ito._on_stream(lambda: 5, s, a, None, b) == 5
    assert seen == [(a, s), (b, s)]


def test_a_step_goes_to_where_the_tensors_are(ito, monkeypatch):
    """Weights and copies that have been given other memory since the constructor: the step's table
    holds their addresses of now; what they may be is checked again. The states' memory stays."""
    import types
    import torch
    seen = []

    def step(table, n, params, stream):
        seen.append([(t.w, t.g, t.copy, t.m, t.v, t.n) for t in table])
        return 0

    monkeypatch.setattr(ito, "_lib", types.SimpleNamespace(ito_adamw_step=step))
    monkeypatch.setattr(ito, "_raw_stream_of", lambda index: 0)

    def stand(dtype, at, n=10):
        t = Stand((n,), dtype)
        t.at = at
        return t

    f, h = torch.float32, torch.bfloat16
    w, c, m, v = ([stand(k, base + 256 * i) for i in range(2)] for k, base in ((f, 4096), (h, 8192), (f, 12288), (f, 16384)))
    g = [stand(h, 65536 + 256 * i) for i in range(2)]
    opt = ito.AdamW(w, copies=c, states=[m, v])
    opt.step(g, lr=0.1)
    w[1].at, c[0].at, m[1].at, v[0].at = 20480, 24576, 28672, 32768
    opt.step(g, lr=0.1)
    assert seen[0] == [(4096, 65536, 8192, 12288, 16384, 10), (4352, 65792, 8448, 12544, 16640, 10)]
    assert seen[1] == [(4096, 65536, 24576, 12288, 16384, 10), (20480, 65792, 8448, 12544, 16640, 10)]
    w[0].at, w[0].dtype = 36864, h
    with pytest.raises(ito.ItoError):
        opt.step(g, lr=0.1)
    w[0].dtype, w[0].shape = f, (9,)
    with pytest.raises(ito.ItoError):
        opt.step(g, lr=0.1)
    w[0].shape = (10,)
    opt.step(g, lr=0.1)
    assert len(seen) == 3 and seen[2][0][0] == 36864 and opt.steps == 3


def test_a_step_without_a_gradient_is_refused(ito):
    import torch
    opt = ito.AdamW([Stand((10,), torch.float32) for _ in range(2)],
                    states=[[Stand((10,), torch.float32) for _ in range(2)] for _ in range(2)])
    g = Stand((10,), torch.bfloat16)
    for grads in ([g, None], [None, g], [None, None]):
        with pytest.raises(ito.ItoError) as e:
            opt.step(grads, lr=0.1)
        assert e.value.code == ito.ITO_ERR_ARG and opt.steps == 0


def test_alternatives_are_refused_before_their_results_are_allocated(ito):
    import torch
    x = Stand((4, 16), torch.bfloat16)
    for k, code in ((-1, ito.ITO_ERR_ARG), (33, ito.ITO_ERR_ARG), (1 << 40, ito.ITO_ERR_ARG), (17, ito.ITO_ERR_SHAPE)):
        with pytest.raises(ito.ItoError) as e:
            ito.ito_token_logprobs_fwd(x, None, k=k)
        assert e.value.code == code
