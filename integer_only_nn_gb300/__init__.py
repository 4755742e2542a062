"""Python binding of libito.so, the integer-only (NITI / DFP16) training library
for one GB300 GPU.

Argument marshalling only: every function here hands torch tensors' device
pointers and the current CUDA stream to the C ABI declared in include/ito.h,
under the same names. All arithmetic runs in the library's CUDA kernels. If the
shared library has not been built, importing this package raises ImportError;
there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import itertools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libito.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libito.so is not built: run `python -m integer_only_nn_gb300.build` "
                      "(or __graft_entry__.build()) on a machine with nvcc")

_lib = ctypes.CDLL(LIB_PATH)

ITO_OK, ITO_ERR_ARG, ITO_ERR_SHAPE, ITO_ERR_CUDA, ITO_ERR_TIMEOUT, ITO_ERR_EXPONENT, ITO_ERR_UNSUPPORTED = range(7)
ITO_LAYER_LINEAR, ITO_LAYER_LINEAR_RELU, ITO_LAYER_CONV3X3_RELU, ITO_LAYER_GAP = range(4)
ITO_F32, ITO_BF16, ITO_F16 = range(3)
ITO_ACT_NONE, ITO_ACT_RELU, ITO_ACT_GELU, ITO_ACT_GELU_TANH, ITO_ACT_SILU = range(5)

_P = ctypes.c_void_p
_I = ctypes.c_int
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


class NitiParams(ctypes.Structure):
    _fields_ = [("target_bits", ctypes.c_int32), ("mu_weight", ctypes.c_int32)]


class ModelOptions(ctypes.Structure):
    _fields_ = [("input_uint8", ctypes.c_int32), ("trainable_from", ctypes.c_int32),
                ("packed_masks", ctypes.c_int32), ("pingpong_grads", ctypes.c_int32),
                ("speculate_min_elems", ctypes.c_int32)]


class AptParams(ctypes.Structure):
    _fields_ = [("k_init", ctypes.c_int32), ("k_min", ctypes.c_int32), ("k_max", ctypes.c_int32),
                ("eval_every", ctypes.c_int32), ("t_min", ctypes.c_double), ("t_max", ctypes.c_double)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("in_h", ctypes.c_int32), ("in_w", ctypes.c_int32), ("stride", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("weight_decay", ctypes.c_double)]


class AdamwParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_double), ("step", ctypes.c_int64),
                ("state_bits", ctypes.c_int32), ("grad_type", ctypes.c_int32), ("copy_type", ctypes.c_int32),
                ("seed", ctypes.c_uint32)]


_SIGS = {
    "ito_version": (_I, []),
    "ito_get_error": (_I, []),
    "ito_last_error_string": (ctypes.c_char_p, []),
    "ito_selftest_wait_timeout": (_I, [_P]),
    "ito_linear_workspace_size": (_SZ, [_I, _I, _I]),
    "ito_linear_fwd": (_I, [_P, _P, _I, _I, _I, _I, NitiParams, _P, _SZ, _P, _P, _P, _P, _P]),
    "ito_linear_fwd_noalloc": (_I, [_P, _P, _I, _I, _I, _I, NitiParams, _P, _P, _P, _P, _P]),
    "ito_linear_bwd_delta": (_I, [_P, _P, _P, _I, _I, _I, NitiParams, _P, _SZ, _P, _P, _P, _P, _P]),
    "ito_linear_wgrad": (_I, [_P, _P, _I, _I, _I, _P, _SZ, _P, _P, _P]),
    "ito_niti_update": (_I, [_P, _P, _I64, _P, NitiParams, _P, _P, _P, _P]),
    "ito_top_error": (_I, [_P, _P, _I, _I, _I32, _P, _P]),
    "ito_conv2d_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "ito_conv2d_fwd": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, NitiParams, _P, _SZ, _P, _P, _P, _P, _P]),
    "ito_conv2d_bwd_delta": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, NitiParams, _P, _SZ, _P, _P, _P, _P,
                                  _P]),
    "ito_conv2d_wgrad": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P, _P, _P]),
    "ito_gap_fwd": (_I, [_P, _I, _I, _I, NitiParams, _P, _P, _P, _P, _P]),
    "ito_gap_bwd": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "ito_model_create": (_I, [ctypes.POINTER(LayerDesc), _I, _I, NitiParams, _I32, ctypes.POINTER(_P)]),
    "ito_model_create_ex": (_I, [ctypes.POINTER(LayerDesc), _I, _I, NitiParams, _I32, ctypes.POINTER(ModelOptions),
                                 ctypes.POINTER(_P)]),
    "ito_model_destroy": (_I, [_P]),
    "ito_model_set_weights": (_I, [_P, _I, _P, _I, _P]),
    "ito_model_get_weights": (_I, [_P, _I, _P, _I, _P]),
    "ito_model_tensor": (_I, [_P, ctypes.c_char_p, ctypes.POINTER(_P), ctypes.POINTER(_I), ctypes.POINTER(_I64)]),
    "ito_model_stat_index": (_I, [_P, ctypes.c_char_p]),
    "ito_model_num_stats": (_I, [_P]),
    "ito_train_step": (_I, [_P, _P, _P, _P]),
    "ito_train_step_host": (_I, [_P, _P, _P, _P, _P]),
    "ito_train_step_host_async": (_I, [_P, _P, _P, _P, _P]),
    "ito_infer": (_I, [_P, _P, _P, _P]),
    "ito_model_save": (_I, [_P, ctypes.c_char_p]),
    "ito_model_load": (_I, [_P, ctypes.c_char_p]),
    "ito_dfp16_workspace_size": (_SZ, [_I, _I, _I]),
    "ito_dfp16_linear_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P, _P, _P, _P, _P, _P]),
    "ito_dfp16_linear_bwd_delta": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P, _P, _P, _P, _P, _P]),
    "ito_dfp16_linear_wgrad": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P, _P, _P, _P, _P, _P]),
    "ito_dfp16_update": (_I, [_P, _P, _P, _I64, _I32, _I32, _P, _P, _P]),
    "ito_dfp16_from_float": (_I, [_P, _I64, _P, _P, _P, _P]),
    "ito_dfp16_to_float": (_I, [_P, _P, _I64, _P, _P]),
    "ito_dfp16_linear_fwd_f32": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P, _P, _P, _P]),
    "ito_dfp16_linear_fwd_f32_chained": (_I, [_P, _P, _P, _P, _I, _I, _I, _I32, _I32, _P, _SZ, _P, _P]),
    "ito_dfp16_model_create": (_I, [_P, _I, _I, _I32, _I32, ctypes.POINTER(_P)]),
    "ito_dfp16_model_destroy": (_I, [_P]),
    "ito_dfp16_model_set_weights": (_I, [_P, _I, _P, _I, _P]),
    "ito_dfp16_model_tensor": (_I, [_P, ctypes.c_char_p, ctypes.POINTER(_P), ctypes.POINTER(_I),
                                    ctypes.POINTER(_I64)]),
    "ito_dfp16_model_num_stats": (_I, [_P]),
    "ito_dfp16_model_stat_index": (_I, [_P, ctypes.c_char_p]),
    "ito_dfp16_model_read_stats": (_I, [_P, _P, _I]),
    "ito_dfp16_train_step": (_I, [_P, _P, _I32, _P]),
    "ito_dfp16_train_step_host_async": (_I, [_P, _P, _I32, _P, _P]),
    "ito_dfp16_model_profile": (_I, [_P, _I]),
    "ito_dfp16_model_profile_read": (_I, [_P, _P, _P, _P]),
    "ito_dfp16_model_kernels_per_step": (_I, [_P]),
    "ito_model_use_graphs": (_I, [_P, _I]),
    "ito_model_set_overlap": (_I, [_P, _I]),
    "ito_model_set_speculation": (_I, [_P, _I]),
    "ito_model_get_speculation": (_I, [_P, _P]),
    "ito_model_get_overlap": (_I, [_P, _P]),
    "ito_model_set_static_requant": (_I, [_P, _I, _P, _P, _P, _I, _P]),
    "ito_model_profile": (_I, [_P, _I]),
    "ito_model_profile_read": (_I, [_P, _P, _P, _P]),
    "ito_model_kernels_per_step": (_I, [_P]),
    "ito_dfp16_update_bits": (_I, [_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "ito_dfp_set_bits": (_I, [_P, _I64, _I32, _I32, _P]),
    "ito_bdfp16_from_float": (_I, [_P, _I64, _I64, _I32, _P, _P, _P]),
    "ito_bdfp16_to_float": (_I, [_P, _P, _I64, _I64, _I32, _P, _P]),
    "ito_bdfp16_linear_fwd_f32": (_I, [_P, _P, _P, _P, _I, _I, _I, _I32, _P, _SZ, _P, _P]),
    "ito_dfp16_model_get_precision": (_I, [_P, _I, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "ito_dfp16_model_set_precision": (_I, [_P, _I, _I32, _P]),
    "ito_dfp16_model_apt_enable": (_I, [_P, ctypes.POINTER(AptParams), _P]),
    "ito_dfp16_model_apt_epoch_end": (_I, [_P, _P, _P, _P]),
    "ito_fp_linear_fwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _I, _I, _I]),
    "ito_fp_linear_fwd": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _I, _I, _I, _I, _I, _I, _I, _P, _SZ, _P, _I64, _P,
                               _I64, _P]),
    "ito_fp_linear_bwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _I]),
    "ito_fp_linear_bwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _I, _I, _I, _P, _SZ, _P, _I64, _P,
                               _I64, _P, _P]),
    "ito_fp_gated_linear_fwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _I]),
    "ito_fp_gated_linear_fwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P, _I64, _P,
                                     _I64, _P, _I64, _P]),
    "ito_fp_gated_linear_bwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _I]),
    "ito_fp_gated_linear_bwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _I, _I, _I,
                                     _P, _SZ, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P]),
    "ito_layer_norm_fwd": (_I, [_P, _I64, _I, _P, _P, _I, _I64, _I, ctypes.c_float, _P, _I64, _P, _P, _P]),
    "ito_layer_norm_bwd_workspace_size": (_SZ, [_I64, _I]),
    "ito_layer_norm_bwd": (_I, [_P, _I64, _P, _I64, _I, _P, _I, _P, _P, _I64, _I, _P, _SZ, _P, _I64, _P, _P, _P]),
    "ito_token_logprobs_fwd": (_I, [_P, _I64, _I, _P, _I64, _I, _I, _P, _P, _P, _P, _P, _P]),
    "ito_token_logprobs_bwd": (_I, [_P, _I64, _I, _P, _P, _P, _I64, _I, _P, _P, _P, _I64, _P]),
    "ito_linear_cross_entropy_fwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _I, _I, _I]),
    "ito_linear_cross_entropy_fwd": (_I, [_P, _I64, _P, _I64, _I, _P, _I, _I, _I, _P, _SZ, _P, _P, _P]),
    "ito_linear_cross_entropy_bwd_workspace_size": (_SZ, [_P, _I64, _P, _I64, _I, _I, _I]),
    "ito_linear_cross_entropy_bwd": (_I, [_P, _I64, _P, _I64, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P, _I64, _P,
                                          _I64, _P]),
    "ito_embedding_fwd": (_I, [_P, _I64, _P, _I64, _I, _I, _I, ctypes.c_float, _I, _P, _I64, _P]),
    "ito_embedding_bwd_workspace_size": (_SZ, [_I64, _I, _I]),
    "ito_embedding_bwd": (_I, [_P, _I64, _I, _P, _I64, _I, _I, ctypes.c_float, _I, _I, _P, _SZ, _P, _I64, _P]),
    "ito_adamw_step": (_I, [_P, _I, ctypes.POINTER(AdamwParams), _P]),
    "ito_adamw_moments": (_I, [_P, _I, _I, _P, _P, _P]),
}

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class ItoError(RuntimeError):
    def __init__(self, code, text):
        super().__init__("ito status %d: %s" % (code, text))
        self.code = code


def _check(code):
    if code != ITO_OK:
        raise ItoError(code, _lib.ito_last_error_string().decode(errors="replace"))
    return code


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def params(target_bits=7, mu_weight=2) -> NitiParams:
    return NitiParams(target_bits, mu_weight)


def ito_version() -> int:
    return _lib.ito_version()


def ito_get_error() -> int:
    return _lib.ito_get_error()


def ito_selftest_wait_timeout(stream=None):
    """A kernel whose bounded wait runs out (about 2 s); ito_get_error() then reports ITO_ERR_TIMEOUT."""
    _check(_lib.ito_selftest_wait_timeout(_stream(stream)))


# ----------------------------------------------------------- single layer

def _workspace(B, IC, OC, device):
    torch = _torch()
    n = _lib.ito_linear_workspace_size(B, IC, OC)
    return torch.empty(n + 256, dtype=torch.uint8, device=device), n


def _aligned256(buf):
    off = (-buf.data_ptr()) % 256
    return ctypes.c_void_p(buf.data_ptr() + off)


def ito_linear_fwd(x, W, relu, p=None, stream=None):
    """-> (y32 int32 [B][OC], d_max uint32 as int32 [1], d_shift int32 [1], y int8 [B][OC])"""
    torch = _torch()
    B, IC = x.shape
    OC = W.shape[0]
    dev = x.device
    y32 = torch.empty((B, OC), dtype=torch.int32, device=dev)
    y = torch.empty((B, OC), dtype=torch.int8, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _workspace(B, IC, OC, dev)
    _check(_lib.ito_linear_fwd(_ptr(x), _ptr(W), B, IC, OC, int(relu), p or params(), _aligned256(ws), n,
                               _ptr(y32), _ptr(mx), _ptr(sh), _ptr(y), _stream(stream)))
    return y32, mx, sh, y


def ito_linear_fwd_noalloc(x, W, relu, p=None, stream=None, out=None):
    """ito_linear_fwd using the library's built-in scratch instead of a
    workspace (the library allocates nothing). `out` may hold preallocated
    (y32, d_max, d_shift, y) tensors; -> the same four tensors."""
    torch = _torch()
    B, IC = x.shape
    OC = W.shape[0]
    dev = x.device
    if out is None:
        out = (torch.empty((B, OC), dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev),
               torch.zeros(1, dtype=torch.int32, device=dev), torch.empty((B, OC), dtype=torch.int8, device=dev))
    y32, mx, sh, y = out
    _check(_lib.ito_linear_fwd_noalloc(_ptr(x), _ptr(W), B, IC, OC, int(relu), p or params(), _ptr(y32), _ptr(mx),
                                       _ptr(sh), _ptr(y), _stream(stream)))
    return y32, mx, sh, y


def ito_linear_bwd_delta(delta, W, a_prev, p=None, stream=None):
    """-> (d32 int32 [B][IC], d_max, d_shift, delta_prev int8 [B][IC])"""
    torch = _torch()
    B, OC = delta.shape
    IC = W.shape[1]
    dev = delta.device
    d32 = torch.empty((B, IC), dtype=torch.int32, device=dev)
    dp = torch.empty((B, IC), dtype=torch.int8, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _workspace(B, IC, OC, dev)
    _check(_lib.ito_linear_bwd_delta(_ptr(delta), _ptr(W), _ptr(a_prev), B, IC, OC, p or params(),
                                     _aligned256(ws), n, _ptr(d32), _ptr(mx), _ptr(sh), _ptr(dp), _stream(stream)))
    return d32, mx, sh, dp


def ito_linear_wgrad(delta, a_prev, stream=None):
    """-> (G int32 [OC][IC], d_max)"""
    torch = _torch()
    B, OC = delta.shape
    IC = a_prev.shape[1]
    dev = delta.device
    G = torch.empty((OC, IC), dtype=torch.int32, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _workspace(B, IC, OC, dev)
    _check(_lib.ito_linear_wgrad(_ptr(delta), _ptr(a_prev), B, IC, OC, _aligned256(ws), n, _ptr(G), _ptr(mx),
                                 _stream(stream)))
    return G, mx


def ito_niti_update(W, G, d_max, p=None, stream=None):
    """In place on W; -> (d_shift, d_wshift, d_nonzero) device int32 [1] each."""
    torch = _torch()
    dev = W.device
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.zeros(1, dtype=torch.int32, device=dev)
    nz = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(_lib.ito_niti_update(_ptr(W), _ptr(G), W.numel(), _ptr(d_max), p or params(), _ptr(sh), _ptr(ws),
                                _ptr(nz), _stream(stream)))
    return sh, ws, nz


def ito_top_error(logits, labels, target_mag=64, stream=None):
    torch = _torch()
    B, C = logits.shape
    d = torch.empty((B, C), dtype=torch.int8, device=logits.device)
    _check(_lib.ito_top_error(_ptr(logits), _ptr(labels), B, C, target_mag, _ptr(d), _stream(stream)))
    return d


def _conv_ws(B, H, W, IC, OC, stride, device):
    torch = _torch()
    n = _lib.ito_conv2d_workspace_size(B, H, W, IC, OC, stride)
    if n == 0:
        raise ItoError(ITO_ERR_SHAPE, "invalid conv sizes")
    return torch.empty(n + 256, dtype=torch.uint8, device=device), n


def _conv_out(n, stride):
    return (n - 1) // stride + 1


def ito_conv2d_fwd(x, Wt, stride, relu, p=None, stream=None):
    """x int8 [B][H][W][IC], Wt int8 [OC][3][3][IC] -> (y32 int32 [B][OH][OW][OC],
    d_max, d_shift, y int8 [B][OH][OW][OC])"""
    torch = _torch()
    B, H, W, IC = x.shape
    OC = Wt.shape[0]
    OH, OW = _conv_out(H, stride), _conv_out(W, stride)
    dev = x.device
    y32 = torch.empty((B, OH, OW, OC), dtype=torch.int32, device=dev)
    y = torch.empty((B, OH, OW, OC), dtype=torch.int8, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _conv_ws(B, H, W, IC, OC, stride, dev)
    _check(_lib.ito_conv2d_fwd(_ptr(x), _ptr(Wt), B, H, W, IC, OC, stride, int(relu), p or params(),
                               _aligned256(ws), n, _ptr(y32), _ptr(mx), _ptr(sh), _ptr(y), _stream(stream)))
    return y32, mx, sh, y


def ito_conv2d_bwd_delta(delta, Wt, a_prev, in_hw, stride, p=None, stream=None):
    """delta int8 [B][OH][OW][OC], a_prev int8 [B][H][W][IC] or None ->
    (d32 int32 [B][H][W][IC], d_max, d_shift, delta_prev int8 [B][H][W][IC])"""
    torch = _torch()
    B, OC = delta.shape[0], delta.shape[3]
    IC = Wt.shape[3]
    H, W = in_hw
    dev = delta.device
    d32 = torch.empty((B, H, W, IC), dtype=torch.int32, device=dev)
    dp = torch.empty((B, H, W, IC), dtype=torch.int8, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _conv_ws(B, H, W, IC, OC, stride, dev)
    _check(_lib.ito_conv2d_bwd_delta(_ptr(delta), _ptr(Wt), _ptr(a_prev), B, H, W, IC, OC, stride, p or params(),
                                     _aligned256(ws), n, _ptr(d32), _ptr(mx), _ptr(sh), _ptr(dp), _stream(stream)))
    return d32, mx, sh, dp


def ito_conv2d_wgrad(delta, x, stride, stream=None):
    """-> (G int32 [OC][3][3][IC], d_max)"""
    torch = _torch()
    B, H, W, IC = x.shape
    OC = delta.shape[3]
    dev = x.device
    G = torch.empty((OC, 3, 3, IC), dtype=torch.int32, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    ws, n = _conv_ws(B, H, W, IC, OC, stride, dev)
    _check(_lib.ito_conv2d_wgrad(_ptr(delta), _ptr(x), B, H, W, IC, OC, stride, _aligned256(ws), n, _ptr(G),
                                 _ptr(mx), _stream(stream)))
    return G, mx


def ito_gap_fwd(a, p=None, stream=None):
    """a int8 [B][H][W][C] -> (P32 int32 [B][C], d_max, d_shift, pa int8 [B][C])"""
    torch = _torch()
    B, H, W, C = a.shape
    dev = a.device
    P = torch.empty((B, C), dtype=torch.int32, device=dev)
    pa = torch.empty((B, C), dtype=torch.int8, device=dev)
    mx = torch.zeros(1, dtype=torch.int32, device=dev)
    sh = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(_lib.ito_gap_fwd(_ptr(a), B, H * W, C, p or params(), _ptr(P), _ptr(mx), _ptr(sh), _ptr(pa),
                            _stream(stream)))
    return P, mx, sh, pa


def ito_gap_bwd(dP, a, stream=None):
    """dP int8 [B][C], a int8 [B][H][W][C] -> delta int8 [B][H][W][C]"""
    torch = _torch()
    B, H, W, C = a.shape
    d = torch.empty(a.shape, dtype=torch.int8, device=a.device)
    _check(_lib.ito_gap_bwd(_ptr(dP), _ptr(a), B, H * W, C, _ptr(d), _stream(stream)))
    return d


# ------------------------------------------------------------------ model

_DTYPES = {1: "int8", 2: "int16", 4: "int32", 8: "int64"}


def layers_for(workload):
    """ito layer descriptors of a seeded_inputs.Workload (mlp or cnn)."""
    out = []
    if workload.kind == "mlp":
        d = workload.dims
        for i in range(len(d) - 1):
            kind = ITO_LAYER_LINEAR if i == len(d) - 2 else ITO_LAYER_LINEAR_RELU
            out.append(LayerDesc(kind, d[i], d[i + 1], 0, 0, 0))
    elif workload.kind == "cnn":
        H, W, C = workload.image
        for (ic, oc, s) in workload.convs:
            out.append(LayerDesc(ITO_LAYER_CONV3X3_RELU, ic, oc, H, W, s))
            H, W = (H + 2 - 3) // s + 1, (W + 2 - 3) // s + 1
        out.append(LayerDesc(ITO_LAYER_GAP, workload.convs[-1][1], workload.convs[-1][1], H, W, 0))
        out.append(LayerDesc(ITO_LAYER_LINEAR, workload.fc[0], workload.fc[1], 0, 0, 0))
    else:
        raise ValueError(workload.kind)
    return out


class Model:
    """An ito_model: a sequential int8 layer stack that trains with NITI."""

    def __init__(self, layers, batch, target_bits=7, mu_weight=2, target_mag=64, input_uint8=False,
                 trainable_from=0, packed_masks=False, pingpong_grads=False, speculate_min_elems=0):
        arr = (LayerDesc * len(layers))(*layers)
        h = ctypes.c_void_p()
        opt = ModelOptions(int(input_uint8), int(trainable_from), int(packed_masks), int(pingpong_grads),
                           int(speculate_min_elems))
        _check(_lib.ito_model_create_ex(arr, len(layers), batch, NitiParams(target_bits, mu_weight), target_mag,
                                        ctypes.byref(opt), ctypes.byref(h)))
        self._h = h
        self.batch = batch
        self.n_weight_layers = sum(1 for l in layers if l.kind != ITO_LAYER_GAP)

    def close(self):
        if getattr(self, "_h", None):
            _lib.ito_model_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_weights(self, layer, W, stream=None):
        """W: torch int8 tensor on the GPU, or a numpy int8 array (host)."""
        if hasattr(W, "data_ptr"):
            _check(_lib.ito_model_set_weights(self._h, layer, _ptr(W.contiguous()), 0, _stream(stream)))
        else:
            import numpy as np
            a = np.ascontiguousarray(W, dtype=np.int8)
            _check(_lib.ito_model_set_weights(self._h, layer, a.ctypes.data_as(ctypes.c_void_p), 1,
                                              _stream(stream)))

    def set_static_requant(self, layer, offset, mult, shift, stream=None):
        """numpy int32 [OC] arrays (host)."""
        import numpy as np
        arrs = [np.ascontiguousarray(a, dtype=np.int32) for a in (offset, mult, shift)]
        _check(_lib.ito_model_set_static_requant(self._h, layer, *[a.ctypes.data_as(ctypes.c_void_p) for a in arrs],
                                                 1, _stream(stream)))

    def tensor(self, name):
        """A torch view (on the GPU) of a named model tensor."""
        torch = _torch()
        ptr, eb, n = ctypes.c_void_p(), ctypes.c_int(), ctypes.c_int64()
        _check(_lib.ito_model_tensor(self._h, name.encode(), ctypes.byref(ptr), ctypes.byref(eb), ctypes.byref(n)))
        dt = getattr(torch, _DTYPES[eb.value])
        return _from_ptr(ptr.value, n.value, dt, eb.value)

    def stat_index(self, name) -> int:
        return _lib.ito_model_stat_index(self._h, name.encode())

    def num_stats(self) -> int:
        return _lib.ito_model_num_stats(self._h)

    def stats(self) -> dict:
        """All named scalars of the last step, read back to the host."""
        v = self.tensor("stats").cpu().tolist()
        out = {}
        for key in ("ymax", "ys", "dmax", "ds", "gmax", "gs", "ws", "nz", "ogmax", "ogs", "ows", "onz"):
            l = 0
            while True:
                i = self.stat_index("%s%d" % (key, l))
                if i < 0:
                    break
                val = v[i]
                out["%s%d" % (key, l)] = val & 0xFFFFFFFF if key in ("ymax", "dmax", "gmax", "nz", "ogmax", "onz") else val
                l += 1
        for key in ("pmax", "ps"):
            i = self.stat_index(key)
            out[key] = v[i] & 0xFFFFFFFF if key == "pmax" else v[i]
        return out

    def train_step(self, x, labels, stream=None):
        _check(_lib.ito_train_step(self._h, _ptr(x), _ptr(labels), _stream(stream)))

    def train_step_host(self, x_host, labels_host, stats_host=None, stream=None):
        """Host (pinned) torch tensors in, stats out; synchronises."""
        _check(_lib.ito_train_step_host(self._h, _ptr(x_host), _ptr(labels_host), _ptr(stats_host),
                                        _stream(stream)))

    def train_step_host_async(self, x_host, labels_host, stats_host=None, stream=None):
        """Host (pinned) torch tensors in, no wait: the next call's input copy overlaps this
        step; synchronise the stream before reading stats_host or reusing the buffers."""
        _check(_lib.ito_train_step_host_async(self._h, _ptr(x_host), _ptr(labels_host), _ptr(stats_host),
                                              _stream(stream)))

    def infer(self, x, logits, stream=None):
        _check(_lib.ito_infer(self._h, _ptr(x), _ptr(logits), _stream(stream)))

    def set_overlap(self, mode):
        """0: one stream; 1: backward bandwidth passes beside the contractions; 2: updates only"""
        _check(_lib.ito_model_set_overlap(self._h, int(mode)))

    def set_speculation(self, enable=True):
        """speculative requantisation in the contraction epilogues (exact; see include/ito.h)"""
        _check(_lib.ito_model_set_speculation(self._h, int(bool(enable))))

    def overlap(self) -> int:
        mode = ctypes.c_int()
        _check(_lib.ito_model_get_overlap(self._h, ctypes.byref(mode)))
        return mode.value

    def speculation(self) -> bool:
        on = ctypes.c_int()
        _check(_lib.ito_model_get_speculation(self._h, ctypes.byref(on)))
        return on.value == 1

    def use_graphs(self, enable=True):
        _check(_lib.ito_model_use_graphs(self._h, int(enable)))

    def profile(self, enable=True):
        _check(_lib.ito_model_profile(self._h, int(enable)))

    def profile_read(self):
        """{class: (ms, work, launches)} summed since the last read."""
        ms = (ctypes.c_double * 4)()
        work = (ctypes.c_double * 4)()
        n = (ctypes.c_int64 * 4)()
        _check(_lib.ito_model_profile_read(self._h, ms, work, n))
        return {name: (ms[i], work[i], n[i]) for i, name in enumerate(("gemm", "requant", "update", "other"))}

    def kernels_per_step(self) -> int:
        return _lib.ito_model_kernels_per_step(self._h)

    def save(self, path):
        _check(_lib.ito_model_save(self._h, path.encode()))

    def load(self, path):
        _check(_lib.ito_model_load(self._h, path.encode()))


# ------------------------------------------------------------------ DFP16

def _i32dev(v):
    torch = _torch()
    return torch.tensor([int(v)], dtype=torch.int32, device="cuda")


def _dfp_ws(B, IC, OC):
    torch = _torch()
    n = _lib.ito_dfp16_workspace_size(B, IC, OC)
    return torch.empty(n + 256, dtype=torch.uint8, device="cuda"), n


def _dfp_call(fn, a, ea, b, eb, B, IC, OC, p_shape, out_shape, stream):
    torch = _torch()
    p64 = torch.empty(p_shape, dtype=torch.int64, device="cuda")
    out = torch.empty(out_shape, dtype=torch.int16, device="cuda")
    mx = torch.zeros(1, dtype=torch.int64, device="cuda")
    e_out = torch.zeros(1, dtype=torch.int32, device="cuda")
    rs = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, n = _dfp_ws(B, IC, OC)
    _check(fn(_ptr(a), _ptr(ea), _ptr(b), _ptr(eb), B, IC, OC, _aligned256(ws), n, _ptr(p64), _ptr(mx), _ptr(out),
              _ptr(e_out), _ptr(rs), _stream(stream)))
    return p64, mx, out, e_out, rs


def ito_dfp16_linear_fwd(x, exp_x, W, exp_w, stream=None):
    """exp_x / exp_w: device int32 [1] tensors -> (p64, max, y, exp_y, rs)"""
    B, IC = x.shape
    OC = W.shape[0]
    return _dfp_call(_lib.ito_dfp16_linear_fwd, x, exp_x, W, exp_w, B, IC, OC, (B, OC), (B, OC), stream)


def ito_dfp16_linear_bwd_delta(delta, exp_delta, W, exp_w, stream=None):
    B, OC = delta.shape
    IC = W.shape[1]
    return _dfp_call(_lib.ito_dfp16_linear_bwd_delta, delta, exp_delta, W, exp_w, B, IC, OC, (B, IC), (B, IC),
                     stream)


def ito_dfp16_linear_wgrad(delta, exp_delta, x, exp_x, stream=None):
    B, OC = delta.shape
    IC = x.shape[1]
    return _dfp_call(_lib.ito_dfp16_linear_wgrad, delta, exp_delta, x, exp_x, B, IC, OC, (OC, IC), (OC, IC), stream)


def ito_dfp16_update(W, g, exp_g, exp_w, eta, stream=None):
    """In place on W -> (k, nonzero) device int32 [1] each."""
    torch = _torch()
    k = torch.zeros(1, dtype=torch.int32, device="cuda")
    nz = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(_lib.ito_dfp16_update(_ptr(W), _ptr(g), _ptr(exp_g), W.numel(), exp_w, eta, _ptr(k), _ptr(nz),
                                 _stream(stream)))
    return k, nz


def ito_dfp16_update_bits(W, g, exp_g, exp_w, eta, bits, stream=None):
    """ito_dfp16_update saturating to +-(2^(bits-1) - 1); in place on W -> (k, nonzero)."""
    torch = _torch()
    k = torch.zeros(1, dtype=torch.int32, device="cuda")
    nz = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(_lib.ito_dfp16_update_bits(_ptr(W), _ptr(g), _ptr(exp_g), W.numel(), exp_w, eta, bits, _ptr(k),
                                      _ptr(nz), _stream(stream)))
    return k, nz


def ito_dfp_set_bits(W, bits_old, bits_new, stream=None):
    """Precision change of an int16 mantissa tensor, in place (the exponent changes by bits_old - bits_new)."""
    _check(_lib.ito_dfp_set_bits(_ptr(W), W.numel(), bits_old, bits_new, _stream(stream)))
    return W


def ito_bdfp16_from_float(f, block, stream=None):
    """float32 [rows][cols] -> (int16 mantissas, int8 exponents [rows][ceil(cols / block)])"""
    torch = _torch()
    rows, cols = f.shape
    nb = (cols + block - 1) // block
    m = torch.empty((rows, cols), dtype=torch.int16, device=f.device)
    e = torch.empty((rows, nb), dtype=torch.int8, device=f.device)
    _check(_lib.ito_bdfp16_from_float(_ptr(f), rows, cols, block, _ptr(m), _ptr(e), _stream(stream)))
    return m, e


def ito_bdfp16_to_float(m, e, block, stream=None):
    torch = _torch()
    rows, cols = m.shape
    f = torch.empty((rows, cols), dtype=torch.float32, device=m.device)
    _check(_lib.ito_bdfp16_to_float(_ptr(m), _ptr(e), rows, cols, block, _ptr(f), _stream(stream)))
    return f


def ito_bdfp16_linear_fwd_f32(x, ex, W, ew, block, stream=None):
    """Blocked-DFP x [B][IC], W [OC][IC] (int8 exponents per block of IC) -> float32 [B][OC]"""
    torch = _torch()
    B, IC = x.shape
    OC = W.shape[0]
    y = torch.empty((B, OC), dtype=torch.float32, device=x.device)
    ws, n = _dfp_ws(B, IC, OC)
    _check(_lib.ito_bdfp16_linear_fwd_f32(_ptr(x), _ptr(ex), _ptr(W), _ptr(ew), B, IC, OC, block, _aligned256(ws), n,
                                          _ptr(y), _stream(stream)))
    return y


def ito_dfp16_from_float(f, stream=None):
    """float32 device tensor -> (int16 mantissas, device int32 [1] exponent)."""
    torch = _torch()
    mant = torch.empty(f.shape, dtype=torch.int16, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(_lib.ito_dfp16_from_float(_ptr(f), f.numel(), _ptr(bits), _ptr(mant), _ptr(e), _stream(stream)))
    return mant, e


def ito_dfp16_to_float(mant, exp, stream=None):
    torch = _torch()
    f = torch.empty(mant.shape, dtype=torch.float32, device="cuda")
    _check(_lib.ito_dfp16_to_float(_ptr(mant), _ptr(exp), mant.numel(), _ptr(f), _stream(stream)))
    return f


def ito_dfp16_linear_fwd_f32(x, exp_x, W, exp_w, stream=None):
    """-> (p64 int64 [B][OC], y float32 [B][OC])"""
    torch = _torch()
    B, IC = x.shape
    OC = W.shape[0]
    p64 = torch.empty((B, OC), dtype=torch.int64, device="cuda")
    y = torch.empty((B, OC), dtype=torch.float32, device="cuda")
    mx = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws, n = _dfp_ws(B, IC, OC)
    _check(_lib.ito_dfp16_linear_fwd_f32(_ptr(x), _ptr(exp_x), _ptr(W), _ptr(exp_w), B, IC, OC, _aligned256(ws), n,
                                         _ptr(p64), _ptr(mx), _ptr(y), _stream(stream)))
    return p64, y


def ito_dfp16_linear_fwd_f32_chained(x, exp_x, W, exp_w, chain, input_shift=1, stream=None):
    """-> y float32 [B][OC] (FP32 partial accumulation over INT32 chains of `chain` terms)"""
    torch = _torch()
    B, IC = x.shape
    OC = W.shape[0]
    y = torch.empty((B, OC), dtype=torch.float32, device="cuda")
    ws, n = _dfp_ws(B, IC, OC)
    _check(_lib.ito_dfp16_linear_fwd_f32_chained(_ptr(x), _ptr(exp_x), _ptr(W), _ptr(exp_w), B, IC, OC, int(chain),
                                                 int(input_shift), _aligned256(ws), n, _ptr(y), _stream(stream)))
    return y


class Dfp16Model:
    """An ito_dfp16_model: DFP16 Linear layers trained with integer SGD."""

    def __init__(self, dims, batch, exp_w, eta):
        arr = (ctypes.c_int32 * len(dims))(*dims)
        h = ctypes.c_void_p()
        _check(_lib.ito_dfp16_model_create(arr, len(dims) - 1, batch, exp_w, eta, ctypes.byref(h)))
        self._h = h
        self.batch = batch
        self.n_layers = len(dims) - 1

    def close(self):
        if getattr(self, "_h", None):
            _lib.ito_dfp16_model_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_weights(self, layer, W, stream=None):
        import numpy as np
        a = np.ascontiguousarray(W, dtype=np.int16)
        _check(_lib.ito_dfp16_model_set_weights(self._h, layer, a.ctypes.data_as(ctypes.c_void_p), 1,
                                                _stream(stream)))

    def tensor(self, name):
        ptr, eb, n = ctypes.c_void_p(), ctypes.c_int(), ctypes.c_int64()
        _check(_lib.ito_dfp16_model_tensor(self._h, name.encode(), ctypes.byref(ptr), ctypes.byref(eb),
                                           ctypes.byref(n)))
        return _from_ptr(ptr.value, n.value, None, eb.value)

    def stats(self) -> dict:
        n = _lib.ito_dfp16_model_num_stats(self._h)
        buf = (ctypes.c_int64 * n)()
        _check(_lib.ito_dfp16_model_read_stats(self._h, buf, n))
        out = {}
        for l in range(self.n_layers):
            for key in ("ey", "ee", "rs", "rsd", "rsg", "eg", "k", "nz", "pmax", "pdmax", "pgmax", "gabs"):
                i = _lib.ito_dfp16_model_stat_index(self._h, ("%s%d" % (key, l)).encode())
                out["%s%d" % (key, l)] = buf[i]
        return out

    def train_step(self, x, exp_x, stream=None):
        _check(_lib.ito_dfp16_train_step(self._h, _ptr(x), int(exp_x), _stream(stream)))

    def train_step_host_async(self, x_host, exp_x, stats_host=None, stream=None):
        """Host (pinned) int16 mantissas in, no wait: the next call's input copy overlaps this
        step; stats_host (int64, num_stats()) holds the step's statistics once the stream
        has passed it."""
        _check(_lib.ito_dfp16_train_step_host_async(self._h, _ptr(x_host), int(exp_x), _ptr(stats_host),
                                                    _stream(stream)))

    def num_stats(self) -> int:
        return _lib.ito_dfp16_model_num_stats(self._h)

    def profile(self, enable=True):
        _check(_lib.ito_dfp16_model_profile(self._h, int(enable)))

    def profile_read(self):
        """{class: (ms, work, launches)} summed since the last read."""
        ms = (ctypes.c_double * 4)()
        work = (ctypes.c_double * 4)()
        n = (ctypes.c_int64 * 4)()
        _check(_lib.ito_dfp16_model_profile_read(self._h, ms, work, n))
        return {name: (ms[i], work[i], n[i]) for i, name in enumerate(("gemm", "down", "update", "other"))}

    def kernels_per_step(self) -> int:
        return _lib.ito_dfp16_model_kernels_per_step(self._h)

    def precision(self, layer):
        """-> (bits, exp_w) of a layer's weights"""
        b, e = ctypes.c_int32(), ctypes.c_int32()
        _check(_lib.ito_dfp16_model_get_precision(self._h, layer, ctypes.byref(b), ctypes.byref(e)))
        return b.value, e.value

    def set_precision(self, layer, bits, stream=None):
        _check(_lib.ito_dfp16_model_set_precision(self._h, layer, bits, _stream(stream)))

    def apt_enable(self, k_init, k_min, k_max, t_min, t_max, eval_every=1, stream=None):
        p = AptParams(k_init, k_min, k_max, eval_every, float(t_min), float(t_max))
        _check(_lib.ito_dfp16_model_apt_enable(self._h, ctypes.byref(p), _stream(stream)))

    def apt_epoch_end(self, stream=None):
        """Algorithm 1 at the end of an epoch -> (mean Gavg per layer, new bits per layer)"""
        g = (ctypes.c_double * self.n_layers)()
        b = (ctypes.c_int32 * self.n_layers)()
        _check(_lib.ito_dfp16_model_apt_epoch_end(self._h, g, b, _stream(stream)))
        return list(g), list(b)


class _CudaArray:
    """Minimal __cuda_array_interface__ holder to view library-owned memory."""

    def __init__(self, ptr, n, typestr):
        self.__cuda_array_interface__ = {"shape": (n,), "typestr": typestr, "data": (ptr, False), "version": 3}


def _from_ptr(ptr, n, dtype, eb):
    torch = _torch()
    typestr = {1: "|i1", 2: "<i2", 4: "<i4", 8: "<i8"}[eb]
    return torch.as_tensor(_CudaArray(ptr, n, typestr), device="cuda")


# ---------------------------------------------------------- float operators
#
# Checks and marshalling here are on the path of calls whose kernels take 2 to 10 us, so they
# stay few: one look at each tensor, one allocation for each result. All tensors of a call are on the
# current device.

_ACTS = {"none": ITO_ACT_NONE, "relu": ITO_ACT_RELU, "gelu": ITO_ACT_GELU, "gelu_tanh": ITO_ACT_GELU_TANH,
         "silu": ITO_ACT_SILU}
_TYPE_IDS = {}          # torch dtype -> ito_type
_F32 = None             # torch.float32, once torch is there
_raw_stream_of = None   # device index -> the current stream's handle
_current_device = None  # -> the current device's index
_address = None         # Tensor.data_ptr
_INT = (1 << 31) - 1    # the largest int of the library: ctypes would pass on the low 32 bits of a larger one
_LONG = (1 << 63) - 1
_MOST_CLASSES = 1 << 30     # of an embedding


def _float_setup():
    """torch, and what this part needs of it."""
    global _F32, _raw_stream_of, _current_device, _address
    import torch
    _TYPE_IDS.update({torch.float32: ITO_F32, torch.bfloat16: ITO_BF16, torch.float16: ITO_F16})
    # (torch.cuda.current_stream() makes an object, which takes as long as a small kernel's launch)
    _raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _address = torch.Tensor.data_ptr
    _F32 = torch.float32
    return torch


def _type_id(dtype, name):
    """ito_type of a torch dtype."""
    r = _TYPE_IDS.get(dtype)
    if r is None:
        raise ItoError(ITO_ERR_ARG, "%s: type %s (float32, bfloat16 and float16 are taken)" % (name, dtype))
    return r


def _act_id(act):
    r = _ACTS.get(act, act)
    if not isinstance(r, int) or not ITO_ACT_NONE <= r <= ITO_ACT_SILU:
        raise ItoError(ITO_ERR_ARG, "unknown activation %r" % (act,))
    return r


def _device_index(t, name):
    """The device that a call runs on: that of its first tensor, which has to be the current one (the
    library launches there)."""
    index = t.get_device()
    if index < 0:
        raise ItoError(ITO_ERR_ARG, "%s: not on the GPU" % name)
    if index != _current_device():
        raise ItoError(ITO_ERR_ARG, "%s: on device %d, the current one is %d" % (name, index, _current_device()))
    return index


def _elsewhere(t, name, index):
    raise ItoError(ITO_ERR_ARG, "%s: on %s, expected cuda:%d" % (name, t.device, index))


def _matrix(t, name, rows, cols, dtype, index, most=_INT):
    """Checks a 2-D tensor on the device `index` whose rows' elements are consecutive (rows, cols,
    dtype: None for any; any rows up to `most`, columns up to an int); -> its row stride."""
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ItoError(ITO_ERR_SHAPE, "%s: shape %s, expected [%s][%s]" % (
            name, list(shape), "rows" if rows is None else rows, "columns" if cols is None else cols))
    if not shape[0] or not shape[1]:
        raise ItoError(ITO_ERR_SHAPE, "%s: no elements" % name)
    if shape[1] > _INT or (rows is None and shape[0] > most):
        raise ItoError(ITO_ERR_SHAPE, "%s: shape %s, a size that 32 bits do not hold" % (name, list(shape)))
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if dtype is not None and t.dtype is not dtype:
        raise ItoError(ITO_ERR_ARG, "%s: type %s, expected %s" % (name, t.dtype, dtype))
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ItoError(ITO_ERR_ARG, "%s: the elements of a row are not consecutive" % name)
    return s0


def _vector(t, name, n, index, dtype, other=None):
    """Checks a dense 1-D tensor on the device `index` of one of two types (None passes); -> its address."""
    if t is None:
        return None
    shape = t.shape
    if len(shape) != 1 or shape[0] != n:
        raise ItoError(ITO_ERR_SHAPE, "%s: shape %s, expected [%d]" % (name, list(shape), n))
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if t.dtype is not dtype and t.dtype is not other:
        raise ItoError(ITO_ERR_ARG, "%s: type %s" % (name, t.dtype))
    if n > 1 and t.stride(0) != 1:
        raise ItoError(ITO_ERR_ARG, "%s: not contiguous" % name)
    return t.data_ptr()


def _length(t, name):
    """The length of a 1-D tensor with elements."""
    shape = t.shape
    if len(shape) != 1 or not shape[0]:
        raise ItoError(ITO_ERR_SHAPE, "%s: shape %s, expected [n] with n >= 1" % (name, list(shape)))
    return shape[0]


def _on_stream(call, stream, *tensors):
    """Runs a call with `stream` as torch's current stream, so that what it allocates belongs to
    the stream that it launches on. The call's tensors (None passes) may be dropped after it: their
    memory is not given away before the stream has passed the call. What the stream has to wait for
    (the work that makes the tensors, the use of the results) is the caller's to order."""
    with _torch().cuda.stream(stream):
        r = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return r


class _Scratch(threading.local):
    """Workspaces kept from call to call: one for each host thread and stream, because calls
    that share one have to be in order, on the GPU and between a call's own launches."""

    KEEP = 32 << 20     # a larger one is the allocator's, call by call

    def __init__(self):
        self.kept = {}

    def get(self, n, device, stream, torch):
        """-> (the 256-byte aligned address of n bytes, their owner to hold until the launch)"""
        key = (device.index, stream)
        have = self.kept.get(key)
        if have is not None and have[1] >= n and not torch.cuda.is_current_stream_capturing():
            return have[0], None
        t = torch.empty(n + 255, dtype=torch.uint8, device=device)
        at = (t.data_ptr() + 255) & ~255
        # (a graph's replays may run beside other calls: what it uses is its own)
        if n <= self.KEEP and not torch.cuda.is_current_stream_capturing():
            self.kept[key] = (at, n, t)
        return at, t


_scratch = _Scratch()


def ito_fp_linear_fwd(x, W, bias=None, act="none", residual=None, save_z=False, out_dtype=None, stream=None):
    """y = act(x W^T + bias) + residual for bf16 or f16 x [B][IC], W [OC][IC]; -> y, or (y, z)
    with z = x W^T + bias in x's type where save_z. out_dtype (of y and residual): x's type
    or float32. bias: x's type or float32."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_fp_linear_fwd(x, W, bias, act, residual, save_z, out_dtype), stream, x, W, bias,
                          residual)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    B, IC = x.shape
    ldw = _matrix(W, "W", None, IC, dtype, index)
    OC = W.shape[0]
    ty = _type_id(dtype, "x")
    out = dtype if out_dtype is None else out_dtype
    pb = _vector(bias, "bias", OC, index, dtype, _F32)
    pr, ldr = (None, 0) if residual is None else (residual.data_ptr(), _matrix(residual, "residual", B, OC, out, index))
    y = torch.empty((B, OC), dtype=out, device=dev)
    z = torch.empty((B, OC), dtype=dtype, device=dev) if save_z else None
    s = _raw_stream_of(index)
    px, pw = x.data_ptr(), W.data_ptr()
    ws, hold = None, None
    n = _lib.ito_fp_linear_fwd_workspace_size(px, ldx, pw, ldw, B, IC, OC)
    if n:
        ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_fp_linear_fwd(px, ldx, pw, ldw, pb, pr, ldr, ty, _type_id(out, "out_dtype"),
                               ITO_F32 if bias is None else _TYPE_IDS[bias.dtype], _act_id(act), B, IC, OC, ws, n,
                               z.data_ptr() if save_z else None, OC, y.data_ptr(), OC, s)
    if r:
        _check(r)
    return (y, z) if save_z else y


def ito_fp_linear_bwd(dy, x, W, z=None, act="none", need_dx=True, need_dw=True, need_dbias=True, dw_dtype=None,
                      stream=None):
    """Gradients of ito_fp_linear_fwd -> (dx [B][IC] in x's type, dW [OC][IC] in dw_dtype (x's
    type or float32), dbias float32 [OC]); None for those not needed."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_fp_linear_bwd(dy, x, W, z, act, need_dx, need_dw, need_dbias, dw_dtype), stream, dy, x,
                          W, z)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    B, IC = x.shape
    ldw = _matrix(W, "W", None, IC, dtype, index)
    OC = W.shape[0]
    lddy = _matrix(dy, "dy", B, OC, dtype, index)
    pz, ldz = (None, 0) if z is None else (z.data_ptr(), _matrix(z, "z", B, OC, dtype, index))
    ty = _type_id(dtype, "x")
    a = _act_id(act)
    dwt = dtype if dw_dtype is None else dw_dtype
    dx = torch.empty((B, IC), dtype=dtype, device=dev) if need_dx else None
    dw = torch.empty((OC, IC), dtype=dwt, device=dev) if need_dw else None
    db = torch.empty(OC, dtype=_F32, device=dev) if need_dbias else None
    s = _raw_stream_of(index)
    pd, px, pw = dy.data_ptr(), x.data_ptr(), W.data_ptr()
    ws, hold = None, None
    n = _lib.ito_fp_linear_bwd_workspace_size(pd, lddy, px, ldx, pw, ldw, a, B, IC, OC)
    if n:
        ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_fp_linear_bwd(pd, lddy, pz, ldz, px, ldx, pw, ldw, ty, _type_id(dwt, "dw_dtype"), a, B, IC, OC, ws, n,
                               dx.data_ptr() if need_dx else None, IC, dw.data_ptr() if need_dw else None, IC,
                               db.data_ptr() if need_dbias else None, s)
    if r:
        _check(r)
    return dx, dw, db


def ito_fp_gated_linear_fwd(x, Wg, Wu, bias_g=None, bias_u=None, act="silu", save_z=False, stream=None):
    """h = act(zg) zu with zg = x Wg^T + bias_g, zu = x Wu^T + bias_u for bf16 or f16 x [B][IC], Wg and Wu
    [OC][IC]; -> h, or (h, zg, zu) where save_z, all in x's type. Biases: x's type or float32, both alike."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_fp_gated_linear_fwd(x, Wg, Wu, bias_g, bias_u, act, save_z), stream, x, Wg, Wu,
                          bias_g, bias_u)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    B, IC = x.shape
    ldg = _matrix(Wg, "Wg", None, IC, dtype, index)
    OC = Wg.shape[0]
    ldu = _matrix(Wu, "Wu", OC, IC, dtype, index)
    pbg, pbu = _vector(bias_g, "bias_g", OC, index, dtype, _F32), _vector(bias_u, "bias_u", OC, index, dtype, _F32)
    if pbg is not None and pbu is not None and bias_g.dtype is not bias_u.dtype:
        raise ItoError(ITO_ERR_ARG, "bias_g and bias_u of one type")
    b = bias_g if bias_g is not None else bias_u
    ty, a = _type_id(dtype, "x"), _act_id(act)
    px, pg, pu = x.data_ptr(), Wg.data_ptr(), Wu.data_ptr()
    h = torch.empty((B, OC), dtype=dtype, device=dev)
    zg, zu = (torch.empty_like(h), torch.empty_like(h)) if save_z else (None, None)
    s = _raw_stream_of(index)
    ws, hold = None, None
    n = _lib.ito_fp_gated_linear_fwd_workspace_size(px, ldx, pg, ldg, pu, ldu, B, IC, OC)
    if n:
        ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_fp_gated_linear_fwd(px, ldx, pg, ldg, pu, ldu, pbg, pbu, ty, ITO_F32 if b is None else _TYPE_IDS[b.dtype],
                                     a, B, IC, OC, ws, n, zg.data_ptr() if save_z else None, OC,
                                     zu.data_ptr() if save_z else None, OC, h.data_ptr(), OC, s)
    if r:
        _check(r)
    return (h, zg, zu) if save_z else h


def ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, act="silu", need_dx=True, need_dw=True, need_dbias=False,
                            dw_dtype=None, stream=None):
    """Gradients of ito_fp_gated_linear_fwd -> (dx [B][IC] in x's type, dWg and dWu [OC][IC] in dw_dtype (x's
    type or float32), dbias_g and dbias_u float32 [OC]); None for those not needed."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_fp_gated_linear_bwd(dh, x, Wg, Wu, zg, zu, act, need_dx, need_dw, need_dbias,
                                                          dw_dtype), stream, dh, x, Wg, Wu, zg, zu)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    B, IC = x.shape
    ldg = _matrix(Wg, "Wg", None, IC, dtype, index)
    OC = Wg.shape[0]
    ldu = _matrix(Wu, "Wu", OC, IC, dtype, index)
    lddh, ldzg, ldzu = (_matrix(t, name, B, OC, dtype, index) for t, name in ((dh, "dh"), (zg, "zg"), (zu, "zu")))
    ty, a = _type_id(dtype, "x"), _act_id(act)
    dwt = dtype if dw_dtype is None else dw_dtype
    out = _type_id(dwt, "dw_dtype")
    px, pg, pu = x.data_ptr(), Wg.data_ptr(), Wu.data_ptr()
    dx = torch.empty((B, IC), dtype=dtype, device=dev) if need_dx else None
    dwg = dwu = dbg = dbu = None
    if need_dw:
        dwg = torch.empty((OC, IC), dtype=dwt, device=dev)
        dwu = torch.empty_like(dwg)
    if need_dbias:
        dbg = torch.empty(OC, dtype=_F32, device=dev)
        dbu = torch.empty_like(dbg)
    s = _raw_stream_of(index)
    n = _lib.ito_fp_gated_linear_bwd_workspace_size(px, ldx, pg, ldg, pu, ldu, B, IC, OC)
    ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_fp_gated_linear_bwd(dh.data_ptr(), lddh, zg.data_ptr(), ldzg, zu.data_ptr(), ldzu, px, ldx, pg, ldg, pu,
                                     ldu, ty, out, a, B, IC, OC, ws, n, dx.data_ptr() if need_dx else None, IC,
                                     dwg.data_ptr() if need_dw else None, IC, dwu.data_ptr() if need_dw else None, IC,
                                     dbg.data_ptr() if need_dbias else None, dbu.data_ptr() if need_dbias else None, s)
    if r:
        _check(r)
    return dx, dwg, dwu, dbg, dbu


def ito_layer_norm_fwd(x, gamma=None, beta=None, eps=1e-5, stream=None):
    """x [rows][cols] of float32, bfloat16 or float16 -> (y, mean float32 [rows], rstd float32 [rows])"""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_layer_norm_fwd(x, gamma, beta, eps), stream, x, gamma, beta)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index, _LONG)
    rows, cols = x.shape
    pg, pb = _vector(gamma, "gamma", cols, index, dtype, _F32), _vector(beta, "beta", cols, index, dtype, _F32)
    if pg is not None and pb is not None and gamma.dtype is not beta.dtype:
        raise ItoError(ITO_ERR_ARG, "gamma and beta of one type")
    w = gamma if gamma is not None else beta
    ty = _type_id(dtype, "x")
    y = torch.empty((rows, cols), dtype=dtype, device=dev)
    mean = torch.empty(rows, dtype=_F32, device=dev)
    rstd = torch.empty_like(mean)
    r = _lib.ito_layer_norm_fwd(x.data_ptr(), ldx, ty, pg, pb, ITO_F32 if w is None else _TYPE_IDS[w.dtype], rows, cols,
                                eps, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(), _raw_stream_of(index))
    if r:
        _check(r)
    return y, mean, rstd


def ito_layer_norm_bwd(dy, x, gamma, mean, rstd, need_dx=True, need_dw=True, stream=None):
    """-> (dx in x's type, dgamma float32 [cols], dbeta float32 [cols]); None for those not needed."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_layer_norm_bwd(dy, x, gamma, mean, rstd, need_dx, need_dw), stream, dy, x, gamma, mean,
                          rstd)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index, _LONG)
    rows, cols = x.shape
    lddy = _matrix(dy, "dy", rows, cols, dtype, index)
    pg = _vector(gamma, "gamma", cols, index, dtype, _F32)
    pm, ps = _vector(mean, "mean", rows, index, _F32), _vector(rstd, "rstd", rows, index, _F32)
    ty = _type_id(dtype, "x")
    dx = torch.empty((rows, cols), dtype=dtype, device=dev) if need_dx else None
    s = _raw_stream_of(index)
    dg = db = ws = hold = None
    n = 0
    if need_dw:
        dg = torch.empty(cols, dtype=_F32, device=dev)
        db = torch.empty_like(dg)
        n = _lib.ito_layer_norm_bwd_workspace_size(rows, cols)
        ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_layer_norm_bwd(dy.data_ptr(), lddy, x.data_ptr(), ldx, ty, pg,
                                ITO_F32 if gamma is None else _TYPE_IDS[gamma.dtype], pm, ps, rows, cols, ws, n,
                                dx.data_ptr() if need_dx else None, cols, dg.data_ptr() if need_dw else None,
                                db.data_ptr() if need_dw else None, s)
    if r:
        _check(r)
    return dx, dg, db


def ito_token_logprobs_fwd(logits, targets=None, k=0, stream=None):
    """logits [rows][classes] (float32, bfloat16, float16), targets int32 [rows] or None ->
    (logp (None without targets), entropy, lse float32 [rows], top_ids int32 [rows][k], top_logp float32 [rows][k])"""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_token_logprobs_fwd(logits, targets, k), stream, logits, targets)
    dev, index = logits.device, _device_index(logits, "logits")
    ld = _matrix(logits, "logits", None, None, None, index, _LONG)
    rows, classes = logits.shape
    pt = _vector(targets, "targets", rows, index, torch.int32)
    if not 0 <= k <= 32:
        raise ItoError(ITO_ERR_ARG, "k must be in 0 .. 32")
    if k > classes:
        raise ItoError(ITO_ERR_SHAPE, "k above classes")
    ty = _type_id(logits.dtype, "logits")
    entropy = torch.empty(rows, dtype=_F32, device=dev)
    lse = torch.empty_like(entropy)
    logp = None if pt is None else torch.empty_like(entropy)
    top = torch.empty((rows, k), dtype=_F32, device=dev)
    ids = torch.empty((rows, k), dtype=torch.int32, device=dev)
    r = _lib.ito_token_logprobs_fwd(logits.data_ptr(), ld, ty, pt, rows, classes, k,
                                    None if pt is None else logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
                                    ids.data_ptr(), top.data_ptr(), _raw_stream_of(index))
    if r:
        _check(r)
    return logp, entropy, lse, ids, top


def ito_token_logprobs_bwd(logits, targets, lse, entropy, g_logp=None, g_entropy=None, out=None, stream=None):
    """-> dlogits in the logits' type (out: a tensor to write it to, which may be the logits)."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_token_logprobs_bwd(logits, targets, lse, entropy, g_logp, g_entropy, out), stream, logits,
                          targets, lse, entropy, g_logp, g_entropy, out)
    dtype, dev, index = logits.dtype, logits.device, _device_index(logits, "logits")
    ld = _matrix(logits, "logits", None, None, None, index, _LONG)
    rows, classes = logits.shape
    pt = _vector(targets, "targets", rows, index, torch.int32)
    pl, pe = _vector(lse, "lse", rows, index, _F32), _vector(entropy, "entropy", rows, index, _F32)
    pg, ph = _vector(g_logp, "g_logp", rows, index, _F32), _vector(g_entropy, "g_entropy", rows, index, _F32)
    ty = _type_id(dtype, "logits")
    d = torch.empty((rows, classes), dtype=dtype, device=dev) if out is None else out
    ldd = classes if out is None else _matrix(d, "out", rows, classes, dtype, index)
    r = _lib.ito_token_logprobs_bwd(logits.data_ptr(), ld, ty, pt, pl, pe, rows, classes, pg, ph, d.data_ptr(), ldd,
                                    _raw_stream_of(index))
    if r:
        _check(r)
    return d


def ito_linear_cross_entropy_fwd(x, W, targets, stream=None):
    """bf16 or f16 x [rows][d], W [classes][d], targets int32 [rows] (-1: no token) -> (loss, lse float32 [rows]):
    lse of the logits x W^T and loss = lse - the target's logit (0 without one). The logits are not stored."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_linear_cross_entropy_fwd(x, W, targets), stream, x, W, targets)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    rows, d = x.shape
    ldw = _matrix(W, "W", None, d, dtype, index)
    classes = W.shape[0]
    pt = _vector(targets, "targets", rows, index, torch.int32)
    ty = _type_id(dtype, "x")
    loss = torch.empty(rows, dtype=_F32, device=dev)
    lse = torch.empty_like(loss)
    s = _raw_stream_of(index)
    px, pw = x.data_ptr(), W.data_ptr()
    n = _lib.ito_linear_cross_entropy_fwd_workspace_size(px, ldx, pw, ldw, rows, d, classes)
    ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_linear_cross_entropy_fwd(px, ldx, pw, ldw, ty, pt, rows, d, classes, ws, n, loss.data_ptr(),
                                          lse.data_ptr(), s)
    if r:
        _check(r)
    return loss, lse


def ito_linear_cross_entropy_bwd(x, W, targets, lse, g_loss, g_lse=None, need_dx=True, need_dw=True, dw_dtype=None,
                                 stream=None):
    """Gradients of sum(g_loss loss + g_lse lse) -> (dx [rows][d] in x's type, dW [classes][d] in dw_dtype (x's type or
    float32)); None for those not needed. g_loss, g_lse: float32 [rows]. lse: of the forward pass of these rows, x and W, whose
    sums are formed again."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_linear_cross_entropy_bwd(x, W, targets, lse, g_loss, g_lse, need_dx, need_dw,
                                                               dw_dtype), stream, x, W, targets, lse, g_loss, g_lse)
    dtype, dev, index = x.dtype, x.device, _device_index(x, "x")
    ldx = _matrix(x, "x", None, None, None, index)
    rows, d = x.shape
    ldw = _matrix(W, "W", None, d, dtype, index)
    classes = W.shape[0]
    pt = _vector(targets, "targets", rows, index, torch.int32)
    pl = _vector(lse, "lse", rows, index, _F32)
    pg, pe = _vector(g_loss, "g_loss", rows, index, _F32), _vector(g_lse, "g_lse", rows, index, _F32)
    ty = _type_id(dtype, "x")
    dwt = dtype if dw_dtype is None else dw_dtype
    out = _type_id(dwt, "dw_dtype")
    dx = torch.empty((rows, d), dtype=dtype, device=dev) if need_dx else None
    dw = torch.empty((classes, d), dtype=dwt, device=dev) if need_dw else None
    s = _raw_stream_of(index)
    px, pw = x.data_ptr(), W.data_ptr()
    n = _lib.ito_linear_cross_entropy_bwd_workspace_size(px, ldx, pw, ldw, rows, d, classes)
    ws, hold = _scratch.get(n, dev, s, torch)
    r = _lib.ito_linear_cross_entropy_bwd(px, ldx, pw, ldw, ty, pt, pl, pg, pe, out, rows, d, classes, ws, n,
                                          dx.data_ptr() if need_dx else None, d, dw.data_ptr() if need_dw else None, d, s)
    if r:
        _check(r)
    return dx, dw


def ito_embedding_fwd(ids, table, scale=1.0, out_dtype=None, stream=None):
    """y [n][d] = scale table[ids] in out_dtype (the table's type by default; float32, bfloat16, float16 each);
    ids int32 [n], -1: no token (zeros)."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_embedding_fwd(ids, table, scale, out_dtype), stream, ids, table)
    dtype, dev, index = table.dtype, table.device, _device_index(table, "table")
    ldt = _matrix(table, "table", None, None, None, index)
    classes, d = table.shape
    n = _length(ids, "ids")
    pi = _vector(ids, "ids", n, index, torch.int32)
    out = dtype if out_dtype is None else out_dtype
    ty, oty = _type_id(dtype, "table"), _type_id(out, "out_dtype")
    y = torch.empty((n, d), dtype=out, device=dev)
    r = _lib.ito_embedding_fwd(pi, n, table.data_ptr(), ldt, ty, classes, d, scale, oty, y.data_ptr(), d,
                               _raw_stream_of(index))
    if r:
        _check(r)
    return y


def ito_embedding_bwd(dy, ids, classes, scale=1.0, dtype=None, add_to=None, stream=None):
    """The table's gradient [classes][d] in dtype (float32 by default, or dy's type): scale times the sums of dy's
    rows by token, zeros for tokens that do not occur. add_to: a gradient to which the sums are added instead (rows of
    absent tokens are not touched); it is returned."""
    torch = _torch() if _F32 is not None else _float_setup()
    if stream is not None:
        return _on_stream(lambda: ito_embedding_bwd(dy, ids, classes, scale, dtype, add_to), stream, dy, ids, add_to)
    dev, index = dy.device, _device_index(dy, "dy")
    n = _length(ids, "ids")
    lddy = _matrix(dy, "dy", n, None, None, index)
    d = dy.shape[1]
    pi = _vector(ids, "ids", n, index, torch.int32)
    if not 1 <= classes <= _MOST_CLASSES:
        raise ItoError(ITO_ERR_SHAPE, "classes must be in 1 .. 2^30")
    if add_to is not None:
        if dtype is not None and add_to.dtype is not dtype:
            raise ItoError(ITO_ERR_ARG, "add_to: type %s, expected %s" % (add_to.dtype, dtype))
        ldt, out = _matrix(add_to, "add_to", classes, d, None, index), add_to
    else:
        ldt, out = d, None
    oty = _type_id(add_to.dtype if out is not None else _F32 if dtype is None else dtype, "dtype")
    ty = _type_id(dy.dtype, "dy")
    if out is None:
        out = torch.empty((classes, d), dtype=_F32 if dtype is None else dtype, device=dev)
    s = _raw_stream_of(index)
    m = _lib.ito_embedding_bwd_workspace_size(n, classes, d)
    ws, hold = _scratch.get(m, dev, s, torch)
    r = _lib.ito_embedding_bwd(dy.data_ptr(), lddy, ty, pi, n, classes, d, scale, int(add_to is not None), oty, ws, m,
                               out.data_ptr(), ldt, s)
    if r:
        _check(r)
    return out


class AdamW:
    """AdamW over many weight tensors (float32, dense, updated in place), one launch a step
    for up to a few dozen of them (two with 8-bit moments and large tensors), with moments in 32 bits or
    in 8 (see include/ito.h).

    copies: bfloat16 or float16 tensors that receive the updated weights (None: none).
    weight_decay: a number, or one for each tensor. states: [m, v] lists (bits=32: float32) or
    [m, v, m_exp, v_exp] lists (bits=8: uint8 codes and int8 exponents); None starts from zero.
    step: steps taken so far. The object keeps the tensors and a table of their addresses. Weights and
    copies that have been given other memory since (w.data = .., module.to(), resize_) are found by
    their addresses, checked as in the constructor, and stepped where they are now. The states' memory is the
    object's: it stays in use whatever a state tensor is given, and must not be resized."""

    def __init__(self, weights, bits=32, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, copies=None, states=None,
                 step=0, seed=0):
        import numpy as np
        torch = _float_setup()
        if bits not in (32, 8):
            raise ItoError(ITO_ERR_ARG, "bits must be 32 or 8")
        if not weights:
            raise ItoError(ITO_ERR_SHAPE, "no weights")
        self.bits, self.betas, self.eps, self.seed, self.steps = bits, tuple(betas), eps, seed, int(step)
        self.weights = list(weights)
        sizes = [w.numel() for w in self.weights]
        blocks = [(n + 127) // 128 for n in sizes]
        dev = self.weights[0].device
        _device_index(self.weights[0], "weights[0]")
        if states is None:
            if bits == 32:
                states = [[torch.zeros(n, dtype=torch.float32, device=dev) for n in sizes] for _ in range(2)]
            else:
                states = [[torch.zeros(n, dtype=torch.uint8, device=dev) for n in sizes] for _ in range(2)] + \
                         [[torch.zeros(n, dtype=torch.int8, device=dev) for n in blocks] for _ in range(2)]
        kinds = [(torch.float32, sizes)] * 2 if bits == 32 else [(torch.uint8, sizes)] * 2 + [(torch.int8, blocks)] * 2
        if len(states) != len(kinds):
            raise ItoError(ITO_ERR_ARG, "%d state lists, expected %d" % (len(states), len(kinds)))
        self.states = [list(s) for s in states]
        self.copies = None if copies is None else list(copies)
        decays = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * len(sizes)
        if self.copies is not None and (not self.copies or self.copies[0].dtype not in (torch.bfloat16, torch.float16)):
            raise ItoError(ITO_ERR_ARG, "copies must be bfloat16 or float16")
        # the table's fields, their tensors, and what those have to be
        groups = [("w", self.weights, torch.float32, sizes, "weights")]
        if self.copies is not None:
            groups.append(("copy", self.copies, self.copies[0].dtype, sizes, "copies"))
        held = [(f, s, d, n, "states") for f, s, (d, n) in zip(("m", "v", "m_exp", "v_exp"), self.states, kinds)]
        if len(decays) != len(sizes):
            raise ItoError(ITO_ERR_SHAPE, "weight_decay: %d values, expected %d" % (len(decays), len(sizes)))
        self._copy_type = ITO_BF16 if self.copies is None else _type_id(self.copies[0].dtype, "copies")
        self._n, self._sizes, self.total, self._groups = len(sizes), sizes, sum(sizes), groups
        self._table = (AdamwTensor * self._n)()
        tab = self._fields = np.frombuffer(self._table, dtype=np.dtype(
            [(f, np.float64 if f == "weight_decay" else np.int64) for f, _ in AdamwTensor._fields_]))
        tab["n"] = sizes
        tab["weight_decay"] = decays
        index = _device_index(self.weights[0], "weights[0]")
        self._fill(held, index)
        self._held = [[t.detach() for t in ts] for ts in self.states]     # (they hold the memory)
        self._lists = [ts for _, ts, _, _, _ in groups]
        self._at, self._streams = None, {}
        self._bind()

    def _fill(self, groups, index):
        """Checks tensors and puts their addresses in the table."""
        for _, ts, dtype, lengths, name in groups:
            if len(ts) != self._n:
                raise ItoError(ITO_ERR_SHAPE, "%s: %d tensors, expected %d" % (name, len(ts), self._n))
            self._dense(ts, dtype, lengths, name, index)
        for field, ts, _, _, _ in groups:
            self._fields[field] = [t.data_ptr() for t in ts]

    def _bind(self):
        """Weights and copies where they are now, in the table. -> their device"""
        index = _device_index(self.weights[0], "weights[0]")
        # (a small model's 28 addresses take 1.7 us of its step's 12)
        at = list(map(_address, itertools.chain.from_iterable(self._lists)))
        if at != self._at:
            self._at = None
            self._fill(self._groups, index)
            self._at = at
        return index

    @staticmethod
    def _dense(ts, dtype, lengths, name, index):
        for i, (t, n) in enumerate(zip(ts, lengths)):
            if t.numel() != n:
                raise ItoError(ITO_ERR_SHAPE, "%s[%d]: %d elements, expected %d" % (name, i, t.numel(), n))
            if t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
                raise ItoError(ITO_ERR_ARG, "%s[%d]: a dense %s tensor on cuda:%d is expected" % (name, i, dtype, index))

    def step(self, grads, lr, grad_scale=1.0, stream=None):
        """One step with a gradient for each tensor (all of one type: float32, bfloat16 or float16; a
        tensor without one has to be left out of the object, or given zeros)."""
        if stream is not None:
            return _on_stream(lambda: self.step(grads, lr, grad_scale), stream, *grads, *self._new_to(stream))
        if len(grads) != self._n:
            raise ItoError(ITO_ERR_SHAPE, "%d gradients, expected %d" % (len(grads), self._n))
        index = self._bind()
        try:
            dtype = grads[0].dtype
            for g, n in zip(grads, self._sizes):
                if g.numel() != n or g.dtype is not dtype or g.get_device() != index or not g.is_contiguous():
                    self._dense(grads, dtype, self._sizes, "grads", index)     # says which and why
        except AttributeError:
            raise ItoError(ITO_ERR_ARG, "grads: %s, expected tensors" % sorted({type(g).__name__ for g in grads})) from None
        self._fields["g"] = list(map(_address, grads))
        p = AdamwParams(lr, self.betas[0], self.betas[1], self.eps, grad_scale, self.steps + 1, self.bits,
                        _type_id(dtype, "grads"), self._copy_type, self.seed & 0xFFFFFFFF)
        _check(_lib.ito_adamw_step(self._table, self._n, ctypes.byref(p), _raw_stream_of(index)))
        self.steps += 1

    def _new_to(self, stream):
        """The object's own tensors at its first call on a stream, which has to be recorded once for each
        of them and their memory; then none."""
        at = list(map(_address, itertools.chain.from_iterable(self._lists)))
        if self._streams.get(stream.cuda_stream) == at:
            return []
        self._streams[stream.cuda_stream] = at
        return [t for ts in self._lists + self._held for t in ts]

    def moments(self, dtype=None, stream=None):
        """The moments' values (m, v), the tensors' one after another: bfloat16 (exact; default)
        or float32 for 8-bit states, float32 for 32-bit ones."""
        if stream is not None:
            return _on_stream(lambda: self.moments(dtype), stream, *self._new_to(stream))
        torch = _torch()
        if self.bits == 32:
            return tuple(torch.cat([t.reshape(-1) for t in s]) for s in self._held)
        dtype = dtype or torch.bfloat16
        dev, index = self.weights[0].device, self._bind()
        m, v = (torch.empty(self.total, dtype=dtype, device=dev) for _ in range(2))
        if self.total:
            _check(_lib.ito_adamw_moments(self._table, self._n, _type_id(dtype, "dtype"), m.data_ptr(), v.data_ptr(),
                                          _raw_stream_of(index)))
        return m, v
