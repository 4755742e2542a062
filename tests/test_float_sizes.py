"""Sizes that a 32-bit argument cannot hold are refused, not taken for their low 32 bits (stand-ins for tensors: no GPU
needed)."""
import pytest

from test_float_devices import Stand
from test_float_devices import ito as stand_ito  # noqa: F401  (a fixture)

SIZES = [1 << 31, (1 << 31) + 5, (1 << 32) + 5, (1 << 33) + 1]


def calls(m, rows, cols):
    """Every wrapper of a float operator whose rows or columns are an int of the library, on tensors of that size."""
    import torch
    h, f, i32 = torch.bfloat16, torch.float32, torch.int32

    def t(shape, dtype=h):
        return Stand(shape, dtype)

    x, W, y, yw = t((rows, cols)), t((8, cols)), t((rows, 8)), t((8, cols))
    v, w = t((rows,), f), t((rows,), i32)
    wide, few = t((rows, cols)), t((3, cols))           # a weight or table with as many rows, and a few rows of x
    out = t((3, rows))
    return {
        "linear_fwd": lambda: m.ito_fp_linear_fwd(x, W), "linear_fwd W": lambda: m.ito_fp_linear_fwd(few, wide),
        "linear_bwd": lambda: m.ito_fp_linear_bwd(y, x, W), "linear_bwd W": lambda: m.ito_fp_linear_bwd(out, few, wide),
        "gated_fwd": lambda: m.ito_fp_gated_linear_fwd(x, W, W),
        "gated_fwd W": lambda: m.ito_fp_gated_linear_fwd(few, wide, wide),
        "gated_bwd": lambda: m.ito_fp_gated_linear_bwd(y, x, W, W, y, y),
        "gated_bwd W": lambda: m.ito_fp_gated_linear_bwd(out, few, wide, wide, out, out),
        "ce_fwd": lambda: m.ito_linear_cross_entropy_fwd(x, W, w),
        "ce_fwd W": lambda: m.ito_linear_cross_entropy_fwd(few, wide, t((3,), i32)),
        "ce_bwd": lambda: m.ito_linear_cross_entropy_bwd(x, W, w, v, v),
        "ce_bwd W": lambda: m.ito_linear_cross_entropy_bwd(few, wide, t((3,), i32), t((3,), f), t((3,), f)),
        "embedding_fwd": lambda: m.ito_embedding_fwd(t((3,), i32), wide),
        "embedding_bwd": lambda: m.ito_embedding_bwd(few, t((3,), i32), rows),
        "embedding_bwd add": lambda: m.ito_embedding_bwd(few, t((3,), i32), rows, add_to=wide),
    }


def by_columns(m, cols):
    """And those of which the columns alone are."""
    import torch
    h, f, i32 = torch.bfloat16, torch.float32, torch.int32
    x, v, w = Stand((3, cols), h), Stand((3,), f), Stand((3,), i32)
    return {
        "layer_norm_fwd": lambda: m.ito_layer_norm_fwd(x), "layer_norm_bwd": lambda: m.ito_layer_norm_bwd(x, x, None, v, v),
        "logprobs_fwd": lambda: m.ito_token_logprobs_fwd(x, w),
        "logprobs_bwd": lambda: m.ito_token_logprobs_bwd(x, w, v, v, v),
        "embedding_fwd": lambda: m.ito_embedding_fwd(w, x), "embedding_bwd": lambda: m.ito_embedding_bwd(x, w, 9),
    }


ROWS = ["linear_fwd", "linear_fwd W", "linear_bwd", "linear_bwd W", "gated_fwd", "gated_fwd W", "gated_bwd", "gated_bwd W",
        "ce_fwd", "ce_fwd W", "ce_bwd", "ce_bwd W", "embedding_fwd", "embedding_bwd", "embedding_bwd add"]
COLUMNS = ["layer_norm_fwd", "layer_norm_bwd", "logprobs_fwd", "logprobs_bwd", "embedding_fwd", "embedding_bwd"]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("name", ROWS)
def test_rows_beyond_32_bits(stand_ito, name, size):  # noqa: F811
    with pytest.raises(stand_ito.ItoError) as e:
        calls(stand_ito, size, 16)[name]()
    assert e.value.code == stand_ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("name", [n for n in ROWS if not n.startswith("embedding_bwd")])
def test_columns_beyond_32_bits(stand_ito, name, size):  # noqa: F811
    with pytest.raises(stand_ito.ItoError) as e:
        calls(stand_ito, 5, size)[name]()
    assert e.value.code == stand_ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("name", COLUMNS)
def test_rows_of_more_columns_than_32_bits_count(stand_ito, name, size):  # noqa: F811
    with pytest.raises(stand_ito.ItoError) as e:
        by_columns(stand_ito, size)[name]()
    assert e.value.code == stand_ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("classes", [(1 << 30) + 1, 1 << 31, (1 << 32) + 9, -(1 << 32) + 9])
def test_more_classes_than_the_library_takes_are_refused_before_anything_is_allocated(stand_ito, classes):  # noqa: F811
    import torch
    with pytest.raises(stand_ito.ItoError) as e:
        stand_ito.ito_embedding_bwd(Stand((3, 16), torch.bfloat16), Stand((3,), torch.int32), classes)
    assert e.value.code == stand_ito.ITO_ERR_SHAPE


@pytest.mark.parametrize("act", [1 << 32, (1 << 32) + 4, -(1 << 32)])
def test_activations_beyond_32_bits(stand_ito, act):  # noqa: F811
    import torch
    x, W = Stand((3, 16), torch.bfloat16), Stand((8, 16), torch.bfloat16)
    for call in (lambda: stand_ito.ito_fp_linear_bwd(Stand((3, 8), torch.bfloat16), x, W, act=act),
                 lambda: stand_ito.ito_fp_gated_linear_fwd(x, W, W, act=act)):
        with pytest.raises(stand_ito.ItoError) as e:
            call()
        assert e.value.code == stand_ito.ITO_ERR_ARG


def test_operators_that_count_rows_in_64_bits_still_take_them(stand_ito):  # noqa: F811
    import torch
    x = Stand((1 << 33, 16), torch.bfloat16)
    v, t = Stand((1 << 33,), torch.float32), Stand((1 << 33,), torch.int32)
    for call in (lambda: stand_ito.ito_layer_norm_fwd(x), lambda: stand_ito.ito_layer_norm_bwd(x, x, None, v, v),
                 lambda: stand_ito.ito_token_logprobs_fwd(x, t), lambda: stand_ito.ito_token_logprobs_bwd(x, t, v, v, v)):
        with pytest.raises(AssertionError, match="past its checks"):
            call()
