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
