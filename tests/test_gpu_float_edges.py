"""The float operators where they were wrong once: results written over their inputs, values far
from 0, masks under large factors, rows of many waves of tiles."""
import math

import numpy as np
import pytest

from test_gpu_float_ops import TINY, U, dt, f64, normal, slope64, within, within_rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ito(torch):
    from gpu_util import import_ito
    return import_ito()


# -------------------------------------------------------------- layer norm

@pytest.mark.parametrize("rows,cols,dtype", [
    (50, 520, "bfloat16"), (40000, 24, "float32"), (1300, 768, "bfloat16"), (700, 5001, "bfloat16"),
    (650, 10000, "bfloat16"), (9, 10000, "bfloat16"), (9, 8193, "float32"), (40, 20000, "float32"), (3, 40000, "bfloat16"),
    (2, 16385, "float16")])
def test_layer_norm_backward_in_place(torch, ito, rows, cols, dtype):
    """dx written over dy, with dgamma and dbeta: the bits of the call that writes dx elsewhere."""
    x, dy = normal(torch, (rows, cols), 1, 1.5, dtype), normal(torch, (rows, cols), 2, 1.0, dtype)
    gamma = 1 + normal(torch, (cols,), 3, 0.2)
    _, mean, rstd = ito.ito_layer_norm_fwd(x, gamma)
    dx, dgamma, dbeta = ito.ito_layer_norm_bwd(dy, x, gamma, mean, rstd)
    within(dbeta, f64(dy).sum(0), (rows + 2) * U * np.abs(f64(dy)).sum(0), "dbeta")
    n = ito._lib.ito_layer_norm_bwd_workspace_size(rows, cols)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    dg, db = torch.empty_like(dgamma), torch.empty_like(dbeta)
    ty = {"float32": ito.ITO_F32, "bfloat16": ito.ITO_BF16, "float16": ito.ITO_F16}[dtype]
    assert ito._lib.ito_layer_norm_bwd(dy.data_ptr(), cols, x.data_ptr(), cols, ty, gamma.data_ptr(), ito.ITO_F32,
                                       mean.data_ptr(), rstd.data_ptr(), rows, cols, ito._aligned256(ws), n,
                                       dy.data_ptr(), cols, dg.data_ptr(), db.data_ptr(), ito._stream()) == 0
    assert torch.equal(db, dbeta)
    assert torch.equal(dg, dgamma)
    assert torch.equal(dy, dx)
