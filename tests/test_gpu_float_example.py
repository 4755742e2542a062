"""The float residual MLP on a DFP16 layer: its gradients against the same model in 64 bits, and
its training."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from gpu_util import import_ito
    import_ito()
    spec = importlib.util.spec_from_file_location("float_residual_mlp",
                                                  os.path.join(ROOT, "examples", "float_residual_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_64_bits(ex):
    """bf16 activations and gradients carry a relative rounding of 2^-9 at each of about a dozen
    places between a weight and the loss; independent, they add up to about sqrt(12) 2^-9 = 0.7 %
    of a gradient's norm, and to 12 * 2^-8 = 4.7 % if all of them pull one way at their worst."""
    import torch
    model = ex.ResidualMlp(32, 64, 2, 10)
    x, labels = next(ex.batches(256, 32, 10))
    loss, _, keep = model.forward(x, labels)
    grads = model.backward(keep)
    ws = [w.double().requires_grad_() for w in model.weights]
    # the copies the products read are bf16: compare at those weights
    at = [w if i in (0,) or w.dim() == 1 and (i - 1) % 6 < 2 and i < len(ws) - 2 else c.double().requires_grad_()
          for i, (w, c) in enumerate(zip(ws, model.copies))]
    h = x.double() @ at[0].T
    for i in range(2):
        gamma, beta, w1, b1, w2, b2 = at[1 + 6 * i:7 + 6 * i]
        n = torch.nn.functional.layer_norm(h, (64,), gamma, beta, 1e-5)
        h = h + torch.nn.functional.gelu(n @ w1.T + b1) @ w2.T + b2
    want = torch.nn.functional.cross_entropy(h @ at[-2].T + at[-1], labels.long())
    assert abs(float(loss) - float(want)) <= 12 * 2.0 ** -8 * abs(float(want))
    for i, (g, w) in enumerate(zip(grads, torch.autograd.grad(want, at))):
        assert g.shape == w.shape
        assert float((g.double() - w).norm()) <= 12 * 2.0 ** -8 * float(w.norm()), i


@pytest.mark.parametrize("bits", [8, 32])
def test_training(ex, bits):
    """The loss falls to less than half of a uniform guess's, log 10, and does so again bit for bit."""
    import math
    import torch

    def train():
        model = ex.ResidualMlp(32, 128, 2, 10, bits=bits)
        data = ex.batches(512, 32, 10)
        return torch.stack([model.step(*next(data), lr=2e-3) for _ in range(150)])

    losses = train()
    assert float(losses[:5].mean()) > 0.8 * math.log(10)
    assert float(losses[-10:].mean()) < 0.5 * math.log(10)
    assert torch.equal(losses, train())
