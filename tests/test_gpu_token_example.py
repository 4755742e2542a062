"""The gated token model: its gradients against the same model in 64 bits, and that it trains."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from gpu_util import import_ito
    import_ito()
    spec = importlib.util.spec_from_file_location("token_gated_mlp", os.path.join(ROOT, "examples", "token_gated_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("places", [5, 300])
def test_gradients_against_64_bits(ex, places):
    """bf16 activations and gradients carry a relative rounding of 2^-9 at each of about sixteen places between
    a weight and the loss, 2^-8 at the worst: 16 * 2^-8 of a gradient's norm where all pull one way."""
    import torch
    model = ex.TokenGatedMlp(101, 72, 136, 2)
    ids, targets = next(ex.batches(places, 101))
    ids[1], targets[2] = -1, -1
    loss, keep = model.forward(ids, targets)
    g = torch.rand((places,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") / places
    grads = model.backward(keep, g)
    # the weights that the products read are bf16, the norms' float32
    at = [(w if w.dim() == 1 else c).double().requires_grad_() for w, c in zip(model.weights, model.copies)]
    x = at[0][ids.long().clamp(min=0)] * model.scale * (ids >= 0)[:, None]
    norm = torch.nn.functional.layer_norm
    for i in range(2):
        gamma, beta, wg, wu, wd = at[1 + 5 * i:6 + 5 * i]
        n = norm(x, (72,), gamma, beta, 1e-5)
        x = x + (torch.nn.functional.silu(n @ wg.T) * (n @ wu.T)) @ wd.T
    logits = norm(x, (72,), at[-2], at[-1], 1e-5) @ at[0].T
    want = torch.nn.functional.cross_entropy(logits, targets.long(), ignore_index=-1, reduction="none")
    assert float((loss.double() - want).detach().norm()) <= 16 * 2.0 ** -8 * float(want.detach().norm())
    for i, (got, w) in enumerate(zip(grads, torch.autograd.grad((want * g.double()).sum(), at))):
        assert got.shape == w.shape and got.dtype == torch.float32
        assert float((got.double() - w).norm()) <= 16 * 2.0 ** -8 * float(w.norm()), i


@pytest.mark.parametrize("bits", [8, 32])
def test_steps(ex, bits):
    """Steps run, change the weights and their copies, and give the same bits again."""
    import torch

    def train():
        model = ex.TokenGatedMlp(120, 64, 96, 1, bits=bits)
        before = [w.clone() for w in model.weights]
        data = ex.batches(256, 120)
        losses = torch.stack([model.step(*next(data), lr=1e-3) for _ in range(6)])
        assert all(not torch.equal(a, b) for a, b in zip(before, model.weights))
        assert all(torch.equal(c, w.to(torch.bfloat16)) for w, c in zip(model.weights, model.copies))
        return losses

    losses = train()
    assert bool(torch.isfinite(losses).all()) and torch.equal(losses, train())


def test_program(ex, monkeypatch, capsys):
    import sys
    monkeypatch.setattr(sys, "argv", ["token_gated_mlp.py", "--steps", "3", "--places", "128", "--tokens", "50", "--width",
                                      "32", "--hidden", "48", "--blocks", "1"])
    ex.main()
    assert "one place" in capsys.readouterr().out
