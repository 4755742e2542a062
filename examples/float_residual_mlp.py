"""Trains a float residual MLP on top of a DFP16 layer, on seeded synthetic data.

    python examples/float_residual_mlp.py [--steps 200] [--bits 8|32]

One step runs the library's operators as a training program uses them:

  features   an integer layer: float input and master weights quantised to DFP16
             (ito_dfp16_from_float), the exact product with FP32 output (ito_dfp16_linear_fwd_f32)
  blocks     h = h + W2 gelu(W1 norm(h) + b1) + b2 in bf16 (ito_layer_norm_fwd, ito_fp_linear_fwd
             with activation, residual and the saved z in the products' epilogues)
  loss       the mean negative log probability of the labels (ito_token_logprobs_fwd)
  backward   ito_token_logprobs_bwd, ito_fp_linear_bwd, ito_layer_norm_bwd; the integer layer's
             weight gradient is the DFP16 product ito_dfp16_linear_wgrad
  update     AdamW over all tensors in one call, FP32 master weights with bf16 copies for the
             float layers, moments in 8 or 32 bits

The page behind the DFP16 layers (Mixed Precision Training of Convolutional Neural Networks
using Integer Operations, sections 3 and 4) trains so: integer products with FP32 outputs, FP32
master weights that an FP32 optimizer updates and that are quantised for the next step.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import integer_only_nn_gb300 as ito


class ResidualMlp:
    """The model's master weights (float32), their bf16 copies, and the steps over them."""

    def __init__(self, inputs, width, blocks, classes, bits=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, fan):
            return torch.randn(shape, generator=gen, device=device) * fan ** -0.5

        zeros = lambda n: torch.zeros(n, device=device)                  # noqa: E731
        ones = lambda n: torch.ones(n, device=device)                    # noqa: E731
        self.blocks = blocks
        self.weights = [normal(width, inputs, fan=inputs)]
        for _ in range(blocks):
            self.weights += [ones(width), zeros(width), normal(width, width, fan=width), zeros(width),
                             normal(width, width, fan=width), zeros(width)]
        self.weights += [normal(classes, width, fan=width), zeros(classes)]
        self.copies = [w.to(torch.bfloat16) for w in self.weights]
        decay = [0.01 if w.dim() == 2 else 0.0 for w in self.weights]    # matrices only
        self.optimizer = ito.AdamW(self.weights, bits=bits, weight_decay=decay, copies=self.copies, seed=seed)

    def _block(self, i):
        """norm weight and bias (float32), W1, b1, W2, b2 (bf16 copies)."""
        at = 1 + 6 * i
        return self.weights[at:at + 2] + self.copies[at + 2:at + 6]

    def forward(self, x, labels, k=0):
        """-> (mean loss, entropy and the k alternatives of each row, what the backward pass needs)"""
        keep = {"labels": labels}
        xm, xe = ito.ito_dfp16_from_float(x)
        wm, we = ito.ito_dfp16_from_float(self.weights[0])
        _, features = ito.ito_dfp16_linear_fwd_f32(xm, xe, wm, we)
        keep["x"] = (xm, xe)
        h = features.to(torch.bfloat16)
        keep["blocks"] = []
        for i in range(self.blocks):
            gamma, beta, w1, b1, w2, b2 = self._block(i)
            n, mean, rstd = ito.ito_layer_norm_fwd(h, gamma, beta)
            a, z = ito.ito_fp_linear_fwd(n, w1, bias=b1, act="gelu", save_z=True)
            keep["blocks"].append((h, mean, rstd, n, z, a))
            h = ito.ito_fp_linear_fwd(a, w2, bias=b2, residual=h)
        logits = ito.ito_fp_linear_fwd(h, self.copies[-2], bias=self.copies[-1], out_dtype=torch.float32)
        logp, entropy, lse, ids, top = ito.ito_token_logprobs_fwd(logits, labels, k=k)
        keep.update(h=h, logits=logits, lse=lse, entropy=entropy)
        return -logp.mean(), (entropy, ids, top), keep

    def backward(self, keep):
        """The gradients of the mean loss, in the order of the weights (float32)."""
        rows = keep["logits"].shape[0]
        g = torch.full((rows,), -1.0 / rows, device=keep["logits"].device)
        d = ito.ito_token_logprobs_bwd(keep["logits"], keep["labels"], keep["lse"], keep["entropy"], g)
        d, dw, db = ito.ito_fp_linear_bwd(d.to(torch.bfloat16), keep["h"], self.copies[-2], dw_dtype=torch.float32)
        grads = [db, dw]
        for i in reversed(range(self.blocks)):
            gamma, _, w1, _, w2, _ = self._block(i)
            h, mean, rstd, n, z, a = keep["blocks"][i]
            da, dw2, db2 = ito.ito_fp_linear_bwd(d, a, w2, dw_dtype=torch.float32)
            dn, dw1, db1 = ito.ito_fp_linear_bwd(da, n, w1, z=z, act="gelu", dw_dtype=torch.float32)
            dh, dgamma, dbeta = ito.ito_layer_norm_bwd(dn, h, gamma, mean, rstd)
            grads += [db2, dw2, db1, dw1, dbeta, dgamma]
            d = d + dh                                                   # past the block and through it
        dm, de = ito.ito_dfp16_from_float(d.float())
        xm, xe = keep["x"]
        _, _, gm, ge, _ = ito.ito_dfp16_linear_wgrad(dm, de, xm, xe)
        grads.append(ito.ito_dfp16_to_float(gm, ge))
        return grads[::-1]

    def step(self, x, labels, lr):
        loss, _, keep = self.forward(x, labels)
        self.optimizer.step(self.backward(keep), lr=lr)
        return loss


def batches(rows, inputs, classes, seed=1, device="cuda"):
    """Seeded inputs whose labels a fixed random two-layer net gives."""
    gen = torch.Generator(device=device).manual_seed(seed)
    a = torch.randn((inputs, 2 * inputs), generator=gen, device=device) * inputs ** -0.5
    b = torch.randn((2 * inputs, classes), generator=gen, device=device)
    while True:
        x = torch.randn((rows, inputs), generator=gen, device=device)
        yield x, (torch.relu(x @ a) @ b).argmax(1).to(torch.int32)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--inputs", type=int, default=64)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--classes", type=int, default=10)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args()
    model = ResidualMlp(a.inputs, a.width, a.blocks, a.classes, bits=a.bits)
    data = batches(a.rows, a.inputs, a.classes)
    for t in range(a.steps):
        loss = model.step(*next(data), lr=a.lr)
        if t % 20 == 0 or t == a.steps - 1:
            print("step %4d  loss %.4f" % (t, float(loss)))
    x, labels = next(data)
    loss, (entropy, ids, top), _ = model.forward(x, labels, k=3)
    right = float((ids[:, 0] == labels).float().mean())
    print("held-out loss %.4f, %.1f %% right, mean entropy %.3f" % (float(loss), 100 * right, float(entropy.mean())))
    print("row 0: label %d, alternatives %s with log probabilities %s" % (
        int(labels[0]), ids[0].tolist(), ["%.2f" % v for v in top[0].tolist()]))


if __name__ == "__main__":
    main()
