"""Trains a token model of gated blocks with a tied table, on seeded synthetic text.

    python examples/token_gated_mlp.py [--steps 200] [--bits 8|32]

A model of the next token given the one before it (no attention: a block sees one place). One step runs
the library's operators as a training program uses them:

  input      x = sqrt(width) table[token] (ito_embedding_fwd)
  blocks     x = x + Wd h, h = silu(Wg n) * (Wu n), n = norm(x), in bf16 (ito_layer_norm_fwd,
             ito_fp_gated_linear_fwd, ito_fp_linear_fwd with the residual in its epilogue)
  loss       the cross entropy of the next token under table norm(x), without the logits in memory
             (ito_linear_cross_entropy_fwd); places without a next token have the target -1
  backward   ito_linear_cross_entropy_bwd, whose table gradient the input's is added to in place
             (ito_embedding_bwd with add_to), ito_fp_linear_bwd, ito_fp_gated_linear_bwd, ito_layer_norm_bwd
  update     AdamW over all tensors in one call, FP32 master weights with bf16 copies
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import integer_only_nn_gb300 as ito


class TokenGatedMlp:
    """The model's master weights (float32), their bf16 copies, and the steps over them."""

    PER = 5              # tensors of a block: norm weight and bias, Wg, Wu, Wd

    def __init__(self, tokens, width, hidden, blocks, bits=32, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, fan):
            return torch.randn(shape, generator=gen, device=device) * fan ** -0.5

        self.tokens, self.blocks, self.scale = tokens, blocks, width ** 0.5
        self.weights = [normal(tokens, width, fan=width)]
        for _ in range(blocks):
            self.weights += [torch.ones(width, device=device), torch.zeros(width, device=device),
                             normal(hidden, width, fan=width), normal(hidden, width, fan=width),
                             normal(width, hidden, fan=hidden)]
        self.weights += [torch.ones(width, device=device), torch.zeros(width, device=device)]
        self.copies = [w.to(torch.bfloat16) for w in self.weights]
        decay = [0.01 if w.dim() == 2 else 0.0 for w in self.weights]
        self.optimizer = ito.AdamW(self.weights, bits=bits, weight_decay=decay, copies=self.copies, seed=seed)

    def _block(self, i):
        """norm weight and bias (float32), Wg, Wu, Wd (bf16 copies)."""
        at = 1 + self.PER * i
        return self.weights[at:at + 2] + self.copies[at + 2:at + 5]

    def forward(self, ids, targets):
        """-> (each place's loss, what the backward pass needs)"""
        x = ito.ito_embedding_fwd(ids, self.copies[0], scale=self.scale)
        kept = []
        for i in range(self.blocks):
            gamma, beta, wg, wu, wd = self._block(i)
            n, mean, rstd = ito.ito_layer_norm_fwd(x, gamma, beta)
            h, zg, zu = ito.ito_fp_gated_linear_fwd(n, wg, wu, act="silu", save_z=True)
            kept.append((x, mean, rstd, n, h, zg, zu))
            x = ito.ito_fp_linear_fwd(h, wd, residual=x)
        n, mean, rstd = ito.ito_layer_norm_fwd(x, self.weights[-2], self.weights[-1])
        loss, lse = ito.ito_linear_cross_entropy_fwd(n, self.copies[0], targets)
        return loss, dict(ids=ids, targets=targets, blocks=kept, last=(x, mean, rstd, n), lse=lse)

    def backward(self, keep, g):
        """The gradients of sum(g loss) in the order of the weights (float32)."""
        x, mean, rstd, n = keep["last"]
        dn, dtable = ito.ito_linear_cross_entropy_bwd(n, self.copies[0], keep["targets"], keep["lse"], g,
                                                      dw_dtype=torch.float32)
        dx, dgamma, dbeta = ito.ito_layer_norm_bwd(dn, x, self.weights[-2], mean, rstd)
        grads = [dbeta, dgamma]
        for i in reversed(range(self.blocks)):
            gamma, _, wg, wu, wd = self._block(i)
            x, mean, rstd, n, h, zg, zu = keep["blocks"][i]
            dh, dwd, _ = ito.ito_fp_linear_bwd(dx, h, wd, need_dbias=False, dw_dtype=torch.float32)
            dn, dwg, dwu, _, _ = ito.ito_fp_gated_linear_bwd(dh, n, wg, wu, zg, zu, act="silu", dw_dtype=torch.float32)
            d, dgamma, dbeta = ito.ito_layer_norm_bwd(dn, x, gamma, mean, rstd)
            grads += [dwd, dwu, dwg, dbeta, dgamma]
            dx = dx + d                                              # past the block and through it
        grads.append(ito.ito_embedding_bwd(dx, keep["ids"], self.tokens, scale=self.scale, add_to=dtable))
        return grads[::-1]

    def step(self, ids, targets, lr):
        loss, keep = self.forward(ids, targets)
        n = (targets >= 0).sum().clamp(min=1)
        self.optimizer.step(self.backward(keep, (1.0 / n).expand(loss.shape[0]).contiguous()), lr=lr)
        return loss.sum() / n


def batches(places, tokens, seed=1, device="cuda"):
    """Seeded text of a fixed random successor of each token, followed three times in four; some targets missing."""
    gen = torch.Generator(device=device).manual_seed(seed)
    after = torch.randperm(tokens, generator=gen, device=device)
    while True:
        ids = torch.randint(0, tokens, (places,), generator=gen, device=device)
        other = torch.randint(0, tokens, (places,), generator=gen, device=device)
        u = torch.rand((places,), generator=gen, device=device)
        targets = torch.where(u < 0.75, after[ids], other)
        targets[u > 0.97] = -1
        yield ids.to(torch.int32), targets.to(torch.int32)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--places", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args()
    model = TokenGatedMlp(a.tokens, a.width, a.hidden, a.blocks, bits=a.bits)
    data = batches(a.places, a.tokens)
    for t in range(a.steps):
        loss = model.step(*next(data), lr=a.lr)
        if t % 20 == 0 or t == a.steps - 1:
            print("step %4d  loss %.4f" % (t, float(loss)))
    ids, targets = next(data)
    loss, _ = model.forward(ids[:1], targets[:1])
    print("one place: token %d, next %d, loss %.4f" % (int(ids[0]), int(targets[0]), float(loss)))


if __name__ == "__main__":
    main()
