"""A two-layer token model trained wholly through the library: the next token
is predicted from the embedding of the current one.

    python examples/train_bigram.py [--tied] [--steps 60]

Both weights live as FP32 master tiles in one rank's shard and are read as the
row-major FP8 codes and scale grids that the step writes.  A step:

    embed            hidden = FP8 rows of the embedding
    vocab_loss       loss over the FP8 head, logits never stored
    vocab_loss_grad  gradients of the hidden rows and of the head
    embed_grad       gradient of the embedding (tied: added to the head's)
    shard_grad_norm  the norm, and the factor that clips it
    fold_adamw_fp8_step_unpack  clipping, AdamW and requantization in one pass
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blockwise_fp8_zero_amd as bfz  # noqa: E402


class Bigram:
    """Weights, FP8 copies and workspaces for batches of n tokens."""

    def __init__(self, vocab, dim, n, tied=False, max_norm=1.0, lr=1e-2):
        self.tied, self.max_norm, self.lr, self.t = tied, max_norm, lr, 1
        weights = 1 if tied else 2
        dims = [(1, vocab, dim)] * weights
        f32 = dict(dtype=torch.float32, device="cuda")
        self.plan = bfz.Plan(dims)
        q = self.plan.shard_tiles
        self.state = torch.zeros(q, bfz.STATE_STRIDE, **f32)
        self.master, self.m, self.v = (self.state[:, k * 16384:(k + 1) * 16384] for k in range(3))
        bfz.pack_shard(self.plan, [torch.randn(vocab, dim, **f32) * dim ** -0.5 for _ in dims], self.master)
        self.codes = torch.empty(q * 16384, dtype=torch.uint8, device="cuda")
        self.scale_inv = torch.empty(q, **f32)
        self.fp8 = [torch.zeros(vocab, dim, dtype=torch.uint8, device="cuda") for _ in dims]
        self.grid = [torch.zeros(-(-vocab // 128), -(-dim // 128), **f32) for _ in dims]
        self.grads = [torch.zeros(vocab, dim, **f32) for _ in dims]
        # a step with zero gradients and no decay leaves the master as it is
        # and writes its FP8 copies
        self._update(weight_decay=0.0)
        self.hidden = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
        self.dhidden = torch.empty_like(self.hidden)
        self.loss, self.lse = torch.empty(n, **f32), torch.empty(n, **f32)
        self.norm, self.coef = torch.empty(1, **f32), torch.empty(1, **f32)
        self.norm_work = bfz.norm_workspace()
        self.embed_work = bfz.embed_grad_workspace(n, dim)
        self.loss_work = bfz.vocab_loss_workspace(n, vocab, dim)

    def _update(self, weight_decay=0.01, coef=None):
        hp = bfz.AdamW(lr=self.lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=weight_decay, step=self.t)
        bfz.fold_adamw_fp8_step_unpack(self.plan, self.grads, self.master, self.m, self.v, self.codes, self.scale_inv,
                                       self.fp8, self.grid, hp, grad_scale=coef)

    def step(self, tokens, targets):
        """One training step; returns the mean loss (a device scalar).  A target
        of -1 counts for nothing."""
        head = len(self.fp8) - 1
        dloss = torch.full_like(self.loss, 1.0 / tokens.numel())
        bfz.embed(tokens, self.fp8[0], self.hidden, grid=self.grid[0], scale=self.hidden.shape[1] ** 0.5)
        bfz.vocab_loss(self.hidden, self.fp8[head], targets, self.loss, self.lse, self.loss_work, grid=self.grid[head])
        bfz.vocab_loss_grad(self.hidden, self.fp8[head], targets, self.lse, dloss, self.dhidden, self.grads[head],
                            self.loss_work, grid=self.grid[head])
        bfz.embed_grad(tokens, self.dhidden, self.grads[0], self.embed_work, scale=self.hidden.shape[1] ** 0.5,
                       accumulate=self.tied)
        bfz.shard_grad_norm(self.plan, self.grads, self.norm, self.norm_work, max_norm=self.max_norm, coef=self.coef)
        self._update(coef=self.coef)
        self.t += 1
        return self.loss.mean()


def batches(vocab, n, seed=0):
    """Tokens whose successor is one of two, by a fixed rule."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    while True:
        tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
        coin = torch.randint(0, 2, (n,), generator=gen, device="cuda")
        yield tokens, (7 * tokens + 13 + coin * 101) % vocab


def train(vocab=1000, dim=256, n=2048, steps=60, tied=False, verbose=True):
    torch.manual_seed(0)
    model, losses = Bigram(vocab, dim, n, tied), []
    for t, (tokens, targets) in zip(range(steps), batches(vocab, n)):
        losses.append(float(model.step(tokens, targets)))
        if verbose and (t % 10 == 0 or t == steps - 1):
            print(f"step {t + 1}: loss {losses[-1]:.4f}, gradient norm {float(model.norm):.4f}", flush=True)
    return model, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tied", action="store_true")
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    train(steps=a.steps, tied=a.tied)
