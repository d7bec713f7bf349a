"""A two-layer token model trained wholly through the library: the next token
is predicted from the embedding of the current one.

    python examples/train_bigram.py [--tied] [--layer] [--steps 60]

The weights live as FP32 master tiles in one rank's shard and are read as the
row-major FP8 codes and scale grids that the step writes.  A step:

    embed            hidden = FP8 rows of the embedding
    vocab_loss       loss over the FP8 head, logits never stored
    vocab_loss_grad  gradients of the hidden rows and of the head
    embed_grad       gradient of the embedding (tied: added to the head's)
    shard_grad_norm  the norm, and the factor that clips it
    fold_adamw_fp8_step_unpack  clipping, AdamW and requantization in one pass

With --layer a layer stands between them: layer norm, whose weight and bias an
AdamWList keeps with 8-bit states, and a square FP8 weight:

    layer_norm, quantize, linear            on the way to the head
    quantize, linear_grad_input, linear_grad_weight, layer_norm_grad   back
    grad_norm, clip_coef, AdamWList.step    norm and step of what is no FP8 weight
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blockwise_fp8_zero_amd as bfz  # noqa: E402


class Bigram:
    """Weights, FP8 copies and workspaces for batches of n tokens."""

    def __init__(self, vocab, dim, n, tied=False, max_norm=1.0, lr=1e-2, layer=False):
        self.tied, self.max_norm, self.lr, self.t, self.layer = tied, max_norm, lr, 1, layer
        weights = 1 if tied else 2
        dims = [(1, vocab, dim)] * weights + [(1, dim, dim)] * layer
        f32 = dict(dtype=torch.float32, device="cuda")
        self.plan = bfz.Plan(dims)
        q = self.plan.shard_tiles
        self.state = torch.zeros(q, bfz.STATE_STRIDE, **f32)
        self.master, self.m, self.v = (self.state[:, k * 16384:(k + 1) * 16384] for k in range(3))
        bfz.pack_shard(self.plan, [torch.randn(H, W, **f32) * dim ** -0.5 for _, H, W in dims], self.master)
        self.codes = torch.empty(q * 16384, dtype=torch.uint8, device="cuda")
        self.scale_inv = torch.empty(q, **f32)
        self.fp8 = [torch.zeros(H, W, dtype=torch.uint8, device="cuda") for _, H, W in dims]
        self.grid = [torch.zeros(-(-H // 128), -(-W // 128), **f32) for _, H, W in dims]
        self.grads = [torch.zeros(H, W, **f32) for _, H, W in dims]
        self.head = weights - 1
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
        if layer:
            self._layer(n, dim, f32)

    def _layer(self, n, dim, f32):
        self.params = [torch.ones(dim, **f32), torch.zeros(dim, **f32)]  # the norm's weight and bias
        self.param_grads = [torch.zeros(dim, **f32) for _ in self.params]
        self.opt = bfz.AdamWList(self.params, *bfz.adamw_states(self.params, bits=8), grads=self.param_grads)
        self.normed, self.out, self.dout, self.dnormed = (torch.empty_like(self.hidden) for _ in range(4))
        self.mean, self.rstd = torch.empty(n, **f32), torch.empty(n, **f32)
        (self.codes_in, self.grid_in), (self.codes_out, self.grid_out) = (bfz.quantize_buffers(n, dim, tiles=True) for _ in range(2))
        self.norm_grad_work, self.linear_work = bfz.layer_norm_workspace(n, dim), bfz.linear_workspace(n, self.fp8[-1])
        self.sums = [torch.empty(1, dtype=torch.float64, device="cuda") for _ in range(2)]

    def _forward(self):
        """The head's input."""
        if not self.layer:
            return self.hidden
        bfz.layer_norm(self.hidden, *self.params, self.normed, mean=self.mean, rstd=self.rstd)
        bfz.quantize(self.normed, self.codes_in, self.grid_in, tiles=True)
        bfz.linear(self.codes_in, self.fp8[-1], self.grid[-1], self.out, self.linear_work, scales=self.grid_in, tiles=True)
        return self.out

    def _backward(self):
        """From the gradient of the head's input to dhidden."""
        bfz.quantize(self.dout, self.codes_out, self.grid_out, tiles=True)
        bfz.linear_grad_weight(self.codes_out, self.grid_out, self.codes_in, self.grid_in, self.grads[-1], self.linear_work)
        bfz.linear_grad_input(self.codes_out, self.fp8[-1], self.grid[-1], self.dnormed, self.linear_work, scales=self.grid_out, tiles=True)
        bfz.layer_norm_grad(self.dnormed, self.hidden, self.params[0], self.mean, self.rstd, self.dhidden, *self.param_grads,
                            self.norm_grad_work)

    def _clip(self):
        """norm and coef over all gradients."""
        if not self.layer:
            bfz.shard_grad_norm(self.plan, self.grads, self.norm, self.norm_work, max_norm=self.max_norm, coef=self.coef)
            return
        bfz.shard_grad_norm(self.plan, self.grads, None, self.norm_work, sumsq=self.sums[0])
        bfz.grad_norm(self.param_grads, None, self.norm_work, sumsq=self.sums[1])
        bfz.clip_coef(self.sums[0] + self.sums[1], self.max_norm, self.norm, self.coef)

    def _update(self, weight_decay=0.01, coef=None):
        hp = bfz.AdamW(lr=self.lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=weight_decay, step=self.t)
        bfz.fold_adamw_fp8_step_unpack(self.plan, self.grads, self.master, self.m, self.v, self.codes, self.scale_inv,
                                       self.fp8, self.grid, hp, grad_scale=coef)
        if self.layer and coef is not None:
            self.opt.step(hp, grad_scale=coef)

    def step(self, tokens, targets):
        """One training step; returns the mean loss (a device scalar).  A target
        of -1 counts for nothing."""
        head = self.head
        dloss = torch.full_like(self.loss, 1.0 / tokens.numel())
        bfz.embed(tokens, self.fp8[0], self.hidden, grid=self.grid[0], scale=self.hidden.shape[1] ** 0.5)
        x, dx = self._forward(), self.dout if self.layer else self.dhidden
        bfz.vocab_loss(x, self.fp8[head], targets, self.loss, self.lse, self.loss_work, grid=self.grid[head])
        bfz.vocab_loss_grad(x, self.fp8[head], targets, self.lse, dloss, dx, self.grads[head], self.loss_work, grid=self.grid[head])
        if self.layer:
            self._backward()
        bfz.embed_grad(tokens, self.dhidden, self.grads[0], self.embed_work, scale=self.hidden.shape[1] ** 0.5,
                       accumulate=self.tied)
        self._clip()
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


def train(vocab=1000, dim=256, n=2048, steps=60, tied=False, verbose=True, layer=False):
    torch.manual_seed(0)
    model, losses = Bigram(vocab, dim, n, tied, layer=layer), []
    for t, (tokens, targets) in zip(range(steps), batches(vocab, n)):
        losses.append(float(model.step(tokens, targets)))
        if verbose and (t % 10 == 0 or t == steps - 1):
            print(f"step {t + 1}: loss {losses[-1]:.4f}, gradient norm {float(model.norm):.4f}", flush=True)
    return model, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tied", action="store_true")
    ap.add_argument("--layer", action="store_true")
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    train(steps=a.steps, tied=a.tied, layer=a.layer)
