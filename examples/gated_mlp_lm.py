"""Trains a small language model whose passes run on the operators of the package and whose step is dp_step.

The model is a stack of gated MLP blocks over single tokens (next token from this one): embedding with scaling, norms before and
after each block with a gate into the residual stream, SwiGLU, a tied output layer.  n data-parallel ranks with a micro-steps
each hold their bf16 gradients in flat buffers; every gradient is written by the operator that computes it straight into its
slice.  Between the passes a block's input and activations are kept as 8-bit checkpoints.  Library products (torch.mm) do the
forward and input-gradient matrix products.

    python examples/gated_mlp_lm.py [--steps 60] [--layers 3] [--dim 256] [--hidden 704] [--vocab 1000] [--tokens 2048]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_gradient_sync_gb300 as dp  # noqa: E402
from zero_gradient_sync_gb300.buffers import StepBuffers  # noqa: E402

BF = torch.bfloat16
EPS = 1e-5


class Model:
    """Shapes and offsets of the parameters in the flat space, and the two passes of one micro-step."""

    def __init__(self, vocab: int, dim: int, hidden: int, layers: int, tokens: int):
        self.vocab, self.dim, self.hidden, self.layers, self.tokens = vocab, dim, hidden, layers, tokens
        self.shapes = {"embed": (vocab, dim), "pre0": (dim,)}
        for l in range(layers):
            self.shapes.update({"up%d" % l: (2 * hidden, dim), "down%d" % l: (dim, hidden), "post%d" % l: (dim,), "gate%d" % l: (dim,),
                                "pre%d" % (l + 1): (dim,)})
        self.offset, at = {}, 0
        for k, s in self.shapes.items():
            self.offset[k] = at
            at += math.prod(s)
            at += -at % 8       # 16-byte aligned rows take wider loads
        self.psi = at
        new = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        T = tokens
        # what is kept from the forward to the backward pass, per boundary and block
        self.r = [new(T, dim) for _ in range(layers + 1)]
        self.y = [new(T, dim) for _ in range(layers)]
        self.pre_stats = [new(T, 2, dtype=torch.float32) for _ in range(layers + 1)]
        self.post_stats = [new(T, 2, dtype=torch.float32) for _ in range(layers)]
        self.z8 = [dp.new_ckpt8(T, dim) for _ in range(layers + 1)]
        self.g8 = [dp.new_ckpt8(T, hidden) for _ in range(layers)]
        self.u8 = [dp.new_ckpt8(T, hidden) for _ in range(layers)]
        # scratch
        self.z, self.h, self.gu, self.dgu, self.dh = new(T, dim), new(T, hidden), new(T, 2 * hidden), new(T, 2 * hidden), new(T, hidden)
        self.dr, self.dy, self.dz = new(T, dim), new(T, dim), new(T, dim)
        need = max([dp.dp_embedding_workspace_size(T, vocab, dim), dp.dp_block_norm_workspace_size(T, dim),
                    dp.dp_wgrad8_workspace_size(T, vocab, dim), dp.dp_wgrad8_workspace_size(T, 2 * hidden, dim)])
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def views(self, flat):
        return {k: flat[o:o + math.prod(s)].view(s) for (k, s), o in zip(self.shapes.items(), self.offset.values())}

    def init(self, seed: int = 0):
        """fp32 starting values of the flat parameter space."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        flat = torch.zeros(self.psi, device="cuda")
        for k, v in self.views(flat).items():
            if v.dim() == 2:
                v.copy_(torch.randn(v.shape, generator=gen, device="cuda") * (1.0 / math.sqrt(v.shape[1])))
            else:
                v.fill_(0.5 if k.startswith("gate") else 1.0)
        return flat

    def forward_backward(self, params, grads, ids, targets, loss_scale: float):
        """One micro-step: writes every gradient (times loss_scale) into the flat buffer `grads`; returns the mean loss."""
        w, g = self.views(params), self.views(grads)
        scale = math.sqrt(self.dim)
        # ---- forward
        dp.dp_embedding(self.r[0], w["embed"], ids, scale=scale)
        dp.dp_block_norm(None, self.z, self.r[0], w_pre=w["pre0"], eps=EPS, pre_stats=self.pre_stats[0])
        for l in range(self.layers):
            dp.dp_ckpt8_encode(*self.z8[l], self.z)
            torch.mm(self.z, w["up%d" % l].t(), out=self.gu)
            dp.dp_act_ckpt8(self.h, self.gu[:, :self.hidden], self.gu[:, self.hidden:], act=dp.DP_ACT_SILU, g8=self.g8[l], u8=self.u8[l])
            torch.mm(self.h, w["down%d" % l].t(), out=self.y[l])
            dp.dp_block_norm(self.r[l + 1], self.z, self.r[l], self.y[l], w_post=w["post%d" % l], gate=w["gate%d" % l],
                             w_pre=w["pre%d" % (l + 1)], eps=EPS, post_stats=self.post_stats[l], pre_stats=self.pre_stats[l + 1])
        dp.dp_ckpt8_encode(*self.z8[-1], self.z)
        logits = torch.mm(self.z, w["embed"].t()).float()
        logp = logits - logits.logsumexp(1, keepdim=True)
        loss = -logp.gather(1, targets[:, None]).mean()
        # ---- backward
        dlogits = logp.exp()
        dlogits.scatter_add_(1, targets[:, None], torch.full_like(targets[:, None], -1.0, dtype=torch.float32))
        dlogits = (dlogits * (loss_scale / self.tokens)).to(BF)
        dp.dp_wgrad8(g["embed"], dlogits, *self.z8[-1], ws=self.ws)          # the output layer's part of the tied weight
        torch.mm(dlogits, w["embed"], out=self.dz)
        dr = None
        for l in reversed(range(self.layers)):
            dp.dp_block_norm_grad(self.dr, self.dy, dr, self.dz, self.r[l + 1], self.y[l], w_post=w["post%d" % l], gate=w["gate%d" % l],
                                  w_pre=w["pre%d" % (l + 1)], post_stats=self.post_stats[l], pre_stats=self.pre_stats[l + 1],
                                  dw_post=g["post%d" % l], dgate=g["gate%d" % l], dw_pre=g["pre%d" % (l + 1)], ws=self.ws)
            dr = self.dr
            torch.mm(self.dy, w["down%d" % l], out=self.dh)
            dp.dp_act_ckpt8_grad(self.dgu[:, :self.hidden], self.dgu[:, self.hidden:], self.dh, act=dp.DP_ACT_SILU, g8=self.g8[l],
                                 u8=self.u8[l], h=self.h)
            torch.mm(self.dy.t(), self.h, out=g["down%d" % l])
            dp.dp_wgrad8(g["up%d" % l], self.dgu, *self.z8[l], ws=self.ws)
            torch.mm(self.dgu, w["up%d" % l], out=self.dz)
        dp.dp_block_norm_grad(self.dr, None, dr, self.dz, self.r[0], w_pre=w["pre0"], pre_stats=self.pre_stats[0], dw_pre=g["pre0"], ws=self.ws)
        dp.dp_embedding_grad(g["embed"], self.dr, ids, scale=scale, accumulate=True, ws=self.ws)   # and the lookup's
        return loss


def batch(vocab: int, tokens: int, gen):
    """A language with a rule: the next token is 7 t + 3 (mod vocab), one time in eight anything."""
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    noise = torch.rand(tokens, generator=gen, device="cuda") < 0.125
    return ids, torch.where(noise, torch.randint(0, vocab, (tokens,), generator=gen, device="cuda"), (7 * ids + 3) % vocab)


def train(steps=60, layers=3, dim=256, hidden=704, vocab=1000, tokens=2048, n=2, a=2, lr=3e-3, loss_scale=256.0, report=None):
    model = Model(vocab, dim, hidden, layers, tokens)
    layout = dp.Layout.even(model.psi, n, stage=1)
    bufs = StepBuffers(layout, a)
    start = model.init()
    for goff, length, owner, loff in layout.segs:
        bufs.master[owner][loff:loff + length].copy_(start[goff:goff + length])
    for rep in bufs.replicas:
        rep.copy_(start)
    for q in bufs.grads:
        q.zero_()                      # the few elements between the tensors
    gen = torch.Generator(device="cuda").manual_seed(1)
    adam, losses = dp.adam(lr=lr), []
    for step in range(steps):
        total = 0.0
        for r in range(n):
            for k in range(a):
                total = total + model.forward_backward(bufs.replicas[r], bufs.grad(r, k), *batch(vocab, tokens, gen), loss_scale)
        # the step adds the a micro-steps: their mean takes a's share of the scale
        bufs.step(adam, loss_scale * a)
        losses.append(float(total) / (n * a))
        if report and (step % 10 == 0 or step == steps - 1):
            report("step %3d  loss %.4f" % (step, losses[-1]))
    return losses, bufs.status()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 60), ("layers", 3), ("dim", 256), ("hidden", 704), ("vocab", 1000), ("tokens", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    train(**vars(args), report=print)
