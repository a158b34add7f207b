"""Fine-tunes the routed experts of a small latent MoE layer on 16-bit weights.

The frozen layer (MXFP4 experts, k3moe.Layer) routes the tokens.  Its experts, dequantised and disturbed by
noise, are trained to give back the latent output of the undisturbed ones: a step runs every training
operator of latent_moe_layer_gb300.experts forwards and backwards, over two micro-batches whose weight
gradients are accumulated in fp32.

With --one-pass the gated block's projections and unit are one kernel (and again one in the backward pass, which
keeps neither projection); its dropout is then left to the residual.

    python examples/finetune_experts.py [--steps 20] [--tokens 512] [--dropout 0.1] [--act silu|situ] [--one-pass]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from latent_moe_layer_gb300 import experts as ex  # noqa: E402
from latent_moe_layer_gb300 import k3moe, synth  # noqa: E402


class RoutedExperts:
    """w13 [E, 2 I, L] (gate rows, then up rows) and w2 [E, L, I]: 16-bit copies of fp32 masters."""

    def __init__(self, w13, w2, dtype=torch.bfloat16, act="silu", p=0.0, seed=0, one_pass=False):
        self.master = [w13.float().clone(), w2.float().clone()]
        self.w13, self.w2 = w13.to(dtype), w2.to(dtype)
        self.grad = [torch.zeros_like(m) for m in self.master]
        self.act, self.p, self.seed, self.calls, self.one_pass = act, p, seed, 0, one_pass

    def forward(self, h, idx, weights, train=True):
        """h [T, L], idx and weights [T, K] -> h + dropout(sum_k weights y), and what backward needs."""
        p = self.p if train else 0.0
        rnd = dict(p=p, seed=self.seed, offset=2 * self.calls)     # every call its own random numbers
        self.calls += 1
        offsets, pos = ex.plan_rows(idx, self.w13.shape[0])
        xs = ex.gather_rows(h, pos)
        gu = None if self.one_pass else ex.group_mm(xs, self.w13, offsets)
        a = ex.group_glu(xs, self.w13, offsets, act=self.act) if self.one_pass else ex.glu_dropout(gu, act=self.act, **rnd)
        y = ex.group_mm(a, self.w2, offsets)
        z = ex.combine_rows(y, pos, weights)
        out = ex.dropout(z, p, self.seed, rnd["offset"] + 1, residual=h)
        return out, (offsets, pos, weights, xs, gu, a, y, rnd)

    def backward(self, dout, saved):
        """Adds the weight gradients to self.grad; returns (dh, dweights)."""
        offsets, pos, weights, xs, gu, a, y, rnd = saved
        dz = ex.dropout(dout, rnd["p"], self.seed, rnd["offset"] + 1)
        dy, dweights = ex.combine_rows_grad(dz, y, pos, weights, out=y)           # y is not needed any more
        ex.group_mm_grad_w(dy, a, offsets, out=self.grad[1], accumulate=True)
        da = ex.group_mm_grad_x(dy, self.w2, offsets)
        if self.one_pass:
            dgu = ex.group_glu_grad(da, xs, self.w13, offsets, act=self.act)
        else:
            dgu = ex.glu_dropout_grad(da, gu, act=self.act, out=gu, **rnd)        # nor is gu
        ex.group_mm_grad_w(dgu, xs, offsets, out=self.grad[0], accumulate=True)
        dxs = ex.group_mm_grad_x(dgu, self.w13, offsets)
        dh = ex.combine_rows(dxs, pos)
        return dh.add_(dout), dweights                                            # the residual's own path

    def step(self, lr):
        for master, grad, w in zip(self.master, self.grad, (self.w13, self.w2)):
            master.add_(grad, alpha=-lr)
            w.copy_(master)
            grad.zero_()


def dequantised(dw, dtype=torch.float32):
    """The layer's MXFP4 experts as w13 [E, 2 I, L] and w2 [E, L, I]."""
    m = [torch.stack([k3moe.debug_dequant(dw.packed[i][e], dw.scale[i][e]) for e in range(dw.cfg.E)]) for i in range(3)]
    return torch.cat([m[0], m[1]], 1).to(dtype), m[2].to(dtype)


def train(steps=20, tokens=512, p=0.1, act="silu", lr=0.2, verbose=True, one_pass=False):
    """-> the losses (mean squared error per step, dropout off) and the trained experts."""
    cfg = synth.SMALL_ALIGNED.with_tokens(tokens)
    dw = k3moe.DeviceWeights(cfg)
    layer = k3moe.Layer(cfg)
    layer.load(dw)
    w13, w2 = dequantised(dw)
    # weights of unit scale in their input width, so that one learning rate serves both
    w13, w2 = w13 / (w13.std() * cfg.L ** 0.5), w2 / (w2.std() * cfg.I ** 0.5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    noisy = [w + 0.3 * w.std() * torch.randn(w.shape, device="cuda", generator=gen) for w in (w13, w2)]
    teacher, student = RoutedExperts(w13, w2, act=act), RoutedExperts(*noisy, act=act, p=p, seed=7, one_pass=one_pass)
    w_down = dw.w_down.view(torch.bfloat16)[None]                                 # [1, L, H]: one "expert"
    all_rows = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    batches = []
    for b in range(2):
        x = torch.randn(tokens, cfg.H, device="cuda", generator=gen).bfloat16()
        idx = torch.empty((tokens, cfg.K), dtype=torch.int32, device="cuda")
        weights = torch.empty((tokens, cfg.K), dtype=torch.float32, device="cuda")
        layer.forward(x, idx_out=idx, w_out=weights)
        h = ex.group_mm(x, w_down, all_rows)
        batches.append((h, idx, weights, teacher.forward(h, idx, weights, train=False)[0]))

    def loss():
        return sum((student.forward(h, i, w, train=False)[0].float() - t.float()).square().mean().item()
                   for h, i, w, t in batches) / 2

    losses = [loss()]
    for s in range(steps):
        for h, idx, weights, target in batches:
            out, saved = student.forward(h, idx, weights)
            # d/dout of half the squared error, scaled so that a step does not depend on the batch's size
            student.backward((out.float() - target.float()).mul_(1.0 / tokens).bfloat16(), saved)
        student.step(lr * cfg.E / cfg.K)
        losses.append(loss())
        if verbose:
            print(f"step {s + 1:3d}  mean squared error {losses[-1]:.5f}")
    if layer.status() or ex.status():
        raise RuntimeError("device-side error")
    return losses, student


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--dropout", type=float, default=0.1)
    ap.add_argument("--act", choices=("silu", "situ"), default="silu")
    ap.add_argument("--one-pass", action="store_true")
    a = ap.parse_args()
    got, _ = train(a.steps, a.tokens, a.dropout, a.act, one_pass=a.one_pass)
    print(f"mean squared error {got[0]:.5f} -> {got[-1]:.5f}")
