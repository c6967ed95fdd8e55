#!/usr/bin/env python3
"""Train a small network with the whole optimizer, then serve it in 4 bits.

    python examples/mixed_step.py [--steps 60] [--tokens 1024]

The layer products run in MX4 (mx4.train_linear); the two weight matrices take
Shampoo's direction with Adam's length per block (pipeline), the tensors that
are not matrices take AdamW with 8-bit moments (adamw), and one norm over all
gradients clips both; a step whose norm is not finite changes nothing.
Afterwards the weights are quantised once and single rows go through them.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from inverse_root_preconditioning_amd import adamw as AW  # noqa: E402
from inverse_root_preconditioning_amd import capi  # noqa: E402
from inverse_root_preconditioning_amd import mx4 as MX  # noqa: E402
from inverse_root_preconditioning_amd import pipeline as PL  # noqa: E402


class Net:
    """y = W2 (gain * relu(W1 x)) + bias, rows of x as tokens."""

    def __init__(self, width, hidden, generator):
        def normal(*shape):
            return torch.randn(*shape, generator=generator, device="cuda")
        self.w1 = normal(hidden, width) / width ** 0.5
        self.w2 = normal(width, hidden) / hidden ** 0.5
        self.gain = torch.ones(hidden, device="cuda")
        self.bias = torch.zeros(width, device="cuda")
        for p in self.matrices + self.vectors:
            p.requires_grad_()

    @property
    def matrices(self):
        return [self.w1, self.w2]

    @property
    def vectors(self):
        return [self.gain, self.bias]

    def forward(self, x):
        h = MX.train_linear(x, self.w1).relu() * self.gain
        return MX.train_linear(h, self.w2) + self.bias

    def serve(self, x, w1, w2):
        h = MX.linear(x, w1).relu() * self.gain.detach()
        return MX.linear(h, w2) + self.bias.detach()


def train(steps=60, tokens=1024, width=256, hidden=512, block=128, lr=2e-2, seed=0, log=print):
    """Returns the losses of all steps and the largest difference between the
    served and the trained network's outputs, relative to their size."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, net = Net(width, hidden, gen), Net(width, hidden, gen)

    # Shampoo with grafting on the matrices: fixed gradient and update buffers, blocked once.
    grads = [torch.zeros_like(p) for p in net.matrices]
    update = [torch.zeros_like(p) for p in net.matrices]
    moment = [[torch.zeros_like(p) for p in net.matrices] for _ in range(2)]
    tables = [PL.BlockTable.from_layers(t, block)
              for t in (grads, update, [p.detach() for p in net.matrices], moment[0], moment[1])]
    shampoo = PL.ShampooBlocks(PL.StepConfig(B=block, variant=capi.NDB_Z, iters=8, eps_rel=1e-6, update_every=5),
                               tables[0].n)
    shampoo.set_start_vectors(torch.randn(2 * tables[0].n, block, 32, generator=gen, device="cuda"))
    # AdamW with 8-bit moments on the rest.
    vgrads = [torch.zeros_like(p) for p in net.vectors]
    vtable = AW.TensorTable(vgrads)
    adamw = AW.AdamW([p.detach() for p in net.vectors], lr=lr, betas=(0.9, 0.95), weight_decay=0.0, state="mx8")
    everything = AW.TensorTable(grads + vgrads)

    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, generator=gen, device="cuda")
        with torch.no_grad():
            target = teacher.forward(x)
        loss = (net.forward(x) - target).square().mean()
        params = net.matrices + net.vectors
        for buf, g in zip(grads + vgrads, torch.autograd.grad(loss, params)):
            buf.copy_(g)
        clip = AW.grad_norm(everything, 1.0)[1:]
        losses.append(loss.detach())
        adamw.step(vtable, grad_scale=clip)      # by itself changes nothing where clip is not finite
        if not torch.isfinite(clip):             # the factor averages would keep a NaN for good
            log(f"step {step:4d}  skipped: the gradients' norm is not finite")
            continue
        torch._foreach_mul_(grads, clip[0])
        shampoo.step(tables[0], tables[1])
        PL.graft_update(*tables, 0.5 * lr, 0.9, 0.95, 1e-8, step)
        if step % 10 == 1 or step == steps:
            log(f"step {step:4d}  loss {losses[-1].item():.4f}  clip {clip.item():.3f}")

    w1, w2 = MX.quantize(net.w1.detach()), MX.quantize(net.w2.detach())
    x = torch.randn(8, width, generator=gen, device="cuda")
    served = torch.cat([net.serve(row[None], w1, w2) for row in x])
    with torch.no_grad():
        whole = net.forward(x)
    off = ((served - whole).norm() / whole.norm()).item()
    log(f"served one row at a time in 4 bits: relative difference {off:.2e}")
    return [v.item() for v in losses], off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    train(a.steps, a.tokens)
