"""A class head trained on a frozen layer's features and answering in 4 bits.

One path through the operators around the convolution layer:

  1. a bf16 3x3 layer (frozen) -> group norm with Mish (trained) -> a class
     score per pixel over many classes;
  2. each training step: the loss of the head (the scores are never stored),
     its gradient to the features and to the head, the gradient through the
     norm, and an Adam update of the head, gamma and beta;
  3. the trained head quantised to 4 bits with group scales, answering for a
     few pixels at a time, beside the bf16 head as a 1x1 layer.

Data and weights are synthetic: the labels are those of a hidden head on the
features, so that there is something to learn.

    python examples/class_head.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_nhwc_implicit_gb300 as cl  # noqa: E402


class Adam:
    """Adam on fp32 copies; `like` receives the rounded parameters."""

    def __init__(self, param, lr):
        self.param, self.master, self.lr, self.t = param, param.float().clone(), lr, 0
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)

    def step(self, grad):
        self.t += 1
        g = grad.float()
        self.m.mul_(0.9).add_(g, alpha=0.1)
        self.v.mul_(0.99).addcmul_(g, g, value=0.01)
        up = (self.m / (1 - 0.9 ** self.t)) / ((self.v / (1 - 0.99 ** self.t)).sqrt() + 1e-8)
        self.master.add_(up, alpha=-self.lr)
        self.param.copy_(self.master)


def main(steps=60, n=8, size=16, c_in=32, c=128, groups=8, classes=1000, rows=4, seed=0, say=print):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    bf16 = torch.bfloat16
    # the frozen layer and its features
    layer = cl.Plan(n, size, size, c_in, c, 3, 3, 1, 1, 1, dtype="bf16")
    x = randn(n, size, size, c_in).to(bf16)
    w = (randn(c, 3, 3, c_in) / (9 * c_in) ** 0.5).to(bf16)
    feat = torch.empty(layer.output_shape, device="cuda", dtype=bf16)
    layer.run(x, w, torch.zeros(c, device="cuda"), feat)
    # the trained part
    norm = cl.GroupNormPlan(n, size, size, c, groups, dtype="bf16", act="mish")
    gamma, beta = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    pixels = n * size * size
    loss_of = cl.ClassLossPlan(pixels, c, classes)
    head = (0.02 * randn(classes, c)).to(bf16)
    z, mean, rstd = torch.empty_like(feat), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    norm.run(feat, gamma, beta, z, mean, rstd)
    target = (z.view(pixels, c).float() @ randn(c, classes)).argmax(dim=1).to(torch.int32)
    target[::17] = -1  # pixels without a label
    loss, lse = torch.empty((), device="cuda"), torch.empty(pixels, device="cuda")
    dz, dfeat, dhead = torch.empty_like(feat), torch.empty_like(feat), torch.empty_like(head)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    adams = [Adam(head, 2e-2), Adam(gamma, 2e-3), Adam(beta, 2e-3)]
    history = []
    for step in range(steps):
        norm.run(feat, gamma, beta, z, mean, rstd)
        loss_of.run(z.view(pixels, c), head, target, loss, lse)
        loss_of.run_backward(z.view(pixels, c), head, target, lse, dz.view(pixels, c), dhead)
        norm.run_backward(feat, gamma, beta, mean, rstd, dz, dfeat, dgamma, dbeta)
        for adam, grad in zip(adams, (dhead, dgamma, dbeta)):
            adam.step(grad)
        history.append(loss.clone())
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {float(loss):.4f}")
    loss_of.check_device_status()
    # the head in 4 bits, a few pixels at a time, beside the bf16 head as a 1x1 layer
    codes, scales = cl.w4_quantize(head, 32)
    small = cl.W4Plan(rows, c, classes, group=32, dtype="bf16")
    packed = small.pack(codes)
    wide = cl.Plan(1, 1, pixels, c, classes, 1, 1, dtype="bf16")
    scores = torch.empty(wide.output_shape, device="cuda", dtype=bf16)
    wide.run(z.view(1, 1, pixels, c), head.view(classes, 1, 1, c), None, scores)
    answers = torch.empty(pixels, classes, device="cuda", dtype=bf16)
    for i in range(0, pixels, rows):
        small.run(z.view(pixels, c)[i:i + rows], packed, scales, None, answers[i:i + rows])
    labelled = target >= 0
    right = [(s.float().argmax(dim=1)[labelled] == target[labelled]).float().mean() for s in (scores.view(pixels, classes), answers)]
    say(f"labelled pixels answered right: bf16 head {float(right[0]):.3f}, 4-bit head {float(right[1]):.3f}")
    return {"losses": [float(v) for v in history], "right_bf16": float(right[0]), "right_w4": float(right[1])}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    main(steps=ap.parse_args().steps)
