"""Trains a block of two pointwise convolutions in 8 bits around a group norm with its
activation to follow another one's outputs, on one MI355X.

Everything but the loss runs in libdeft.so: both layers' products and gradients,
the norm, the gradients' norm with clipping over all tensors, Muon on the two
matrices and AdamW on the vectors, bf16 with fp32 masters.  The matrices' codes are
made anew after each step.

    python examples/train_pointwise.py --steps 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from irregular_gather_cnn_amd.norm import GroupNormAct  # noqa: E402
from irregular_gather_cnn_amd.optim import AdamW, GradNorm, Muon  # noqa: E402
from irregular_gather_cnn_amd.pointwise import Pointwise8  # noqa: E402

MATRICES, VECTORS = ["w1", "w2"], ["b1", "b2", "gamma", "beta"]


class Block:
    """y = w2 act(group norm(w1 x + b1)) + b2 over each position of x, bf16."""

    def __init__(self, n, c, hidden, s, groups, act, layout, device):
        self.first = Pointwise8(n, c, s, hidden, layout=layout, training=True, device=device)
        self.second = Pointwise8(n, hidden, s, c, layout=layout, training=True, device=device)
        self.norm = GroupNormAct(n, hidden, s, groups, act=act, layout=layout, training=True, device=device)
        self.c, self.hidden, self.device = c, hidden, device

    def init(self, gen):
        """fp32 values of the parameters."""
        def rand(*shape, scale):
            return torch.randn(shape, generator=gen, device=self.device) * scale
        c, h = self.c, self.hidden
        return dict(w1=rand(h, c, scale=(2 / c) ** 0.5), w2=rand(c, h, scale=h ** -0.5), b1=rand(h, scale=0.1),
                    b2=rand(c, scale=0.1), gamma=1 + rand(h, scale=0.2), beta=rand(h, scale=0.2))

    def pack(self, p):
        return self.first.pack(p["w1"]), self.second.pack(p["w2"])

    def forward(self, x, p, packed):
        z, saved1 = self.first.forward(x, packed[0], p["b1"])
        a, mean, rstd = self.norm.forward(z, p["gamma"], p["beta"])
        y, saved2 = self.second.forward(a, packed[1], p["b2"])
        return y, (saved1, z, mean, rstd, saved2)

    def backward(self, p, packed, saved, dy, grads):
        """Writes the gradients of all parameters to grads; that of x."""
        saved1, z, mean, rstd, saved2 = saved
        da = self.second.backward(saved2, packed[1], dy, out=dict(dx=torch.empty_like(z), dw=grads["w2"], db=grads["b2"]))["dx"]
        dz = self.norm.backward(z, p["gamma"], p["beta"], mean, rstd, da,
                                out=dict(dx=torch.empty_like(z), dgamma=grads["gamma"], dbeta=grads["beta"]))["dx"]
        return self.first.backward(saved1, packed[0], dz,
                                   out=dict(dx=torch.empty_like(dy), dw=grads["w1"], db=grads["b1"]))["dx"]


def train(steps=60, lr=0.02, n=4, c=64, hidden=256, s=28 * 28, groups=8, act="silu", layout="channels_first", seed=0,
          log=print):
    """The losses of all steps."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    block = Block(n, c, hidden, s, groups, act, layout, device)
    teacher = {k: v.bfloat16() for k, v in block.init(gen).items()}
    masters = block.init(gen)
    params = {k: v.bfloat16() for k, v in masters.items()}
    grads = {k: torch.zeros_like(v) for k, v in params.items()}

    def of(tensors, names):
        return [tensors[k] for k in names]

    muon = Muon(of(params, MATRICES), of(grads, MATRICES), lr=lr, masters=of(masters, MATRICES))
    adam = AdamW(of(params, VECTORS), of(grads, VECTORS), lr=lr / 10, weight_decay=0.0, masters=of(masters, VECTORS))
    norm = GradNorm(of(grads, MATRICES + VECTORS))
    shape = (n, c, s) if layout == "channels_first" else (n, s, c)
    images = [torch.randn(shape, generator=gen, device=device).bfloat16() for _ in range(4)]
    coded = block.pack(teacher)
    targets = [block.forward(x, teacher, coded)[0].float() for x in images]
    losses = []
    for step in range(steps):
        x, target = images[step % 4], targets[step % 4]
        packed = block.pack(params)
        y, saved = block.forward(x, params, packed)
        diff = y.float() - target
        losses.append((diff * diff).mean())
        block.backward(params, packed, saved, (diff * (2.0 / diff.numel())).bfloat16(), grads)
        control = norm(max_norm=1.0)
        muon.step(control=control)
        adam.step(control=control)
        if step % 10 == 0 or step == steps - 1:
            log("step %3d  loss %.4f  gradient norm %.4f" % (step, losses[-1].item(), control[0].item()))
    return torch.stack(losses).cpu().tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--lr", type=float, default=0.02)
    args = ap.parse_args()
    train(args.steps, args.lr)
