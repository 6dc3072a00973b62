"""Trains one deformable block -- convolution, group norm, activation -- to follow
another one's outputs on synthetic images, on one MI355X.

Everything but the loss runs in libdeft.so: the layer's and the norm's forward
and backward, the gradients' norm with clipping, and AdamW on bf16 weights with
fp32 masters and 8-bit (or 32-bit) states.

    python examples/train_block.py --steps 60 --bits 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from irregular_gather_cnn_amd.layer import DeformConv  # noqa: E402
from irregular_gather_cnn_amd.norm import GroupNormAct  # noqa: E402
from irregular_gather_cnn_amd.optim import AdamW  # noqa: E402

NAMES = ["w", "b", "w_off", "b_off", "gamma", "beta"]


class Block:
    """y = act(group norm(deformable convolution(x))), bf16, [n][c][h][w]."""

    def __init__(self, n, c, h, w, groups, act, device):
        self.conv = DeformConv(n, c, h, w, c, dtype="bf16", training=True, device=device)
        self.norm = GroupNormAct(n, c, h * w, groups, act=act, layout="channels_first", dtype="bf16", training=True,
                                 device=device)
        self.c, self.device = c, device

    def init(self, gen):
        """fp32 values of the parameters; the biases, an 18-element one among them, are the small tensors."""
        def rand(*shape, scale):
            return torch.randn(shape, generator=gen, device=self.device) * scale
        c, oc = self.c, self.conv.oc
        k = (9 * c) ** -0.5
        return dict(w=rand(c, c, 3, 3, scale=k * 2 ** 0.5), b=rand(c, scale=0.1), w_off=rand(oc, c, 3, 3, scale=0.3 * k),
                    b_off=rand(oc, scale=0.3), gamma=1 + rand(c, scale=0.2), beta=rand(c, scale=0.2))

    def forward(self, x, p):
        z, offsets = self.conv.forward(x, p["w_off"], p["b_off"], p["w"], p["b"])
        y, mean, rstd = self.norm.forward(z, p["gamma"], p["beta"])
        return y, (z, offsets, mean, rstd)

    def backward(self, x, p, saved, dy, grads):
        """Writes the gradients of all parameters to grads."""
        z, offsets, mean, rstd = saved
        dz = self.norm.backward(z, p["gamma"], p["beta"], mean, rstd, dy,
                                out=dict(dx=torch.empty_like(z), dgamma=grads["gamma"], dbeta=grads["beta"]))["dx"]
        self.conv.backward(x, p["w_off"], p["w"], offsets, dz,
                           out=dict(dx=torch.empty_like(x), dw_off=grads["w_off"], db_off=grads["b_off"],
                                    dw=grads["w"], db=grads["b"]))


def train(steps=60, bits=8, lr=2e-3, n=4, c=64, hw=28, groups=8, act="silu", seed=0, log=print):
    """The losses of all steps."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device).manual_seed(seed)
    block = Block(n, c, hw, hw, groups, act, device)
    teacher = {k: v.bfloat16() for k, v in block.init(gen).items()}
    masters = block.init(gen)
    params = {k: v.bfloat16() for k, v in masters.items()}
    grads = {k: torch.zeros_like(v) for k, v in params.items()}
    decay = [0.01 if k in ("w", "w_off") else 0.0 for k in NAMES]
    opt = AdamW([params[k] for k in NAMES], [grads[k] for k in NAMES], lr=lr, betas=(0.9, 0.99), weight_decay=decay,
                bits=bits, masters=[masters[k] for k in NAMES], seed=seed)
    images = [torch.randn((n, c, hw, hw), generator=gen, device=device).bfloat16() for _ in range(4)]
    targets = [block.forward(x, teacher)[0].float() for x in images]
    losses = []
    for step in range(steps):
        x, target = images[step % 4], targets[step % 4]
        y, saved = block.forward(x, params)
        diff = y.float() - target
        losses.append((diff * diff).mean())
        block.backward(x, params, saved, (diff * (2.0 / diff.numel())).bfloat16(), grads)
        control = opt.grad_norm(max_norm=0.1)
        opt.step(control=control)
        if step % 10 == 0 or step == steps - 1:
            log("step %3d  loss %.4f  gradient norm %.4f" % (step, losses[-1].item(), control[0].item()))
    return torch.stack(losses).cpu().tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--lr", type=float, default=2e-3)
    args = ap.parse_args()
    train(args.steps, args.bits, args.lr)
