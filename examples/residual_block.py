"""A gated residual block trained with the library's operators alone.

x -> norm -> 3x3 grouped convolution -> join(gate, scale, residual, next norm) -> 1x1 convolution -> loss,
backwards through all of them, and a Muon step of both convolutions' weights, whose bf16 form the next
forward pass reads.  The task: reproduce a fixed block of the same form (its teacher) on random inputs.

    python examples/residual_block.py --steps 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_gconv_fwd_gb300 as gc  # noqa: E402


class Block:
    """Parameters, their gradients and the optimiser's state of one block of C channels in G groups."""

    def __init__(self, C, G, dev, seed):
        gen = torch.Generator().manual_seed(seed)
        normal = lambda shape, sd: (sd * torch.randn(shape, generator=gen)).to(dev)  # noqa: E731
        self.C, self.G = C, G
        self.w = {"mid": normal((C, C // G, 3, 3), (9 * C / G) ** -0.5), "out": normal((C, C, 1, 1), C ** -0.5)}
        self.groups = {"mid": G, "out": 1}
        self.bf16 = {k: v.to(torch.bfloat16) for k, v in self.w.items()}
        self.momentum = {k: torch.zeros_like(v) for k, v in self.w.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.w.items()}
        ones = lambda: torch.ones(C, device=dev)  # noqa: E731
        self.vec = {"norm": ones(), "weight": ones(), "scale": 0.5 * ones(), "next": ones()}
        self.dvec = {k: torch.empty_like(v) for k, v in self.vec.items()}

    def forward(self, x, gate):
        self.x, self.gate = x, gate
        new = lambda: torch.empty_like(x)  # noqa: E731
        self.u, self.h, self.sum, self.v, y = new(), new(), new(), new(), new()
        gc.gconv_norm_fwd(x, self.vec["norm"], self.u)
        gc.gconv_fwd(self.u, self.bf16["mid"], None, self.h, padding=1, groups=self.G)
        gc.gconv_join_fwd(x, self.h, self.sum, gate=gate, act="silu", weight=self.vec["weight"], scale=self.vec["scale"],
                          next=self.v, next_weight=self.vec["next"])
        gc.gconv_fwd(self.v, self.bf16["out"], None, y)
        return y

    def backward(self, dy):
        """Gradients of the parameters; returns those of x and the gate."""
        new = lambda: torch.empty_like(dy)  # noqa: E731
        dv, dsum, dh, du, dx, dgate = new(), new(), new(), new(), new(), torch.empty_like(self.gate)
        gc.gconv_bwd_data(dy, self.bf16["out"], dv)
        gc.gconv_bwd_weight(self.v, dy, self.grad["out"])
        gc.gconv_join_bwd(self.h, None, dh, gate=self.gate, act="silu", weight=self.vec["weight"], scale=self.vec["scale"],
                          dgate=dgate, dweight=self.dvec["weight"], dscale=self.dvec["scale"], out=self.sum,
                          next_weight=self.vec["next"], dnext=dv, dres=dsum, dnext_weight=self.dvec["next"])
        gc.gconv_bwd_data(dh, self.bf16["mid"], du, padding=1, groups=self.G)
        gc.gconv_bwd_weight(self.u, dh, self.grad["mid"], padding=1, groups=self.G)
        gc.gconv_norm_bwd(self.x, self.vec["norm"], du, dx, self.dvec["norm"], dres=dsum)
        return dx, dgate

    def update(self, lr, vec_lr):
        for k in self.w:
            gc.gconv_muon_step(self.w[k], self.grad[k], self.momentum[k], w_bf16=self.bf16[k], groups=self.groups[k], lr=lr)
        for k, v in self.vec.items():
            v -= vec_lr * self.dvec[k]


def train(steps=60, C=64, G=4, N=8, hw=16, lr=0.1, seed=0, dev="cuda"):
    """Mean squared errors, one a step."""
    teacher, student = Block(C, G, dev, seed + 1), Block(C, G, dev, seed + 2)
    gen = torch.Generator().manual_seed(seed)
    losses = []
    for step in range(steps):
        x, gate = (torch.randn((N, C, hw, hw), generator=gen).to(dev, torch.bfloat16) for _ in range(2))
        diff = student.forward(x, gate).float() - teacher.forward(x, gate).float()
        losses.append(float(diff.square().mean()))
        student.backward((diff / diff.numel() ** 0.5).to(torch.bfloat16))
        student.update(lr * (1.0 - step / steps), 1e-4)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    losses = train(ap.parse_args().steps)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  mean squared error {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  mean squared error {losses[-1]:.4f}")
