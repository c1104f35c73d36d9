"""Codes of frames, trained and served: every Gaussian's inputs are the code of
its frame (a row of a table, looked up with dropout) beside features of its own;
two layers whose products run in MXFP4, with dropout between them; the table's
gradient goes with the layers' into an Adam step that clips by their global norm.
Then the same field from 4 bits alone: the table in MXFP4, the layers' weights
with group scales, one row at a time or all at once.

    python examples/frame_codes.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from implicit_attribute_decode_amd.pipeline import (Adam, Dropout, Mx4Linear, embedding, embedding_backward,  # noqa: E402
                                                    mx4_quantize, q4_linear, q4_quantize)

FRAMES, CODE, FEATURES, HIDDEN, OUT = 150, 32, 32, 64, 11


class Field:
    """A table of codes and two layers, with what a training step needs."""

    def __init__(self, p: float = 0.1, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.table = 0.1 * randn(FRAMES, CODE)
        self.hidden = Mx4Linear(randn(HIDDEN, CODE + FEATURES) / math.sqrt(CODE + FEATURES), torch.zeros(HIDDEN, device=device),
                                "relu")
        self.out = Mx4Linear(randn(OUT, HIDDEN) / math.sqrt(HIDDEN), torch.zeros(OUT, device=device))
        self.p, self.seed = p, seed

    def groups(self, lr: float) -> dict:
        return {"table": {"param": self.table, "lr": 5 * lr}, "w0": {"param": self.hidden.weight, "lr": lr},
                "b0": {"param": self.hidden.bias, "lr": lr}, "w1": {"param": self.out.weight, "lr": lr},
                "b1": {"param": self.out.bias, "lr": lr}}

    def drops(self, step: int):
        """The dropouts of a step: one of the codes, one of the hidden layer."""
        return Dropout(self.p, self.seed, 2 * step), Dropout(self.p, self.seed, 2 * step + 1)

    def forward(self, frame, features, step: int) -> dict:
        """frame [n] (-1: no frame, a code of zeros), features [n, FEATURES] bfloat16."""
        codes, hidden = self.drops(step)
        x = torch.empty((len(frame), CODE + FEATURES), dtype=torch.bfloat16, device=features.device)
        embedding(self.table, frame, dropout=codes, out=x[:, :CODE])
        x[:, CODE:] = features
        h = self.hidden(x)
        d = hidden(h)
        return {"x": x, "h": h, "d": d, "y": self.out(d)}

    def backward(self, acts: dict, frame, dy, step: int) -> dict:
        """Gradients of every group; dx, that of the layers' input."""
        codes, hidden = self.drops(step)
        g1 = self.out.backward(acts["d"], dy)
        g0 = self.hidden.backward(acts["x"], hidden.backward(g1["x"]), acts["h"])
        return {"table": embedding_backward(g0["x"][:, :CODE], frame, FRAMES, dropout=codes), "w0": g0["weight"],
                "b0": g0["bias"], "w1": g1["weight"], "b1": g1["bias"], "dx": g0["x"]}

    def update(self):
        self.hidden.update()
        self.out.update()

    def serving(self) -> "Served":
        return Served(self)


class Served:
    """A trained field in 4 bits: its codes in MXFP4, its layers' weights with group scales."""

    def __init__(self, f: Field):
        self.table = mx4_quantize(f.table)
        self.w0, self.b0 = q4_quantize(f.hidden.weight, 32), f.hidden.bias
        self.w1, self.b1 = q4_quantize(f.out.weight, 64), f.out.bias

    def __call__(self, frame, features):
        x = torch.cat([embedding(self.table, frame, dtype=features.dtype), features], 1)
        return q4_linear(q4_linear(x, self.w0, self.b0, "relu"), self.w1, self.b1)


def train(steps: int = 60, rows: int = 20_000, seed: int = 0):
    """Fits a smooth function of frame and features; returns (field, frame, features, target, losses)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    frame = torch.randint(-1, FRAMES, (rows,), generator=gen, device="cuda")
    features = torch.randn((rows, FEATURES), generator=gen, device="cuda").to(torch.bfloat16)
    mix = torch.randn((FEATURES, OUT), generator=gen, device="cuda") / math.sqrt(FEATURES)
    target = torch.tanh(features.float() @ mix) + 0.5 * torch.sin(frame.float()[:, None] / 20 + torch.arange(OUT, device="cuda"))
    f = Field(seed=seed)
    opt = Adam(f.groups(2e-3), warmup=5, total=steps)
    losses = []
    for step in range(steps):
        acts = f.forward(frame, features, step)
        err = acts["y"].float() - target
        losses.append(err.square().sum(1).mean())
        grads = f.backward(acts, frame, (err * (2.0 / rows)).to(torch.bfloat16), step)
        opt.step(grads, max_norm=1.0)
        f.update()
    return f, frame, features, target, torch.stack(losses).tolist()


def main():
    f, frame, features, target, losses = train()
    for k in (0, len(losses) // 2, len(losses) - 1):
        print(f"step {k:3d}: loss {losses[k]:.4f}")
    served = f.serving()
    y = served(frame, features)
    print(f"from 4 bits: loss {(y.float() - target).square().sum(1).mean().item():.4f}; "
          f"one row alone: {tuple(served(frame[:1], features[:1]).shape)}")


if __name__ == "__main__":
    main()
