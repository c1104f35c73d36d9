"""Training and storing in 4 bits: a deformation MLP (192 -> 256 -> 256 -> 58,
the HexPlane decoder's widths) whose products and gradients run in MXFP4,
updated by an Adam step that clips by the global gradient norm, then a hash
table stored in 4 bits and read back into its decoder.

    python examples/mx4_training.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from implicit_attribute_decode_amd import scenes as S  # noqa: E402
from implicit_attribute_decode_amd.pipeline import Adam, Decoder, Mx4Linear, mx4_quantize  # noqa: E402

WIDTHS = (192, 256, 256, 58)


def layers(gen, device="cuda"):
    out = []
    for k, (i, o) in enumerate(zip(WIDTHS[:-1], WIDTHS[1:])):
        w = torch.randn((o, i), generator=gen, device=device) * math.sqrt(2.0 / i)
        out.append(Mx4Linear(w, torch.zeros(o, device=device), "relu" if k + 2 < len(WIDTHS) else "none"))
    return out


def train(steps: int = 80, rows: int = 20_000, max_norm: float = 0.5, seed: int = 0):
    """Fits a smooth target; returns (layers, losses, gradient norms, clip factors).

    Activations and their gradients are bfloat16 (half precision would lose
    the small ones), master weights, moments and weight gradients float32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, WIDTHS[0]), generator=gen, device="cuda").to(torch.bfloat16)
    mix = torch.randn((WIDTHS[0], WIDTHS[-1]), generator=gen, device="cuda") / math.sqrt(WIDTHS[0])
    target = torch.tanh(x.float() @ mix)
    net = layers(gen)
    groups = {}
    for k, layer in enumerate(net):
        groups[f"w{k}"] = {"param": layer.weight, "lr": 2e-3}
        groups[f"b{k}"] = {"param": layer.bias, "lr": 2e-3}
    opt = Adam(groups, warmup=5, total=steps)
    losses, stats = [], []
    for _ in range(steps):
        acts = [x]
        for layer in net:
            acts.append(layer(acts[-1]))
        err = acts[-1].float() - target
        losses.append(err.square().sum(1).mean())
        dy = (err * (2.0 / rows)).to(torch.bfloat16)
        grads = {}
        for k in reversed(range(len(net))):
            g = net[k].backward(acts[k], dy, acts[k + 1], want_x=k > 0)
            grads[f"w{k}"], grads[f"b{k}"], dy = g["weight"], g["bias"], g["x"]
        stats.append(opt.step(grads, max_norm=max_norm))
        for layer in net:
            layer.update()  # the masters' new values in 4 bits
    stats = torch.stack(stats)
    return net, torch.stack(losses).tolist(), stats[:, 0].tolist(), stats[:, 1].tolist()


def store_tables(decoder: Decoder):
    """The decoder's hash tables in MXFP4 (one row per level) and back into the
    decoder; returns (bytes before, bytes after)."""
    tables = decoder._tables
    flat = tables.view(tables.shape[0], -1)
    packed = mx4_quantize(flat)
    packed.dequantize(out=flat)
    decoder.update_params()
    return flat.numel() * flat.element_size(), packed.codes.numel() + packed.scales.numel()


def main():
    net, losses, norms, factors = train()
    for k in (0, 1, len(losses) // 2, len(losses) - 1):
        print(f"step {k:3d}: loss {losses[k]:.4f}, gradient norm {norms[k]:.4f}, clip factor {factors[k]:.4f}")
    full = sum(4 * layer.weight.numel() for layer in net)
    four = sum(layer.w.codes.numel() + layer.w.scales.numel() for layer in net)
    one = torch.randn((1, WIDTHS[0]), device="cuda").to(torch.bfloat16)
    for layer in net:
        one = layer(one)
    print(f"weights: {full} bytes in float32, {four} in MXFP4; one row served: {tuple(one.shape)}")

    decoder = Decoder(S.single_decoder())
    xyzt = torch.rand((1000, 4), device="cuda")
    before = decoder.decode_xyzt(xyzt)["colors"].clone()
    a, b = store_tables(decoder)
    moved = (decoder.decode_xyzt(xyzt)["colors"] - before).abs().max().item()
    print(f"hash tables: {a} bytes in float16, {b} in MXFP4; colours of 1,000 Gaussians move by at most {moved:.2e}")


if __name__ == "__main__":
    main()
