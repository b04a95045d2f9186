"""A stack of gated, sandwich-normed residual blocks, trained with its
activations kept in 8 bits, and then served one token at a time.

Layer l, over a residual stream r and the block's input h (both [T, H]):

    y = h Wy^T,  z = h Wz^T                            two projections (torch)
    r, h = block boundary of (y, r) with the gate sigmoid(z)       mhc_block_norm

Between the forward and the backward pass a layer keeps y, r and h as 8-bit
checkpoints, written by the boundary that reads or makes them, the gate z, and
two fp32 numbers a token. The backward pass forms everything else anew:

    d_y, d_r, d_z, d_weights                           mhc_block_norm_backward
    d_Wy = d_y^T h,  d_Wz = d_z^T h                    mhc_ckpt_linear_dw
    d_h = d_y Wy + d_z Wz                              (torch)

    python examples/gated_blocks.py [--format e4m3|int8|none] [--steps N] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from manifold_constrained_hyper_gb300 import ops  # noqa: E402

BLOCK = ops.BlockParams(gate_act="sigmoid")


class Layer:
    def __init__(self, hidden: int, g: torch.Generator):
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.p = {"wy": rand(hidden, hidden) / hidden ** 0.5, "wz": rand(hidden, hidden) / hidden ** 0.5,
                  "post": torch.ones(hidden, device="cuda"), "pre": torch.ones(hidden, device="cuda"),
                  "scale": torch.ones(1, device="cuda")}
        self.grad = {}

    def forward(self, h, r, fmt=None):
        """(r, h) after the layer; with a format, keeps what backward needs in 8 bits."""
        p = self.p
        y, z = h @ p["wy"].to(h.dtype).t(), h @ p["wz"].to(h.dtype).t()
        T, H = y.shape
        y8, r8 = (ops.ckpt_empty(T, H, fmt) for _ in range(2)) if fmt else (None, None)
        r_out, h_out, rstd = ops.mhc_block_norm(y, r, p["post"], p["pre"], z, p["scale"], BLOCK,
                                                ckpt_y=y8, ckpt_residual=r8)
        self.kept = (y8 or y, r8 or r, z, rstd, ops.mhc_ckpt_pack(h, fmt) if fmt else h)
        return r_out, h_out

    def backward(self, d_r, d_h):
        """Gradients of r and h before the layer, from those after it; those of
        the parameters go to self.grad."""
        p = self.p
        y, r, z, rstd, h = self.kept
        d = ops.mhc_block_norm_backward(d_r, d_h, y, r, rstd, p["post"], p["pre"], z, p["scale"], BLOCK)
        if isinstance(h, ops.Checkpoint):
            wy, wz = ops.mhc_ckpt_linear_dw(d.d_y, h), ops.mhc_ckpt_linear_dw(d.d_gate, h)
        else:
            wy, wz = (d.d_y.t() @ h).float(), (d.d_gate.t() @ h).float()
        self.grad = {"wy": wy, "wz": wz, "post": d.d_w_post, "pre": d.d_w_pre, "scale": d.d_res_scale}
        d_h = d.d_y @ p["wy"].to(d_h.dtype) + d.d_gate @ p["wz"].to(d_h.dtype)
        return d.d_residual, d_h

    def kept_bytes(self):
        parts = [t for k in self.kept for t in ((k.codes, k.scales) if isinstance(k, ops.Checkpoint) else (k,))]
        return sum(t.numel() * t.element_size() for t in parts)


class Stack:
    def __init__(self, hidden: int, layers: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(hidden, g) for _ in range(layers)]

    def forward(self, x, fmt=None):
        r, h = x, x
        for layer in self.layers:
            r, h = layer.forward(h, r, fmt)
        return h

    def step(self, x, target, fmt=None, lr=0.02):
        """One step of gradient descent on half a token's squared distance from its target, the mean
        over tokens. Returns half the mean square over tokens and columns before it."""
        h = self.forward(x, fmt)
        diff = h.float() - target.float()
        d_r, d_h = None, (diff / diff.shape[0]).to(h.dtype)
        for layer in reversed(self.layers):
            d_r, d_h = layer.backward(d_r, d_h)
        for layer in self.layers:
            for k, d in layer.grad.items():
                layer.p[k].sub_(d.reshape(layer.p[k].shape), alpha=lr)
        return 0.5 * diff.square().mean()


def data(tokens: int, hidden: int, seed: int = 1):
    """Inputs, and targets that another stack of the same kind makes of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    return x, Stack(hidden, 2, seed=seed + 100).forward(x)


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--format", choices=["e4m3", "int8", "none"], default="e4m3")
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=1024)
    a.add_argument("--layers", type=int, default=4)
    a = a.parse_args()
    fmt = None if a.format == "none" else a.format
    model = Stack(a.hidden, a.layers)
    x, target = data(a.tokens, a.hidden)
    for i in range(a.steps):
        loss = model.step(x, target, fmt)
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss.item():.5f}")
    kept = sum(layer.kept_bytes() for layer in model.layers)
    print(f"kept between the passes: {kept / a.tokens / a.layers / a.hidden:.2f} bytes a token, layer and column")
    # served a token at a time: the same call, one row
    one = model.forward(x[:1])
    print(f"one token by itself: {(one.float() - model.forward(x)[:1].float()).abs().max().item():.4f} from its place in the batch")


if __name__ == "__main__":
    main()
