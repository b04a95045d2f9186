"""A stack of pre-norm blocks, trained with orthogonalised updates and then
served one token at a time.

Layer l, over a residual stream r [T, H]:

    h = layer_norm(r)                                  mhc_layer_norm
    a = act(h W1^T + b1)                               mhc_linear, z kept
    r = a W2^T + b2 + r                                mhc_linear, the residual in its epilogue

and backward, from the gradient d of r after the layer:

    d_W2, d_b2 = d^T a, sum d                          mhc_linear_dw
    d_z = (d W2) * act'(z)                             mhc_linear_dx
    d_W1, d_b1 = d_z^T h, sum d_z                      mhc_linear_dw
    d_r = layer_norm'(d_z W1) + d                      mhc_linear_dx, mhc_layer_norm_backward

A matrix moves by the orthogonalised sum of its gradients (mhc_orthogonalize),
scaled to its shape; vectors by their gradients.

    python examples/norm_mlp.py [--steps N] [--hidden H] [--layers L] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from manifold_constrained_hyper_gb300 import ops  # noqa: E402


class Layer:
    def __init__(self, hidden: int, wide: int, act: str, g: torch.Generator, dtype):
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.act, self.dtype = act, dtype
        self.p = {"w": 1 + 0.1 * rand(hidden), "b": 0.1 * rand(hidden),
                  "w1": rand(wide, hidden) / hidden ** 0.5, "b1": 0.1 * rand(wide),
                  "w2": rand(hidden, wide) / wide ** 0.5, "b2": 0.1 * rand(hidden)}
        self.momentum = {k: torch.zeros_like(v) for k, v in self.p.items()}
        self.cast()

    def cast(self):
        """The weights as the products read them."""
        self.w1, self.w2 = self.p["w1"].to(self.dtype), self.p["w2"].to(self.dtype)

    def forward(self, r, keep=False):
        p = self.p
        h, stats = ops.mhc_layer_norm(r, p["w"], p["b"], dtype=self.dtype)
        if not keep:
            a = ops.mhc_linear(h, self.w1, p["b1"], act=self.act)
            return ops.mhc_linear(a, self.w2, p["b2"], r)
        a, z = ops.mhc_linear(h, self.w1, p["b1"], act=self.act, keep_z=True)
        self.kept = (r, h, stats, a, z)
        return ops.mhc_linear(a, self.w2, p["b2"], r)

    def backward(self, d):
        """The gradient of r before the layer from that after it; those of the parameters go to self.grad."""
        r, h, stats, a, z = self.kept
        d16 = d.to(self.dtype)
        g = {}
        g["w2"], g["b2"] = ops.mhc_linear_dw(d16, a, bias=True)
        d_z = ops.mhc_linear_dx(d16, self.w2, z, self.act)
        g["w1"], g["b1"] = ops.mhc_linear_dw(d_z, h, bias=True)
        d_h = ops.mhc_linear_dx(d_z, self.w1)
        n = ops.mhc_layer_norm_backward(d_h, r, stats, self.p["w"], d_residual=d)
        g["w"], g["b"] = n.d_w, n.d_b
        self.grad = g
        return n.d_x

    def update(self, lr: float, beta: float = 0.9):
        for k, g in self.grad.items():
            p, m = self.p[k], self.momentum[k]
            m.mul_(beta).add_(g)
            if p.dim() == 2:
                step = ops.mhc_orthogonalize(g + beta * m)
                p.sub_(step.float(), alpha=lr * max(1, p.shape[0] / p.shape[1]) ** 0.5)
            else:
                p.sub_(m, alpha=lr)
        self.cast()


class Stack:
    def __init__(self, hidden: int, layers: int, wide: int | None = None, act: str = "gelu_tanh", seed: int = 0,
                 dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(hidden, wide or 4 * hidden, act, g, dtype) for _ in range(layers)]

    def forward(self, x, keep=False):
        """x [T, H] float32, the residual stream."""
        for layer in self.layers:
            x = layer.forward(x, keep)
        return x

    def gradients(self, x, target):
        """Half a token's squared distance from its target, the mean over tokens, and its gradients."""
        diff = self.forward(x, keep=True) - target
        d = diff / diff.shape[0]
        for layer in reversed(self.layers):
            d = layer.backward(d)
        return 0.5 * diff.square().sum(1).mean(), d

    def step(self, x, target, lr: float = 0.01):
        loss, _ = self.gradients(x, target)
        for layer in self.layers:
            layer.update(lr)
        return loss


def data(tokens: int, hidden: int, seed: int = 1):
    """Inputs, and targets that another stack of the same kind makes of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda")
    return x, Stack(hidden, 2, seed=seed + 100).forward(x)


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--tokens", type=int, default=4096)
    a.add_argument("--hidden", type=int, default=512)
    a.add_argument("--layers", type=int, default=4)
    a = a.parse_args()
    model = Stack(a.hidden, a.layers)
    x, target = data(a.tokens, a.hidden)
    for i in range(a.steps):
        loss = model.step(x, target)
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss.item():.5f}")
    # served a token at a time: the same calls, one row
    one = model.forward(x[:1])
    print(f"one token by itself: {(one - model.forward(x)[:1]).abs().max().item():.4f} from its place in the batch")


if __name__ == "__main__":
    main()
