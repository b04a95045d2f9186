"""The example's training loop: the stack learns, and with its activations in
8 bits it learns what it does with them whole."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build, ops
    build.build()
    ops.load()


def _train(fmt, steps=20, tokens=512, hidden=256, layers=3):
    import gated_blocks as ex
    model = ex.Stack(hidden, layers)
    x, target = ex.data(tokens, hidden)
    return [float(model.step(x, target, fmt)) for _ in range(steps)], model, x


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_training_through_checkpoints(fmt):
    whole, _, _ = _train(None)
    held, model, x = _train(fmt)
    # the first loss comes before any checkpoint is read
    assert held[0] == whole[0]
    assert whole[-1] < whole[0] and held[-1] < held[0]
    # what the 8 bits change of the way down is small beside the way itself
    assert abs(held[-1] - whole[-1]) < 0.1 * (whole[0] - whole[-1])
    # a checkpoint is 1 + 1/32 bytes; y, r and h in it and the gate in bf16, two floats a token
    per = model.layers[0].kept_bytes() / x.numel()
    assert per == 3 * (1 + 1 / 32) + 2 + 8 / x.shape[1]


def test_gradients_of_a_layer_against_torch():
    """The layer by autograd in 64 bits, from the same bf16 inputs: the layer's own roundings (y, z, d_y, d_z
    and d_h to bf16, each half a step, and what they reach) stay below 4 half steps of the largest value."""
    import gated_blocks as ex
    g = torch.Generator(device="cuda").manual_seed(3)
    layer = ex.Layer(128, g)
    for k in ("wy", "wz"):
        layer.p[k] = layer.p[k].bfloat16().float()
    h, r, d_r, d_h = (torch.randn(96, 128, generator=g, device="cuda").bfloat16() for _ in range(4))
    layer.forward(h, r)
    got = dict(zip(("r", "h"), layer.backward(d_r, d_h))) | layer.grad
    t = {"h": h, "r": r, **layer.p}
    t = {k: v.double().requires_grad_() for k, v in t.items()}
    y, z = t["h"] @ t["wy"].t(), t["h"] @ t["wz"].t()
    n = y * (y.square().mean(1, keepdim=True) + 1e-6).rsqrt() * t["post"]
    ro = t["scale"] * t["r"] + torch.sigmoid(z) * n
    out = ro * (ro.square().mean(1, keepdim=True) + 1e-6).rsqrt() * t["pre"]
    ((ro * d_r.double()).sum() + (out * d_h.double()).sum()).backward()
    for k, v in t.items():
        far = (got[k].double() - v.grad).abs().max() / v.grad.abs().max()
        assert far < 4 * 2.0 ** -8, (k, float(far))
