"""Layer norm, projections, their gradients and the orthogonalised update as a
model uses them together: the example's gradients against the same model's in
64 bits, one token against its place in the batch, calls at once on two
streams, and the calls that are refused."""
import os
import sys

import pytest
import torch

from manifold_constrained_hyper_gb300 import ops, synth
from tests.mhc_testlib import dev_bf16, dev_f32

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def _act64(z, act):
    f = torch.nn.functional
    return {"relu2": lambda: f.relu(z) ** 2, "silu": lambda: f.silu(z), "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[act]()


def _model64(model, x):
    """The stack in 64 bits with the weights as the products read them, and its parameters."""
    params = []
    r = x.double().requires_grad_(True)
    first = r
    for layer in model.layers:
        p = {k: v.double().requires_grad_(True) for k, v in
             {**layer.p, "w1": layer.w1, "w2": layer.w2}.items()}
        params.append(p)
        h = torch.nn.functional.layer_norm(r, r.shape[-1:], p["w"], p["b"], 1e-5)
        r = _act64(h @ p["w1"].t() + p["b1"], layer.act) @ p["w2"].t() + p["b2"] + r
    return first, r, params


@pytest.mark.parametrize("tokens,hidden,wide,act,dtype", [(300, 192, 520, "gelu_tanh", BF), (33, 128, 384, "silu", FP16),
                                                          (520, 200, 264, "relu2", FP16), (1, 256, 1024, "gelu_tanh", BF)])
def test_the_gradients_of_a_stack(tokens, hidden, wide, act, dtype):
    import norm_mlp as ex
    layers = 2
    model = ex.Stack(hidden, layers, wide, act, seed=tokens, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(tokens, hidden, generator=g, device="cuda")
    target = torch.randn(tokens, hidden, generator=g, device="cuda")
    loss, d_x = model.gradients(x, target)
    first, out, params = _model64(model, x)
    want = 0.5 * (out - target.double()).square().sum(1).mean()
    want.backward()
    # a layer rounds h, z, a, d, d_z and d_h to 16 bits, each by at most half a step of itself; what
    # they are read by passes relative errors on by at most about two (the activations' slopes, the norm)
    eps = torch.finfo(dtype).eps / 2
    bound = 2 * 6 * layers * eps
    want = float(want.detach())
    assert abs(float(loss) - want) < bound * want

    def near(got, exact, name):
        off = float((got.double() - exact).norm() / exact.norm())
        assert off < bound, (name, off, bound)

    near(d_x, first.grad, "d_x")
    for i, (layer, p) in enumerate(zip(model.layers, params)):
        for k, v in layer.grad.items():
            near(v, p[k].grad, (i, k))


def test_a_run_of_training_and_serving():
    import norm_mlp as ex
    model = ex.Stack(256, 2)
    x, target = ex.data(512, 256)
    for _ in range(3):
        model.step(x, target)
    for layer in model.layers:
        for p in layer.p.values():
            assert torch.isfinite(p).all()
    # the same token by itself and in a batch: sums in another order, rounded to bf16 twice a layer
    one, all_ = model.forward(x[5:6]), model.forward(x)[5:6]
    assert float((one - all_).norm() / all_.norm()) < 2 * 2 * 2 * 2.0 ** -8
    assert ops.mhc_get_device_status() == 0


def test_calls_at_once_on_two_streams():
    """Two updates whose products share the SMs, and projections beside them: the same as one after another."""
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = (torch.randn(700, 1000, generator=g, device="cuda") for _ in range(2))
    x, w = (torch.randn(n, 512, generator=g, device="cuda").to(BF) for n in (300, 640))
    want = [ops.mhc_orthogonalize(a), ops.mhc_orthogonalize(b), ops.mhc_linear(x, w), ops.mhc_linear_dw(x, x)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s):
            one = [ops.mhc_orthogonalize(a), ops.mhc_linear(x, w)]
        with torch.cuda.stream(t):
            two = [ops.mhc_orthogonalize(b), ops.mhc_linear_dw(x, x)]
        torch.cuda.synchronize()
        assert ops.mhc_get_device_status() == 0
        assert torch.equal(one[0], want[0]) and torch.equal(two[0], want[1])
        assert torch.equal(one[1], want[2]) and torch.equal(two[1], want[3])


def test_calls_at_once_beside_boundaries_of_small_clusters():
    """Clusters that share SMs: boundaries of a few tokens on two streams, projections of a few tokens and small updates on two
    others. None holds what another's cluster waits for, and all come out as alone."""
    d = synth.make_inputs(4, 256, seed=7)
    dev = {k: dev_bf16(d[k]) if k in ("x", "residual") else dev_f32(d[k])
           for k in ("x", "residual", "post", "comb", "scale", "base", "norm_w", "pre_lag", "fn")}
    weight = ops.mhc_prepare_weight(dev["fn"])
    g = torch.Generator(device="cuda").manual_seed(9)
    a = torch.randn(4, 128, 500, generator=g, device="cuda")
    x, w = (torch.randn(n, 2048, generator=g, device="cuda").to(BF) for n in (64, 1024))

    def boundary():
        return ops.mhc_boundary_fused(dev["x"], dev["residual"], dev["post"], dev["comb"], weight, dev["scale"], dev["base"],
                                      dev["norm_w"], dev["pre_lag"])

    def flat(r):
        return list(r) if isinstance(r, tuple) else [r]
    calls = [boundary, boundary, lambda: ops.mhc_orthogonalize(a), lambda: ops.mhc_linear(x, w, dtype=torch.float32)]
    want = [[t.clone() for t in flat(c())] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(4):
        got = [None] * len(calls)
        for _ in range(8):
            for i, (c, s) in enumerate(zip(calls, streams)):
                with torch.cuda.stream(s):
                    got[i] = flat(c())
        torch.cuda.synchronize()
        assert ops.mhc_get_device_status() == 0
        for one, two in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(one, two))
        # one after another on one stream too
        for c, two in zip(calls, want):
            assert all(torch.equal(p, q) for p, q in zip(flat(c()), two))


def test_two_graphs_that_share_a_workspace():
    """Captured updates of two shapes on one workspace, replayed one after another: nothing of one call is
    read by the next."""
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = torch.randn(300, 700, generator=g, device="cuda"), torch.randn(600, 260, generator=g, device="cuda")
    want = [ops.mhc_orthogonalize(a), ops.mhc_orthogonalize(b)]
    n = max(ops.orthogonalize_workspace_bytes(1, *t.shape) for t in (a, b))
    space = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    held, graphs = [], []
    for t in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(ops.mhc_orthogonalize(t, workspace=space))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
    assert ops.mhc_get_device_status() == 0


def test_a_backward_pass_captured_while_eager_tensors_live():
    """The gradients' calls in a graph, with eager results of the same leaves kept."""
    x = torch.randn(130, 264, device="cuda").to(BF)
    w = torch.randn(96, 264, device="cuda").to(BF)
    d = torch.randn(130, 96, device="cuda").to(BF)
    kept = (ops.mhc_linear_dx(d, w), *ops.mhc_linear_dw(d, x, bias=True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (ops.mhc_linear_dx(d, w), *ops.mhc_linear_dw(d, x, bias=True))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, held))


def test_refusals():
    x = torch.randn(8, 64, device="cuda").to(BF)
    w = torch.randn(32, 64, device="cuda").to(BF)
    d = torch.randn(8, 32, device="cuda").to(BF)
    f = torch.randn(8, 64, device="cuda")
    for call, what in ((lambda: ops.mhc_linear(f, w), "bfloat16 or float16"),
                       (lambda: ops.mhc_linear(x, w.to(FP16)), "w must be"),
                       (lambda: ops.mhc_linear(x, w[:, :60]), "w must be"),
                       (lambda: ops.mhc_linear(x, w, torch.randn(31, device="cuda")), "bias must be"),
                       (lambda: ops.mhc_linear(x, w, torch.randn(32, device="cuda").to(FP16)), "bias must be"),
                       (lambda: ops.mhc_linear(x, w, None, d.to(FP16)), "out must be"),
                       (lambda: ops.mhc_linear(x, w, None, x), "residual must be"),
                       (lambda: ops.mhc_linear(x, w, dtype=FP16), "out must be"),
                       (lambda: ops.mhc_linear(x, w, out=torch.empty(32, 8, device="cuda", dtype=BF).t()), "out must be"),
                       (lambda: ops.mhc_linear(x.t(), w), "contiguous rows"),
                       (lambda: ops.mhc_linear(x, w, z=torch.empty(8, 32, device="cuda")), "z must be"),
                       (lambda: ops.mhc_linear_dx(d, w, act="silu"), "z is needed"),
                       (lambda: ops.mhc_linear_dx(d, w, x), "no use"),
                       (lambda: ops.mhc_linear_dx(d, w[:31]), "w must be"),
                       (lambda: ops.mhc_linear_dx(d, w, d, "silu"), "z must be"),
                       (lambda: ops.mhc_linear_dw(d, x[:7]), "x must be"),
                       (lambda: ops.mhc_linear_dw(d, x, d_w=torch.empty(32, 63, device="cuda")), "d_w must be"),
                       (lambda: ops.mhc_linear_dw(d, x, d_bias=torch.empty(32, device="cuda", dtype=BF)), "d_bias must be"),
                       (lambda: ops.mhc_layer_norm(x, dtype=torch.float32), "out must be"),
                       (lambda: ops.mhc_layer_norm(x, torch.randn(63, device="cuda")), "w must be"),
                       (lambda: ops.mhc_layer_norm(x.int()), "x must be"),
                       (lambda: ops.mhc_layer_norm_backward(x, x, torch.empty(8, 2, device="cuda", dtype=BF)), "stats must be"),
                       (lambda: ops.mhc_layer_norm_backward(f, x, torch.empty(8, 2, device="cuda")), "d_out must be"),
                       (lambda: ops.mhc_layer_norm_backward(x, x, torch.empty(8, 2, device="cuda"), d_residual=f), "d_residual must be"),
                       (lambda: ops.mhc_orthogonalize(x[0]), "2-D or 3-D"),
                       (lambda: ops.mhc_orthogonalize(x.t()), "rows must be contiguous"),
                       (lambda: ops.mhc_orthogonalize(x, dtype=torch.float32), "bfloat16 or float16"),
                       (lambda: ops.mhc_orthogonalize(x.int()), "g must be"),
                       (lambda: ops.mhc_linear(x, w, workspace=torch.empty(8, dtype=torch.uint8)), "workspace must be")):
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: ops.mhc_orthogonalize(x, 0), lambda: ops.mhc_orthogonalize(x, coeffs=(float("nan"), 0, 0)),
                 lambda: ops.mhc_layer_norm(x, eps=-1.0), lambda: ops.mhc_linear(torch.empty(8, 0, device="cuda", dtype=BF), torch.empty(4, 0, device="cuda", dtype=BF))):
        with pytest.raises(ops.MhcError):
            call()
    # nothing records a history
    leaf = w.clone().requires_grad_(True)
    with pytest.raises(ValueError, match="requires grad"):
        ops.mhc_linear(x, leaf)
    with pytest.raises(ValueError, match="requires grad"):
        ops.mhc_orthogonalize(leaf)
    with torch.no_grad():
        assert torch.equal(ops.mhc_linear(x, leaf), ops.mhc_linear(x, w))


def test_more_than_2_to_31_elements():
    """Offsets past 32 bits: the last rows of outputs of 2.3e9 elements, and of inputs of as many."""
    from tests import layers_ref as ref
    T, K, N = 280000, 64, 8200
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF)
    w = torch.randn(N, K, generator=g, device="cuda").to(BF)
    out = ops.mhc_linear(x, w)
    assert out.numel() > 1 << 31
    at = torch.tensor([0, 1, T // 2, T - 257, T - 1], device="cuda")
    want, _, e, _ = ref.linear(x[at], w, None, None, "none")
    ref.within(out[at], want, e)
    # read again, a row of 8200 a row of the summed axis and of the output
    d_x = ops.mhc_linear_dx(out, w)
    want, e = ref.linear_dx(out[at], w, None, "none")
    ref.within(d_x[at], want, e)
    d_w, d_b = ops.mhc_linear_dw(out, x, bias=True)
    cols = [0, N - 1]
    want = out[:, cols].double().t() @ x.double()
    # one chain of 512 products of a piece and the pieces' sums: 2^-21 of the sizes
    size = out[:, cols].double().abs().t() @ x.double().abs()
    assert ((d_w[cols].double() - want).abs() <= 2.0 ** -20 * size).all()
    want = out[:, cols].double().sum(0)
    assert ((d_b[cols].double() - want).abs() <= T * ref.U * out[:, cols].double().abs().sum(0)).all()
    n, stats = ops.mhc_layer_norm(out)
    want, _, e, _ = ref.layer_norm(out[at], None, None, 1e-5)
    ref.within(n[at], want, e)
    del d_x
    d = ops.mhc_layer_norm_backward(n, out, stats, None, bias=False).d_x
    ref.within(d[at], *ref.layer_norm_backward(n[at], out[at], stats[at], None, None)["d_x"])
    assert ops.mhc_get_device_status() == 0
