"""Layer norm and its backward pass on the GPU against the 64-bit forms."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import layers_ref as ref
from tests.test_gpu_linear import BF, FP16, FP32, gen, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


SIZES = [(1, 1), (1, 2), (3, 7), (5, 32), (700, 64), (2, 255), (3, 256), (9, 257), (301, 520), (4, 1000), (130, 1024), (7, 1999),
         (3, 2048), (2, 4104), (1, 7168), (400, 7168), (3, 7169), (5, 8192), (2, 8200), (3, 16385), (1, 65536)]
TYPES = [(BF, BF), (FP16, FP16), (FP32, FP32), (FP32, BF), (FP32, FP16)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("affine,pad,offset", [("fp32", 0, 0), ("none", 3, 0), ("same", 8, 8), ("weight", 1, 1)])
def test_forward_and_backward(T, H, types, affine, pad, offset):
    xt, ot = types
    g = gen(T * 13 + H)
    x = rows(g, T, H, xt, pad, offset)
    w = b = None
    if affine != "none":
        pt = xt if affine == "same" else FP32
        w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(pt)
        b = None if affine == "weight" else torch.randn(H, generator=g, device="cuda").to(pt)
    out, stats = ops.mhc_layer_norm(x, w, b, 1e-5, dtype=ot)
    want, ws, e, es = ref.layer_norm(x, w, b, 1e-5)
    assert out.dtype == ot
    ref.within(out, want, e)
    assert ((stats.double() - ws).abs() <= es).all()

    d = rows(g, T, H, ot, pad, offset, 0.1)
    r = rows(g, T, H, xt, pad) if affine in ("same", "none") else None
    got = ops.mhc_layer_norm_backward(d, x, stats, w, bias=b is not None, d_residual=r)
    bw = ref.layer_norm_backward(d, x, stats, w, r)
    assert got.d_x.dtype == xt and (got.d_w is None) == (w is None) and (got.d_b is None) == (b is None)
    for k in ("d_x", "d_w", "d_b"):
        if getattr(got, k) is not None:
            ref.within(getattr(got, k), *bw[k])


def test_rows_far_off_zero():
    """A mean a thousand times the spread: the centred squares do not cancel."""
    g = gen(1)
    x = 1000 + torch.randn(5, 3000, generator=g, device="cuda")
    out, stats = ops.mhc_layer_norm(x)
    want, ws, e, es = ref.layer_norm(x, None, None, 1e-5)
    ref.within(out, want, e)
    assert float((stats.double() - ws).abs()[:, 1].max()) < 1e-3


def test_constant_rows_and_values_that_are_not_finite():
    x = torch.full((4, 200), 3.0, device="cuda")
    x[1, 7] = float("inf")
    x[2, 199] = float("nan")
    out, stats = ops.mhc_layer_norm(x, None, torch.ones(200, device="cuda"))
    assert out[0].eq(1).all() and out[3].eq(1).all()
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert float(stats[0, 0]) == 3.0


def test_no_tokens_and_given_buffers():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    out, stats = ops.mhc_layer_norm(x, w, w)
    assert out.shape == (0, 64) and stats.shape == (0, 2)
    d = ops.mhc_layer_norm_backward(x, x, stats, w)
    assert not d.d_w.any() and not d.d_b.any()
    g = gen(2)
    x, dy, r = (rows(g, 77, 520, BF) for _ in range(3))
    o, s = torch.empty(77, 520, device="cuda", dtype=BF), torch.empty(77, 2, device="cuda")
    out, stats = ops.mhc_layer_norm(x, out=o, stats=s)
    assert out.data_ptr() == o.data_ptr() and stats.data_ptr() == s.data_ptr()
    want = ops.mhc_layer_norm_backward(dy, x, stats, w.new_ones(520), d_residual=r)
    space = torch.empty(ops.layer_norm_backward_workspace_bytes(77, 520), dtype=torch.uint8, device="cuda")
    got = ops.mhc_layer_norm_backward(dy, x, stats, w.new_ones(520), d_residual=r, d_x=r, workspace=space)
    assert got.d_x.data_ptr() == r.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T,H", [(1, 7168), (300, 520), (2000, 257)])
def test_the_same_run_to_run_in_a_graph_and_on_another_stream(T, H):
    g = gen(T)
    x, d, r = (rows(g, T, H, BF) for _ in range(3))
    w, b = torch.randn(H, generator=g, device="cuda"), torch.randn(H, generator=g, device="cuda")
    call = lambda **k: (lambda f: (*f, *ops.mhc_layer_norm_backward(d, x, f[1], w, d_residual=r, **k)))(ops.mhc_layer_norm(x, w, b, **k))  # noqa: E731
    first = call()
    assert all(torch.equal(p, q) for p, q in zip(first, call()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = call(stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, held))


@pytest.mark.parametrize("T,H,types,pad", [(1300, 520, (BF, BF), 8), (2500, 2048, (FP16, FP16), 0), (2000, 4096, (BF, BF), 0),
                                           (1500, 1544, (FP32, FP32), 8), (1400, 7168, (FP32, BF), 0), (1300, 8192, (FP32, FP32), 0),
                                           (1250, 7168, (BF, BF), 16), (5000, 264, (FP16, FP16), 0), (4000, 64, (BF, BF), 0),
                                           (1300, 1999, (BF, BF), 3), (1600, 1102, (FP32, FP32), 0), (1400, 1999, (FP32, FP16), 1),
                                           (1300, 7167, (FP16, FP16), 2), (1250, 8191, (FP32, FP32), 0), (3000, 514, (BF, BF), 1)])
@pytest.mark.parametrize("res", [False, True])
def test_many_rows(T, H, types, pad, res):
    """More rows than are on the way at once, every place of the stages filled several times."""
    xt, ot = types
    g = gen(T + H)
    x, d = rows(g, T, H, xt, pad), rows(g, T, H, ot, pad, 0, 0.1)
    r = rows(g, T, H, xt, pad) if res else None
    w, b = 1 + 0.1 * torch.randn(H, generator=g, device="cuda"), torch.randn(H, generator=g, device="cuda")
    if res:
        b = None
    out, stats = ops.mhc_layer_norm(x, w, b, 1e-5, dtype=ot)
    want, ws, e, es = ref.layer_norm(x, w, b, 1e-5)
    ref.within(out, want, e)
    assert ((stats.double() - ws).abs() <= es).all()
    got = ops.mhc_layer_norm_backward(d, x, stats, w, bias=b is not None, d_residual=r)
    bw = ref.layer_norm_backward(d, x, stats, w, r)
    for k in ("d_x", "d_w", "d_b"):
        if getattr(got, k) is not None:
            ref.within(getattr(got, k), *bw[k])


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
