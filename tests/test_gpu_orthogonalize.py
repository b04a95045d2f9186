"""The orthogonalised update on the GPU against its 64-bit form."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import layers_ref as ref
from tests.test_gpu_linear import BF, FP16, FP32, gen

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def momentum(g, shape, dtype, scale=1e-3):
    """A few strong directions over a floor."""
    *B, M, N = shape
    r = min(M, N, 8)
    u = torch.randn(*B, M, r, generator=g, device="cuda") * torch.exp2(-torch.arange(r, device="cuda") / 2)
    return (scale * (u @ torch.randn(*B, r, N, generator=g, device="cuda") + 0.5 * torch.randn(*B, M, N, generator=g, device="cuda"))).to(dtype)


def near(got, want, e):
    off = float(((got.double() - want).abs() / e).max())
    assert off <= 1, off


SHAPES = [(1, 1), (1, 70), (70, 1), (5, 3), (64, 64), (65, 130), (130, 65), (200, 72), (128, 500), (300, 300), (257, 600), (513, 260),
          (3, 40, 72), (6, 128, 500), (2, 260, 129), (17, 8, 8), (512, 128), (128, 513),
          (100, 1024), (1025, 127), (33, 2048), (2049, 128), (129, 129), (200, 16, 96), (40, 300, 100)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,out", [(FP32, BF), (BF, FP16), (FP16, BF)])
def test_against_64_bits(shape, dtype, out):
    g = momentum(gen(sum(shape)), shape, dtype)
    got = ops.mhc_orthogonalize(g, dtype=out)
    assert got.shape == g.shape and got.dtype == out
    want, e = ref.orthogonalize_error(g, 5, MUON, 1e-7, out)
    near(got, want, e)


@pytest.mark.parametrize("shape", [(64, 4096), (4097, 64), (32, 8192), (8190, 32), (31, 8193), (33, 1025), (61, 2049), (128, 1000), (3, 2047, 127),
                                   (40, 60, 500), (30, 700, 60), (50, 32, 129), (20, 128, 520), (7, 20, 33), (9, 63, 64)], ids=str)
@pytest.mark.parametrize("dtype,out", [(FP32, BF), (BF, FP16)])
def test_short_sides_in_stretches(shape, dtype, out):
    """A side of at most 64 or 32 lies in two or four stretches of the other, whole and broken ones; batches of more clusters than
    lie on the GPU at once."""
    g = momentum(gen(sum(shape)), shape, dtype)
    got = ops.mhc_orthogonalize(g, dtype=out)
    want, e = ref.orthogonalize_error(g, 5, MUON, 1e-7, out)
    near(got, want, e)


@pytest.mark.parametrize("shape", [(2048, 2600), (2600, 2056), (2, 2050, 2570)], ids=str)
@pytest.mark.parametrize("steps,out", [(2, BF), (3, FP16), (4, BF), (5, BF)])
def test_two_steps_as_one(shape, steps, out):
    """Large enough for two steps to be one product of X."""
    g = momentum(gen(steps), shape, FP32)
    got = ops.mhc_orthogonalize(g, steps, dtype=out)
    want, e = ref.orthogonalize_error(g, steps, MUON, 1e-7, out)
    near(got, want, e)
    # in the 2-norm what was lost stays below the rounding of the result
    assert float((got.double() - want).norm() / want.norm()) < 1.2 * torch.finfo(out).eps / 2


@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, (2.0, -1.5, 0.5)), (12, (1.875, -1.25, 0.375)), (3, (1.5, -0.5, 0.0))])
def test_other_steps_and_coefficients(steps, coeffs):
    g = momentum(gen(steps), (96, 200), FP32)
    got = ops.mhc_orthogonalize(g, steps, coeffs)
    want, e = ref.orthogonalize_error(g, steps, coeffs, 1e-7, BF)
    near(got, want, e)


def test_many_steps_give_the_orthogonal_factor():
    """25 steps of the convergent polynomial: rows orthonormal to what the output's rounding allows."""
    g = torch.randn(64, 256, generator=gen(4), device="cuda")
    o = ops.mhc_orthogonalize(g, 25, (1.875, -1.25, 0.375), dtype=FP16).double()
    # elements of size 1/16, off by 2^-12 of themselves: a dot product of 256 of them
    assert float((o @ o.t() - torch.eye(64, device="cuda", dtype=torch.float64)).abs().max()) < 2.0 ** -10


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_sizes_of_any_magnitude(scale):
    g = momentum(gen(9), (80, 144), FP32, 1.0)
    want, e = ref.orthogonalize_error(g * scale, 5, MUON, 0.0, BF)
    got = ops.mhc_orthogonalize(g * scale, eps=0.0)
    near(got, want, e)


def test_zeros_and_values_that_are_not_finite():
    z = torch.zeros(3, 40, 72, device="cuda")
    z[1] = torch.randn(40, 72, generator=gen(1), device="cuda")
    z[2, 0, 0] = float("nan")
    for eps in (1e-7, 0.0):
        o = ops.mhc_orthogonalize(z, eps=eps)
        assert o[0].eq(0).all() and torch.isnan(o[2]).all()
        assert torch.equal(o[1], ops.mhc_orthogonalize(z[1].contiguous(), eps=eps))


def test_strided_batches_and_no_matrices():
    big = torch.randn(4, 100, 300, generator=gen(2), device="cuda")
    for part in (big[:, 3:67, 1:202], big[::2, :, 8:136], big[:, :50].transpose(0, 1)[:, :, :128]):
        assert torch.equal(ops.mhc_orthogonalize(part), ops.mhc_orthogonalize(part.contiguous()))
    assert ops.mhc_orthogonalize(big[:0]).shape == (0, 100, 300)


@pytest.mark.parametrize("shape", [(300, 130), (5, 64, 200)])
def test_the_same_run_to_run_in_a_graph_and_on_another_stream(shape):
    g = momentum(gen(8), shape, BF)
    first = ops.mhc_orthogonalize(g)
    B = shape[0] if len(shape) == 3 else 1
    space = torch.empty(ops.orthogonalize_workspace_bytes(B, *shape[-2:]), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(first)
    assert torch.equal(first, ops.mhc_orthogonalize(g, out=out, workspace=space)) and torch.equal(out, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ops.mhc_orthogonalize(g, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ops.mhc_orthogonalize(g)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, held)


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
