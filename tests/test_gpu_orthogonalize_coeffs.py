"""The orthogonalised update with coefficients and numbers of steps other than the usual ones, at sizes of every
form, against its 64-bit form; and the workspace's contents, which no result may depend on."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import layers_ref as ref
from tests.test_gpu_linear import BF, FP16, FP32, gen
from tests.test_gpu_orthogonalize import MUON, momentum, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def space(shape):
    """A workspace whose every 16-bit element, and every fp32 one, is a NaN."""
    B = shape[0] if len(shape) == 3 else 1
    n = ops.orthogonalize_workspace_bytes(B, *shape[-2:])
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None


# of the general form: by CTAs and by pairs, wide and tall, a batch, split sums
GENERAL = [(200, 300), (257, 600), (600, 257), (3, 150, 260), (129, 2500), (700, 1000)]


@pytest.mark.parametrize("shape", GENERAL + [(96, 200), (2, 40, 700)], ids=str)
@pytest.mark.parametrize("steps,coeffs", [(1, (1.5, -0.5, 0.0)), (3, (1.5, -0.5, 0.0)), (1, (3.0, -18.0, 1.0)), (1, (1.5, -0.5, 0.02)),
                                          (2, (1.5, -0.5, 0.02)), (4, (2.0, -1.0, 0.01)), (1, MUON), (2, MUON)])
@pytest.mark.parametrize("out", [BF, FP16])
def test_polynomials_that_are_not_completed(shape, steps, coeffs, out):
    """c = 0, or b / 2c above 8: the product of A with itself has b A added to it, in the last step of a bf16
    result from an A that is held in one part."""
    g = momentum(gen(sum(shape) + steps), shape, FP32)
    got = ops.mhc_orthogonalize(g, steps, coeffs, dtype=out, workspace=space(shape))
    want, e = ref.orthogonalize_error(g, steps, coeffs, 1e-7, out)
    near(got, want, e)
    assert torch.equal(got, ops.mhc_orthogonalize(g, steps, coeffs, dtype=out))


@pytest.mark.parametrize("shape", GENERAL + [(96, 200), (2, 40, 700), (300, 30), (2048, 2600)], ids=str)
@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, MUON), (5, MUON), (1, (3.0, -30.0, 2.0)), (1, (3.0, -16.0, 1.0)), (2, (3.0, -16.0, 1.0)),
                                          (1, (9.85, -8.8, 0.0)), (1, (2.13, 8.66, -0.83)), (3, (1.5, -0.5, 0.0))])
def test_a_bf16_result_is_the_fp16_one_rounded(shape, steps, coeffs):
    """Products do not know the type of the result, so either is a rounding of the same value: off by at most half a step, 2^-8
    and 2^-11 of itself, or 2^-25 below fp16's smallest normal values."""
    g = momentum(gen(sum(shape) + steps), shape, FP32)
    bf, half = (ops.mhc_orthogonalize(g, steps, coeffs, dtype=t).double() for t in (BF, FP16))
    assert torch.isfinite(half).all()
    assert ((bf - half).abs() <= half.abs() * (2.0 ** -8 + 2.0 ** -11) * (1 + 2.0 ** -10) + 2.0 ** -24).all()


@pytest.mark.parametrize("shape", [(96, 200), (257, 600), (600, 257), (3, 150, 260)], ids=str)
@pytest.mark.parametrize("steps,coeffs", [(1, (3.0, -30.0, 2.0)), (1, (3.0, -16.0, 1.0)), (2, (3.0, -16.0, 1.0)), (3, (2.0, -1.5, 0.5))])
@pytest.mark.parametrize("out", [BF, FP16])
def test_coefficients_that_all_but_cancel(shape, steps, coeffs, out):
    """c (b / 2c)^2 far above a: what A has on its diagonal cancels in P, 112 beside 3. Rounding takes at most half a step of each
    element, so of the norm too. The tensor cores cut up to 2^-24 of that 112 with each of the 12 instructions for 64 of the
    summed axis, 1.4e-4 of P for 260 of it, and the 22 bits of A leave less: together below a fifth of fp16's half step beside
    the half that its rounding takes at most on average."""
    g = torch.randn(*shape, generator=gen(steps), device="cuda")
    got = ops.mhc_orthogonalize(g, steps, coeffs, dtype=out)
    want = ref.orthogonalize(g, steps, coeffs, 1e-7)
    assert float((got.double() - want).norm() / want.norm()) < 1.2 * torch.finfo(out).eps / 2


@pytest.mark.parametrize("shape", [(96, 200), (257, 600), (2, 130, 140)], ids=str)
@pytest.mark.parametrize("a", [15.99, -15.99])
def test_the_largest_coefficient(shape, a):
    """Just below what is refused: P's diagonal is held, and zeros stay zeros."""
    for coeffs in ((a, 0.0, 0.0), (a, 0.5, 0.25)):
        g = torch.randn(*shape, generator=gen(3), device="cuda")
        got = ops.mhc_orthogonalize(g, 1, coeffs, dtype=FP16)
        want = ref.orthogonalize(g, 1, coeffs, 1e-7)
        assert float((got.double() - want).norm() / want.norm()) < 1.2 * torch.finfo(FP16).eps / 2
        assert not ops.mhc_orthogonalize(torch.zeros_like(g), 1, coeffs).any()


@pytest.mark.parametrize("shape", [(1, 65536), (65536, 1), (3, 50000), (50000, 5), (129, 20000), (2, 33, 9000)], ids=str)
@pytest.mark.parametrize("out", [BF, FP16])
def test_long_and_narrow(shape, out):
    """A side that no cluster holds beside one of a few rows: tiles mostly of rows past the end, sums over up to 65536."""
    g = momentum(gen(sum(shape)), shape, FP32)
    got = ops.mhc_orthogonalize(g, dtype=out, workspace=space(shape))
    want, e = ref.orthogonalize_error(g, 5, MUON, 1e-7, out)
    near(got, want, e)


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
