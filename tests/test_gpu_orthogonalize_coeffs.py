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


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
