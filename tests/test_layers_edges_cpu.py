"""Edges of the projections', layer norm's and the update's host side that need no GPU."""
import os
import subprocess
import sys

import pytest

from manifold_constrained_hyper_gb300 import build as mbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    return mbuild.build()


@pytest.mark.parametrize("m,n,k", [(96, 64, 0), (1, 1, 0), (65536, 65536, 0), (0, 64, 64)])
def test_a_product_over_nothing_has_no_parts(lib, m, n, k):
    """What a weight gradient of no tokens plans: a division by its zero steps would end the process on hosts that trap it, so a
    process of its own asks."""
    code = (f"import ctypes; f = ctypes.CDLL({lib!r})._ZN3mhc19product_parts_bytesExix; f.restype = ctypes.c_size_t; "
            f"f.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong]; assert f({m}, {n}, {k}) == 0")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(lib))
    assert r.returncode == 0, (r.returncode, r.stderr)
