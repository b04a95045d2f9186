"""Edges of the projections', layer norm's and the update's host side that need no GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

from manifold_constrained_hyper_gb300 import build as mbuild
from manifold_constrained_hyper_gb300 import ops


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


@pytest.mark.parametrize("a,refused", [(16.0, True), (-16.0, True), (1000.0, True), (15.99, False), (-15.99, False), (0.0, False)])
def test_coefficients_that_overflow_by_themselves_are_refused(a, refused):
    """P has a on its diagonal, and overflows from 16 on whatever the matrix: zeros gave NaN. Without matrices nothing is launched."""
    f, P, A = ctypes.c_float, ctypes.c_void_p, 0x1000000

    def go(batch):
        return ops.load().mhc_orthogonalize(P(A), 512, 512 * 256, 0, batch, 256, 512, 5, f(a), f(-1.0), f(0.5), f(1e-7), P(A * 2), 1, P(A * 4), 1 << 28, None)

    assert go(0) == (3 if refused else 0)
    if refused:
        assert go(2) == 3


@pytest.mark.parametrize("m,n,ctas,fits", [(128, 2048, 16, True), (128, 2049, 16, False), (128, 2048, 8, False), (1024, 128, 8, True), (128, 1025, 8, False),
                                           (64, 4096, 16, True), (64, 4096, 8, False), (2048, 64, 8, True), (32, 8192, 16, True), (4096, 32, 8, True),
                                           (32, 4097, 8, False), (129, 129, 16, False), (1, 1, 1, True), (1, 1, -1, False)])
def test_small_updates_take_no_larger_cluster_than_the_device_holds(lib, m, n, ctas, fits):
    """16 CTAs in a cluster are not portable: where the device does not hold them (a part of it, say), the general form runs, and its
    workspace is asked for."""
    f = ctypes.CDLL(lib)._ZN3mhc16ns_small_fits_inEiii
    f.restype, f.argtypes = ctypes.c_bool, [ctypes.c_int] * 3
    assert f(m, n, ctas) == fits


SHAPES = r"""
#include <cstdio>
#include <initializer_list>
#include "layer_norm_shape.h"
using namespace mhc;
static int bad = 0;
#define CHECK(c) do { if (!(c)) { ++bad; std::printf("H %d: %s\n", H, #c); } } while (0)
// Groups of several warps wait at barriers 1 .. groups, all of them at kLnAllBarrier; a reduction has 16 places a group at most.
static void group(int H, int R, int warps, int groups, int most_groups) {
    CHECK(R * warps * 256 >= H);
    CHECK(warps >= 1 && warps <= 16 && groups >= 1 && groups <= most_groups);
    CHECK(warps == 1 || groups < kLnAllBarrier);
}
int main() {
    for (int H = 1; H <= kLnMaxHeld; ++H) {
        const LnRows r = ln_rows(H);
        group(H, r.R, r.warps, r.groups, 16);
        CHECK(32 * r.warps * r.groups <= kLnThreads);
        for (int x = 2; x <= 4; x += 2) {
            int place[kLnArrays + 1];
            const int one[kLnArrays] = {H * x, 0, 0};
            ln_places(one, place);
            // a row from any byte of its first 16, and what the last run reads past its end
            CHECK(place[kLnArrays] >= H * x + 15 + 48 && place[kLnArrays] % 128 == 0);
            for (int runs = 0; runs < 2; ++runs)
                for (int affine = 0; affine < 2; ++affine) {
                    const LnRingShape s = ln_ring_shape(H, place[kLnArrays], runs, affine);
                    group(H, s.R, s.warps, s.groups, kLnRingGroups);
                    CHECK(32 * (s.warps * s.groups + 1) <= kLnRingThreads);
                    CHECK(s.stages >= 1 && 16 * s.groups * s.stages <= kLnRingBars);
                    CHECK(s.smem <= kLnRingSmem && kLnRingSmem + 4096 <= 227 * 1024);
                }
            for (int d = 2; d <= x; d += 2)
                for (int residual = 0; residual < 2; ++residual) {
                    const int all[kLnArrays] = {H * x, H * d, residual ? H * x : 0};
                    ln_places(all, place);
                    for (long long T : {1LL, 2432LL, 1LL << 30}) {
                        const LnBack p = ln_back(T, H, 152);
                        group(H, p.R, p.warps, p.groups, 16);
                        CHECK(32 * (p.warps * p.groups + (p.ring && !p.self)) <= kLnThreads);
                        CHECK(p.parts >= 1 && p.parts <= 152 && ln_back_meet(p, H) <= kLnBackMeetSmem);
                        if (!p.ring) continue;
                        const LnBackRing s = ln_back_ring(p, H, place[kLnArrays], residual);
                        CHECK(s.stages >= 0 && 16 * p.groups * s.stages <= kLnBackRingBars);
                        CHECK(!s.stages || (s.smem <= kLnBackRingSmem && kLnBackRingSmem + 8192 <= 227 * 1024));
                        CHECK(s.smem >= kLnBackRingBars + s.params + ln_back_meet(p, H));
                    }
                }
        }
    }
    return bad != 0;
}
"""


def test_layer_norm_s_launch_shapes_keep_the_kernels_limits_for_every_width(tmp_path):
    """Barriers' numbers, threads, places of the reductions, stages and shared memory, of every form, type and width."""
    src, exe = tmp_path / "shapes.cpp", tmp_path / "shapes"
    src.write_text(SHAPES)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-I", mbuild.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[:2000]
