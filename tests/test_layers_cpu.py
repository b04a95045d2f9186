"""What of layer norm, the projections and the orthogonalised update needs no
GPU: the 64-bit forms' gradients against differences, the entry points'
refusals (before any device work), and the workspace sizes."""
import ctypes

import pytest
import torch

from manifold_constrained_hyper_gb300 import build as mbuild
from manifold_constrained_hyper_gb300 import ops
from tests import layers_ref as ref

A = 0x1000000          # an aligned address that is never read


def _P(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return ops.load()


def _against_differences(f, x, d):
    """d = the gradient of the scalar f at x, element by element."""
    for at in range(x.numel()):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[at] = 1e-5
        e = e.reshape(x.shape)
        diff = float(f(x + e) - f(x - e)) / 2e-5
        # the differences' own error: (1e-5)^2 of the third derivative, 1e-16 / 1e-5 of the value
        assert abs(diff - float(d.reshape(-1)[at])) < 1e-7 * (1 + abs(diff)), at


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("res", [True, False])
def test_layer_norm_s_gradients_against_differences(affine, res):
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, d = rand(3, 7), rand(3, 7)
    w, b = (1 + 0.1 * rand(7), rand(7)) if affine else (None, None)
    extra = rand(3, 7) if res else None

    def loss(x=x, w=w, b=b):
        out = ref.layer_norm(x, w, b, 1e-5)[0]
        return (d * out).sum() + ((extra * x).sum() if res else 0)

    stats = ref.layer_norm(x, w, b, 1e-5)[1]
    got = ref.layer_norm_backward(d, x, stats, w, extra)
    _against_differences(lambda v: loss(x=v), x, got["d_x"][0])
    if affine:
        _against_differences(lambda v: loss(w=v), w, got["d_w"][0])
        _against_differences(lambda v: loss(b=v), b, got["d_b"][0])


@pytest.mark.parametrize("act", ref.ACTS)
def test_the_projections_gradients_against_differences(act):
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, K, N = 3, 5, 6
    # out = w act(z) of the layer below: linear_dx takes d_out to z, linear_dw to w
    z, w, d = rand(T, K), rand(N, K), rand(T, N)
    x = ref.act(z, act)[0]
    _against_differences(lambda v: (d * (ref.act(v, act)[0] @ w.t())).sum(), z, ref.linear_dx(d, w, z, act)[0])
    _against_differences(lambda v: (d * (x @ v.t())).sum(), w, d.t() @ x)
    _against_differences(lambda v: (d * (x @ w.t() + v)).sum(), rand(N), d.sum(0))


def test_the_plain_orthogonal_factor():
    g = torch.randn(6, 10, dtype=torch.float64)
    o = ref.orthogonalize(g, 30, (1.875, -1.25, 0.375), 0.0)
    assert float((o @ o.t() - torch.eye(6, dtype=torch.float64)).abs().max()) < 1e-9
    assert torch.allclose(ref.orthogonalize(g.t(), 5, (3.4445, -4.775, 2.0315), 1e-7).t(),
                          ref.orthogonalize(g, 5, (3.4445, -4.775, 2.0315), 1e-7))


def _linear(lib, x=A, xs=64, w=A * 2, wsd=64, t=1, T=4, n=32, k=64, b=A * 3, bt=0, r=A * 4, rs=32, act=1, out=A * 5, ot=1,
            z=A * 6, ws=A * 7, wsb=1 << 20):
    return lib.mhc_linear(_P(x), xs, _P(w), wsd, t, T, n, k, _P(b), bt, _P(r), rs, act, _P(out), ot, _P(z), _P(ws), wsb, None)


def test_refusals_of_the_projection(lib):
    for bad in (dict(T=-1), dict(xs=-1), dict(wsd=-64), dict(rs=-1), dict(act=6), dict(act=-1), dict(xs=1 << 62)):
        assert _linear(lib, **bad) == 3, bad
    for bad in (dict(n=0), dict(k=0), dict(n=65537), dict(k=70000), dict(t=0), dict(t=3), dict(ot=2), dict(bt=2), dict(T=1 << 31)):
        assert _linear(lib, **bad) == 4, bad
    for bad in (dict(x=None), dict(w=None), dict(out=None)):
        assert _linear(lib, **bad) == 1, bad
    for bad in (dict(x=A + 1), dict(w=A * 2 + 1), dict(b=A * 3 + 2), dict(r=A * 4 + 1), dict(out=A * 5 + 1), dict(z=A * 6 + 1),
                dict(ws=A * 7 + 8), dict(ot=0, out=A * 5 + 2)):
        assert _linear(lib, **bad) == 2, bad
    # rows off 16 bytes are copied: the workspace is needed then
    assert _linear(lib, x=A + 2, ws=None) == 1
    assert _linear(lib, xs=66, wsb=16) == 8
    for bad in (dict(out=A), dict(out=A * 2 + 64), dict(out=A * 3), dict(out=A * 4 + 2), dict(z=A * 5), dict(z=A + 8), dict(out=A * 4, rs=40),
                dict(x=A + 2, ws=A * 5)):
        assert _linear(lib, **bad) == 5, bad
    assert _linear(lib, T=0, x=None, w=None, out=None) == 0


def test_refusals_of_its_gradients(lib):
    def dx(d=A, ds=32, w=A * 2, wsd=64, t=1, T=4, n=32, k=64, z=A * 3, zs=64, act=3, out=A * 4, ot=1, ws=A * 5, wsb=1 << 20):
        return lib.mhc_linear_dx(_P(d), ds, _P(w), wsd, t, T, n, k, _P(z), zs, act, _P(out), ot, _P(ws), wsb, None)

    def dw(d=A, ds=32, x=A * 2, xs=64, t=1, T=4, n=32, k=64, out=A * 3, ot=0, b=A * 4, acc=0, ws=A * 5, wsb=1 << 20):
        return lib.mhc_linear_dw(_P(d), ds, _P(x), xs, t, T, n, k, _P(out), ot, _P(b), acc, _P(ws), wsb, None)

    for bad in (dict(T=-1), dict(ds=-1), dict(wsd=-1), dict(zs=-1), dict(act=9), dict(ds=1 << 62), dict(zs=1 << 62)):
        assert dx(**bad) == 3, bad
    for bad in (dict(n=0), dict(k=65537), dict(t=0), dict(ot=2), dict(T=1 << 31)):
        assert dx(**bad) == 4, bad
    for bad in (dict(d=None), dict(w=None), dict(out=None), dict(z=None), dict(d=A + 2, ws=None)):
        assert dx(**bad) == 1, bad
    for bad in (dict(d=A + 1), dict(z=A * 3 + 1), dict(out=A * 4 + 1), dict(ws=A * 5 + 4)):
        assert dx(**bad) == 2, bad
    assert dx(ds=34, wsb=0) == 8
    for bad in (dict(out=A), dict(out=A * 3), dict(out=A * 2 + 64)):
        assert dx(**bad) == 5, bad
    assert dx(T=0, d=None, w=None, z=None, out=None) == 0

    for bad in (dict(T=-1), dict(ds=-1), dict(xs=-1), dict(ot=5), dict(xs=1 << 62)):
        assert dw(**bad) == 3, bad
    for bad in (dict(n=0), dict(k=0), dict(t=0), dict(T=1 << 31)):
        assert dw(**bad) == 4, bad
    for bad in (dict(d=None), dict(x=None), dict(out=None), dict(x=A * 2 + 2, ws=None)):
        assert dw(**bad) == 1, bad
    for bad in (dict(x=A * 2 + 1), dict(out=A * 3 + 2), dict(b=A * 4 + 2), dict(ws=A * 5 + 8)):
        assert dw(**bad) == 2, bad
    assert dw(xs=66, wsb=16) == 8
    for bad in (dict(out=A), dict(b=A * 2 + 32), dict(b=A * 3 + 64)):
        assert dw(**bad) == 5, bad
    assert dw(T=0, acc=1, d=None, x=None) == 0


def test_refusals_of_layer_norm(lib):
    f = ctypes.c_float

    def fwd(x=A, xs=64, t=1, T=4, H=64, w=A * 2, wt=0, b=A * 3, bt=0, eps=1e-5, out=A * 4, ot=1, st=A * 5):
        return lib.mhc_layer_norm(_P(x), xs, t, T, H, _P(w), wt, _P(b), bt, f(eps), _P(out), ot, _P(st), None)

    def back(d=A, ds=64, ot=1, x=A * 2, xs=64, t=1, st=A * 3, T=4, H=64, w=A * 4, wt=0, r=A * 5, rs=64, dx=A * 6, dw=A * 7, db=A * 8,
             ws=A * 9, wsb=1 << 20):
        return lib.mhc_layer_norm_backward(_P(d), ds, ot, _P(x), xs, t, _P(st), T, H, _P(w), wt, _P(r), rs, _P(dx), _P(dw), _P(db), _P(ws),
                                           wsb, None)

    for bad in (dict(T=-1), dict(xs=-1), dict(t=3), dict(ot=-1), dict(wt=7), dict(bt=7), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(xs=1 << 62)):
        assert fwd(**bad) == 3, bad
    for bad in (dict(H=0), dict(H=65537), dict(ot=2), dict(ot=0), dict(T=1 << 31)):
        assert fwd(**bad) == 4, bad
    for bad in (dict(x=None), dict(out=None)):
        assert fwd(**bad) == 1, bad
    for bad in (dict(x=A + 1), dict(w=A * 2 + 2), dict(b=A * 3 + 1), dict(out=A * 4 + 1), dict(st=A * 5 + 2)):
        assert fwd(**bad) == 2, bad
    for bad in (dict(out=A), dict(out=A * 2), dict(st=A * 4 + 64), dict(st=A * 3)):
        assert fwd(**bad) == 5, bad
    assert fwd(T=0, x=None, out=None) == 0

    for bad in (dict(T=-1), dict(ds=-1), dict(xs=-1), dict(rs=-1), dict(t=3), dict(ot=3), dict(wt=-1), dict(ds=1 << 62)):
        assert back(**bad) == 3, bad
    for bad in (dict(H=0), dict(H=65537), dict(ot=2), dict(t=1, ot=0)):
        assert back(**bad) == 4, bad
    for bad in (dict(d=None), dict(x=None), dict(st=None), dict(dx=None), dict(T=400, ws=None)):
        assert back(**bad) == 1, bad
    for bad in (dict(d=A + 1), dict(dx=A * 6 + 1), dict(dw=A * 7 + 2), dict(db=A * 8 + 1), dict(ws=A * 9 + 8), dict(st=A * 3 + 2)):
        assert back(**bad) == 2, bad
    assert back(T=400, wsb=64) == 8
    for bad in (dict(dx=A), dict(dx=A * 2), dict(dx=A * 5 + 2), dict(dx=A * 5, rs=72), dict(dw=A * 8), dict(T=400, ws=A * 7)):
        assert back(**bad) == 5, bad


def test_refusals_of_the_orthogonalised_update(lib):
    f = ctypes.c_float

    def go(g=A, rs=512, bs=512 * 256, t=0, B=2, m=256, n=512, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, out=A * 2, ot=1, ws=A * 4, wsb=1 << 28):
        return lib.mhc_orthogonalize(_P(g), rs, bs, t, B, m, n, steps, f(a), f(b), f(c), f(eps), _P(out), ot, _P(ws), wsb, None)

    for bad in (dict(B=-1), dict(rs=-1), dict(bs=-1), dict(t=3), dict(steps=0), dict(steps=101), dict(eps=-1.0), dict(eps=float("nan")),
                dict(a=float("nan")), dict(b=2000.0), dict(c=float("inf")), dict(rs=1 << 62), dict(bs=1 << 50)):
        assert go(**bad) == 3, bad
    for bad in (dict(m=0), dict(n=65537), dict(B=65536), dict(ot=0)):
        assert go(**bad) == 4, bad
    for bad in (dict(g=None), dict(out=None), dict(ws=None)):
        assert go(**bad) == 1, bad
    for bad in (dict(g=A + 2), dict(out=A * 2 + 1), dict(ws=A * 4 + 8)):
        assert go(**bad) == 2, bad
    assert go(wsb=1 << 10) == 8
    for bad in (dict(out=A), dict(ws=A * 2)):
        assert go(**bad) == 5, bad
    assert go(B=0, g=None, out=None, ws=None) == 0


def test_workspace_sizes(lib):
    assert ops.linear_workspace_bytes(0, 64, 64) == 0 and ops.linear_workspace_bytes(4, 0, 64) == 0
    # a few tokens: only what is copied
    assert ops.linear_workspace_bytes(8, 100, 7, False, True) == 256 and ops.linear_workspace_bytes(8, 4096, 4096) == 0
    assert ops.linear_dx_workspace_bytes(8, 100, 7, True, False) == 100 * 8 * 2 // 256 * 256 + 256
    assert ops.linear_dw_workspace_bytes(3, 8, 8, False, False) == 512
    assert ops.layer_norm_backward_workspace_bytes(0, 64) == 0
    assert ops.layer_norm_backward_workspace_bytes(5, 64) == 0         # one CTA adds them up
    assert ops.layer_norm_backward_workspace_bytes(500, 64) >= 2 * 64 * 4
    assert ops.layer_norm_backward_workspace_bytes(1 << 20, 64) == ops.layer_norm_backward_workspace_bytes(1 << 30, 64)
    assert ops.orthogonalize_workspace_bytes(0, 64, 64) == 0 and ops.orthogonalize_workspace_bytes(3, 128, 2048) == 0
    big = ops.orthogonalize_workspace_bytes(1, 2048, 4096)
    assert big >= 4 * 2048 * 4096 * 2 + 8 * 2048 * 2048 * 2


def test_the_binding_refuses_on_the_host(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: ops.mhc_linear(x, x), lambda: ops.mhc_linear_dx(x, x), lambda: ops.mhc_linear_dw(x, x), lambda: ops.mhc_layer_norm(x),
                 lambda: ops.mhc_layer_norm_backward(x, x, x), lambda: ops.mhc_orthogonalize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="act must be one of"):
        ops.mhc_linear(x, x, act="swish")
    with pytest.raises(ValueError, match="accumulate needs"):
        ops.mhc_linear_dw(x, x, accumulate=True)
    with pytest.raises(ValueError, match="must be float32"):
        ops.mhc_orthogonalize(x, dtype=torch.float64)
