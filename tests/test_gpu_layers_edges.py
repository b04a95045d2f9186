"""Edges of the layers beside a boundary on the GPU that their own files leave out."""
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


def half_ulp(t, value):
    """Half a step of type t in each value's own binade (normal values)."""
    return torch.exp2(torch.floor(torch.log2(value.abs()))) * torch.finfo(t).eps / 2


@pytest.mark.parametrize("T,K,N", [(3, 65536, 19500), (64, 30000, 19500), (2, 65528, 136)])
@pytest.mark.parametrize("dtype", [BF, FP16])
def test_few_tokens_with_a_long_summed_axis_keep_sums_of_16_bit_results(T, K, N, dtype):
    """Products of one sign, so that what the tensor cores cut adds up: pieces of 64 steps, 256 instructions, and the fp32 additions
    of K / 4096 pieces and of at most 8 CTAs' sums. 19500 columns leave nothing to split. An instruction adds 16 products to the sum
    and cuts each of the 17 terms below one and the same bit. bf16 products, 16 bits far below the sum, leave little there: 2^-24 of
    the sum in all, as for the fp32 results elsewhere. fp16 products have 22 bits, so that each of them is cut, by half of that bit
    on average and all of it at most: fp32 results of the same products, in pieces of 32 instructions, are 2.8e-6 too small on average, so
    an instruction cuts 1.5 x 2^-24 on average and twice that, below 2^-22, at most. (One piece of 65536 products came to 4e-4.)"""
    g = gen(K)
    x = rows(g, T, K, dtype).abs()
    w = torch.empty(N, K, dtype=dtype, device="cuda")
    for i in range(0, N, 1000):
        w[i:i + 1000] = torch.randn(min(1000, N - i), K, generator=g, device="cuda").abs_() / K
    out = ops.mhc_linear(x, w)
    d = ops.mhc_linear_dx(x, w[:256].t().contiguous()) if N > 256 else None
    rel = (256 * (4 if dtype == FP16 else 1) + K // 4096 + 1 + 8) * 2.0 ** -24
    for i in range(0, N, 1000):
        want = x.double() @ w[i:i + 1000].double().t()
        assert ((out[:, i:i + 1000].double() - want).abs() <= half_ulp(dtype, want * (1 + rel)) + rel * want).all()
        if i == 0 and d is not None:
            assert ((d.double() - want[:, :256]).abs() <= half_ulp(dtype, want[:, :256] * (1 + rel)) + rel * want[:, :256]).all()


def test_gradients_do_not_go_missing():
    """Every tensor of every call, where gradients of it are being recorded; the same calls without."""
    x, w, d, z = (torch.randn(*n, device="cuda").to(BF) for n in ((8, 64), (32, 64), (8, 32), (8, 64)))
    p, b, r, f = torch.randn(64, device="cuda"), torch.randn(32, device="cuda"), torch.randn(8, 32, device="cuda"), torch.randn(8, 64, device="cuda")
    stats = ops.mhc_layer_norm(x)[1]
    calls = ((lambda x, w, b, r: ops.mhc_linear(x, w, b, r), (x, w, b, r)), (lambda d, w, z: ops.mhc_linear_dx(d, w, z, "silu"), (d, w, z)),
             (ops.mhc_linear_dw, (d, x)), (lambda x, w, b: ops.mhc_layer_norm(x, w, b)[0], (x, p, p)),
             (lambda d, x, s, w, r: ops.mhc_layer_norm_backward(d, x, s, w, d_residual=r).d_x, (x, x, stats, p, z)), (ops.mhc_orthogonalize, (f,)))
    for call, tensors in calls:
        want = call(*tensors)
        for i in range(len(tensors)):
            leaf = [t.clone().requires_grad_(k == i) for k, t in enumerate(tensors)]
            with pytest.raises(ValueError, match="requires grad"):
                call(*leaf)
            with torch.no_grad():
                assert torch.equal(call(*leaf), want)


@pytest.mark.parametrize("T,H,types", [(2500, 2048, (FP16, FP16)), (2000, 4096, (BF, BF)), (1300, 1999, (BF, BF)), (1600, 1102, (FP32, FP32)),
                                       (1400, 7168, (FP32, BF)), (1300, 7167, (FP16, FP16)), (1250, 8191, (FP32, FP32)), (5000, 264, (FP16, FP16)),
                                       (1300, 3585, (BF, BF)), (300, 9001, (BF, BF))])
@pytest.mark.parametrize("affine", [True, False])
def test_a_residual_gradient_in_place_among_many_rows(T, H, types, affine):
    """d_x in d_residual's place, where later rows are on their way to shared memory while earlier ones are written, and rows off 16
    bytes come with words that hold their neighbours' ends: by a warp that orders rows, by the groups' first threads, unstaged."""
    xt, ot = types
    g = gen(T + H)
    x, d, r = rows(g, T, H, xt), rows(g, T, H, ot, 0, 0, 0.1), rows(g, T, H, xt)
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda") if affine else None
    stats = ops.mhc_layer_norm(x, w, w)[1]
    want = ops.mhc_layer_norm_backward(d, x, stats, w, bias=affine, d_residual=r)
    ref.within(want.d_x, *ref.layer_norm_backward(d, x, stats, w, r)["d_x"])
    for _ in range(3):
        place = r.clone()
        got = ops.mhc_layer_norm_backward(d, x, stats, w, bias=affine, d_residual=place, d_x=place)
        assert got.d_x.data_ptr() == place.data_ptr()
        assert all(a is b if a is None else torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T,K,N,act", [(9000, 64, 2304, "gelu"), (9001, 72, 2305, "silu"), (4100, 2048, 1024, "none"), (300, 8192, 264, "relu2")])
@pytest.mark.parametrize("dtype", [BF, FP32])
def test_a_residual_in_place_with_several_tiles_a_cta(T, K, N, act, dtype):
    """out in the residual's place: tiles in turn, and sums that are split and joined."""
    g = gen(T)
    x, w, b, r = rows(g, T, K, BF), rows(g, N, K, BF, 0, 0, K ** -0.5), torch.randn(N, generator=g, device="cuda"), rows(g, T, N, dtype)
    want = ops.mhc_linear(x, w, b, r, act)
    exact, _, e, _ = ref.linear(x, w, b, r, act)
    ref.within(want, exact, e)
    for _ in range(3):
        place = r.clone()
        out, z = ops.mhc_linear(x, w, b, place, act, out=place, keep_z=True)
        assert out.data_ptr() == place.data_ptr() and torch.equal(out, want)


def _spaces(n):
    """None, and a workspace of n bytes whose every element of any type is a NaN."""
    return (None, torch.full((n,), 255, dtype=torch.uint8, device="cuda")) if n else (None,)


@pytest.mark.parametrize("T,K,N,pad", [(5, 300, 200, 3), (64, 4096, 130, 0), (130, 4160, 264, 0), (300, 519, 1096, 3), (1000, 64, 64, 8), (700, 2050, 520, 1)])
def test_workspaces_need_no_initialisation(T, K, N, pad):
    """Copies of rows, parts of split sums and sums over tokens: written before they are read."""
    g = gen(T + K)
    x, w, d = rows(g, T, K, BF, pad), rows(g, N, K, BF, pad, 0, K ** -0.5), rows(g, T, N, BF, pad)
    al = pad % 8 == 0 and K % 8 == 0 and N % 8 == 0
    for call, n in ((lambda s: [ops.mhc_linear(x, w, workspace=s)], ops.linear_workspace_bytes(T, N, K, al, al)),
                    (lambda s: [ops.mhc_linear_dx(d, w, workspace=s)], ops.linear_dx_workspace_bytes(T, N, K, al, al)),
                    (lambda s: list(ops.mhc_linear_dw(d, x, bias=True, workspace=s)), ops.linear_dw_workspace_bytes(T, N, K, al, al))):
        got = [call(s) for s in _spaces(n)]
        assert all(torch.isfinite(t).all() for t in got[0])
        assert all(torch.equal(p, q) for other in got[1:] for p, q in zip(got[0], other))
    for H in (K, 8 * K + 1):
        y, e = rows(g, T, H, FP32), rows(g, T, H, FP32)
        p = torch.randn(H, generator=g, device="cuda")
        stats = ops.mhc_layer_norm(y, p, p)[1]
        got = [ops.mhc_layer_norm_backward(e, y, stats, p, workspace=s) for s in _spaces(ops.layer_norm_backward_workspace_bytes(T, H))]
        assert all(torch.isfinite(t).all() for t in got[0])
        assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
