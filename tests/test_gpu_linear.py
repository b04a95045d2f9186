"""The projection with its epilogue and its gradients on the GPU, against the
64-bit forms: sizes off every tile, strides, types, splits and few tokens."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import layers_ref as ref

pytestmark = pytest.mark.gpu
BF, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def rows(g, T, H, dtype, pad=0, offset=0, std=1.0):
    flat = torch.randn(T * (H + pad) + offset, generator=g, device="cuda") * std
    return flat.to(dtype)[offset:].view(T, H + pad)[:, :H]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


SIZES = [(1, 1, 1), (1, 64, 128), (2, 7, 5), (1, 2048, 384), (3, 4160, 130), (16, 128, 257), (17, 131, 259), (48, 72, 1000),
         (63, 65, 129), (64, 512, 640), (65, 64, 64), (129, 192, 130), (300, 1000, 520), (257, 72, 1000), (513, 2048, 96),
         (200, 4096, 72), (700, 520, 2050)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype,bias,res,act,keep_z,pad,offset", [
    (BF, None, None, "none", False, 0, 0),
    (BF, "same", "same", "silu", True, 0, 0),
    (FP16, "fp32", "fp32", "gelu", True, 8, 0),
    (FP16, "same", None, "relu2", False, 3, 1),
    (BF, "fp32", "fp32", "gelu_tanh", False, 16, 8),
    (BF, None, "same", "relu", True, 1, 0)])
def test_forward(T, K, N, dtype, bias, res, act, keep_z, pad, offset):
    g = gen(T * 31 + K)
    x, w = rows(g, T, K, dtype, pad, offset), rows(g, N, K, dtype, pad, offset, K ** -0.5)
    b = None if bias is None else torch.randn(N, generator=g, device="cuda").to(FP32 if bias == "fp32" else dtype)
    r = None if res is None else rows(g, T, N, FP32 if res == "fp32" else dtype, pad)
    got = ops.mhc_linear(x, w, b, r, act, keep_z=keep_z)
    out, z = got if keep_z else (got, None)
    want, wz, eo, ez = ref.linear(x, w, b, r, act)
    assert out.dtype == (dtype if r is None else r.dtype)
    ref.within(out, want, eo)
    if keep_z:
        assert z.dtype == dtype
        ref.within(z, wz, ez)


@pytest.mark.parametrize("T,K,N", [(5, 300, 200), (64, 1024, 256), (300, 4096, 130), (520, 2048, 2048)])
def test_sums_for_fp32_outputs_do_not_drift(T, K, N):
    """Products of one sign, where what the additions cut shows: 2^-21 of the sum at most, which pieces of
    512 products keep (32 instructions of 2^-24 each and the fp32 additions) and one chain of 4096 would not."""
    g = gen(K)
    x = rows(g, T, K, BF).abs()
    w = rows(g, N, K, BF).abs()
    out = ops.mhc_linear(x, w, dtype=FP32)
    want = x.double() @ w.double().t()
    assert float(((out.double() - want) / want).abs().max()) < 40 * 2.0 ** -24
    d = ops.mhc_linear_dx(x, w.t().contiguous(), dtype=FP32)
    assert float(((d.double() - want) / want).abs().max()) < 40 * 2.0 ** -24


@pytest.mark.parametrize("T,K,N", [(64, 65536, 300), (64, 20000, 4096), (33, 65536, 4096), (2, 65528, 136)])
def test_few_tokens_with_a_long_summed_axis_keep_fp32_sums(T, K, N):
    """Many pieces of a sum and two CTAs on an SM, on two streams at once: each piece is off by 32 instructions of
    2^-24 as above, and beside them stand the fp32 additions of K / 512 pieces and of at most 8 CTAs' sums."""
    g = gen(K)
    x = rows(g, T, K, BF).abs()
    w = rows(g, N, K, BF).abs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [ops.mhc_linear(x, w, dtype=FP32, stream=s) for _ in range(3) for s in (None, side)]
    torch.cuda.synchronize()
    want = x.double() @ w.double().t()
    assert float(((outs[0].double() - want) / want).abs().max()) < (40 + K // 512 + 1) * 2.0 ** -24
    assert all(torch.equal(o, outs[0]) for o in outs)
    d = ops.mhc_linear_dx(x, w.t().contiguous(), dtype=FP32)
    assert float(((d.double() - want) / want).abs().max()) < (40 + K // 512 + 1) * 2.0 ** -24


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 2048, 384), (3, 130, 4160), (17, 259, 131), (64, 640, 512), (65, 64, 64),
                                   (129, 130, 192), (300, 520, 1000), (513, 96, 2048), (700, 2050, 520)])
@pytest.mark.parametrize("dtype,act,out,pad", [(BF, "none", None, 0), (BF, "silu", None, 0), (FP16, "gelu", FP32, 3),
                                               (FP16, "gelu_tanh", None, 8), (BF, "relu2", FP32, 0), (BF, "relu", None, 1)])
def test_the_gradient_of_the_input(T, N, K, dtype, act, out, pad):
    g = gen(T * 7 + N)
    d, w = rows(g, T, N, dtype, pad, std=0.1), rows(g, N, K, dtype, pad, std=N ** -0.5)
    z = None if act == "none" else rows(g, T, K, dtype, pad)
    got = ops.mhc_linear_dx(d, w, z, act, dtype=out)
    assert got.dtype == (out or dtype) and got.shape == (T, K)
    want, e = ref.linear_dx(d, w, z, act)
    ref.within(got, want, e)


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 5, 700), (2, 128, 64), (63, 130, 259), (65, 257, 72), (333, 519, 1096),
                                   (1000, 64, 64), (4100, 96, 200), (2048, 520, 520)])
@pytest.mark.parametrize("dtype,out,bias,pad", [(BF, FP32, True, 0), (FP16, FP16, False, 0), (BF, BF, True, 3), (FP16, FP32, True, 8)])
def test_the_gradients_of_the_weight_and_bias(T, N, K, dtype, out, bias, pad):
    g = gen(T + N * 3)
    d, x = rows(g, T, N, dtype, pad, std=0.1), rows(g, T, K, dtype, pad)
    got = ops.mhc_linear_dw(d, x, dtype=out, bias=bias)
    d_w, d_b = got if bias else (got, None)
    want = d.double().t() @ x.double()
    e = ref.product_error(d.double().t(), x.double().t(), 64 + T // 512)
    ref.within(d_w, want, e)
    if bias:
        wb = d.double().sum(0)
        eb = (T + 64) * ref.U * d.double().abs().sum(0)
        ref.within(d_b, wb, eb)
    # added to what is there
    w0, b0 = torch.randn(N, K, generator=g, device="cuda").to(out), torch.randn(N, generator=g, device="cuda")
    w1, b1 = w0.clone(), b0.clone()
    if bias:
        r = ops.mhc_linear_dw(d, x, d_w=w1, d_bias=b1, accumulate=True)
        assert r[0] is w1 or r[0].data_ptr() == w1.data_ptr()
        ref.within(b1, wb + b0.double(), eb + 2 * ref.U * (wb + b0.double()).abs())
    else:
        ops.mhc_linear_dw(d, x, d_w=w1, accumulate=True)
    s = want + w0.double()
    ref.within(w1, s, e + 2 * ref.U * s.abs())


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", [BF, FP16])
def test_the_activations_and_their_slopes_over_their_range(act, dtype):
    """The weights a unit matrix, so that z is x itself: act(z) in fp32 is off by what its evaluation is, relative to
    itself, far out too."""
    K = 64
    x = torch.cat((torch.linspace(-12, 12, 4000), torch.logspace(-4, 0, 500), -torch.logspace(-4, 0, 500), torch.zeros(120)))
    x = x.to(dtype).view(-1, K).cuda()
    eye = torch.eye(K, device="cuda").to(dtype)
    z = x.double()
    out, slope, ea, es = ref.act(z, act)
    for rows in (x, x[:40]):
        got = ops.mhc_linear(rows, eye, act=act, dtype=FP32).double()
        n = rows.shape[0]
        assert ((got - out[:n]).abs() <= 2 * ref.U * ea[:n] + 1e-37).all()
        if act != "none":
            d = ops.mhc_linear_dx(torch.ones_like(rows), eye, rows, act, dtype=FP32).double()
            assert ((d - slope[:n]).abs() <= 2 * ref.U * es[:n] + 1e-37).all()


@pytest.mark.parametrize("T,N", [(300, 264), (90, 72)])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_rows_of_the_residual_and_of_z_on_any_boundary(T, N, pad):
    g = gen(T + pad)
    K = 96
    x, w = rows(g, T, K, BF), rows(g, N, K, BF, 0, 0, K ** -0.5)
    for dt in (BF, FP32):
        r = rows(g, T, N, dt, pad, 1)
        want, _, e, _ = ref.linear(x, w, None, r, "silu")
        ref.within(ops.mhc_linear(x, w, None, r, "silu"), want, e)
    d, w2, z = rows(g, T, K, BF), rows(g, K, N, BF, 0, 0, K ** -0.5), rows(g, T, N, BF, pad, 1)
    want, e = ref.linear_dx(d, w2, z, "gelu")
    ref.within(ops.mhc_linear_dx(d, w2, z, "gelu"), want, e)


def test_no_tokens():
    w = torch.randn(96, 64, device="cuda").to(BF)
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    assert ops.mhc_linear(x, w).shape == (0, 96)
    d = torch.empty(0, 96, device="cuda", dtype=BF)
    assert ops.mhc_linear_dx(d, w).shape == (0, 64)
    d_w, d_b = ops.mhc_linear_dw(d, x, bias=True)
    assert not d_w.any() and not d_b.any() and d_w.shape == (96, 64) and d_b.shape == (96,)
    keep = torch.ones(96, 64, device="cuda")
    assert ops.mhc_linear_dw(d, x, d_w=keep, accumulate=True).eq(1).all()


@pytest.mark.parametrize("T", [1, 40, 130, 513])
def test_what_is_not_finite_stays_where_it_belongs(T):
    """An infinity or a NaN in one token or one row of the weights reaches that row or column alone, also
    where tiles and stages hold rows past the end."""
    g = gen(T)
    K, N = 200, 130
    x, w = rows(g, T, K, BF), rows(g, N, K, BF)
    clean = ops.mhc_linear(x, w)
    x[T - 1, K - 1] = float("inf")
    w[N - 1, 0] = float("nan")
    out = ops.mhc_linear(x, w)
    assert torch.isnan(out[:, N - 1]).all()
    assert not torch.isfinite(out[T - 1]).any()
    assert torch.equal(out[:T - 1, :N - 1], clean[:T - 1, :N - 1])


@pytest.mark.parametrize("T,N", [(1, 96), (33, 96), (200, 97), (300, 96)])
def test_in_place_and_given_buffers(T, N):
    g = gen(N)
    K = 136
    x, w, r = rows(g, T, K, BF), rows(g, N, K, BF), rows(g, T, N, FP32).contiguous()
    want = ops.mhc_linear(x, w, None, r, "silu")
    z = torch.empty(T, N, device="cuda", dtype=BF)
    space = torch.empty(ops.linear_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    out, zz = ops.mhc_linear(x, w, None, r, "silu", out=r, z=z, workspace=space)
    assert out.data_ptr() == r.data_ptr() and zz.data_ptr() == z.data_ptr()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 17, 64, 65, 400])
def test_the_same_run_to_run_and_in_a_graph(T):
    g = gen(T)
    K, N = 1024, 392
    x, w, d = rows(g, T, K, BF), rows(g, N, K, BF), rows(g, T, N, BF)
    b = torch.randn(N, generator=g, device="cuda")
    first = (*ops.mhc_linear(x, w, b, None, "gelu", keep_z=True), ops.mhc_linear_dx(d, w), *ops.mhc_linear_dw(d, x, bias=True))
    for _ in range(3):
        again = (*ops.mhc_linear(x, w, b, None, "gelu", keep_z=True), ops.mhc_linear_dx(d, w), *ops.mhc_linear_dw(d, x, bias=True))
        assert all(torch.equal(a, c) for a, c in zip(first, again))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = (*ops.mhc_linear(x, w, b, None, "gelu", keep_z=True), ops.mhc_linear_dx(d, w), *ops.mhc_linear_dw(d, x, bias=True))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, held))
    x2 = x.flip(0).contiguous()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], ops.mhc_linear(x2, w, b, None, "gelu"))


def test_another_stream():
    g = gen(3)
    x, w = rows(g, 300, 512, BF), rows(g, 256, 512, BF)
    want = ops.mhc_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.mhc_linear(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_rows_of_one_larger_tensor():
    """Operands that are parts of others, rows far apart, the output between none of them."""
    g = gen(5)
    big = rows(g, 300, 4096, BF)
    x, w = big[:, 128:640], big[:200, 1024:1536]
    want, _, e, _ = ref.linear(x, w, None, None, "none")
    ref.within(ops.mhc_linear(x, w), want, e)
    one = big[7:8].expand(90, 4096)[:, :512]           # stride 0
    want, _, e, _ = ref.linear(one, w, None, None, "none")
    ref.within(ops.mhc_linear(one, w), want, e)


@pytest.mark.parametrize("T,N,K", [(1, 40, 24), (511, 33, 200), (512, 4901, 64), (700, 9736, 16), (3000, 200, 136), (6144, 72, 64),
                                   (6145, 72, 64), (70, 65531, 8)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (1, 1)])
def test_the_bias_gradient_beside_the_products_or_before_them(T, N, K, pad, offset):
    """Columns past the last whole run and several groups of columns a CTA, on both sides of the rule; what lies between
    the rows is not finite."""
    g = gen(T + N)
    flat = torch.full((T * (N + pad) + offset + 16,), float("nan"), device="cuda", dtype=BF)
    d = flat[offset:offset + T * (N + pad)].view(T, N + pad)[:, :N]
    d.copy_(torch.randn(T, N, generator=g, device="cuda"))
    x = rows(g, T, K, BF)
    d_w, d_b = ops.mhc_linear_dw(d, x, bias=True)
    want = d.double().sum(0)
    e = (T + 64) * ref.U * d.double().abs().sum(0)
    ref.within(d_b, want, e)
    ref.within(d_w, d.double().t() @ x.double(), ref.product_error(d.double().t(), x.double().t(), 64 + T // 512))
    b0 = torch.randn(N, generator=g, device="cuda")
    b1 = b0.clone()
    ops.mhc_linear_dw(d, x, d_w=torch.zeros_like(d_w), d_bias=b1, accumulate=True)
    s = want + b0.double()
    ref.within(b1, s, e + 2 * ref.U * s.abs())
    assert torch.equal(ops.mhc_linear_dw(d, x, bias=True)[1], d_b)


def test_device_status_is_clean():
    assert ops.mhc_get_device_status() == 0
