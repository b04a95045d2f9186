"""8-bit activation checkpoints on the GPU: codes and scales bit for bit
against the plain 64-bit form, the block's fused checkpoints and its backward
pass from them, and the weight gradient read from a checkpoint."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import block_ref as ref
from tests.test_gpu_block import BF, FP16, FP32, check_backward, check_forward, make, params, within

pytestmark = pytest.mark.gpu

TYPES = {"bf16": BF, "fp16": FP16, "fp32": FP32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def _same(c, x):
    codes, scales = ref.pack(x, c.fmt)
    assert torch.equal(c.scales, scales)
    assert torch.equal(c.codes, codes)


def _reads_back(c, dtypes=(BF, FP16, FP32)):
    want = ref.unpack(c.codes, c.scales, c.fmt)
    for dt in dtypes:
        got = ops.mhc_ckpt_unpack(c, dt)
        assert got.dtype == dt
        w = want.float().to(dt)            # 64 -> 32 bits is exact: codes of at most 8 bits
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(got[~torch.isnan(got)], w[~torch.isnan(w)])


@pytest.mark.parametrize("T,H,pad,offset", [(1, 1, 0, 0), (3, 5, 0, 0), (1, 32, 0, 0), (2, 33, 0, 0), (5, 64, 0, 0),
                                            (4, 96, 0, 0), (3, 96, 8, 0), (2, 128, 0, 1), (3, 160, 3, 0), (7, 1000, 0, 0),
                                            (2, 1999, 1, 3), (300, 256, 0, 0), (1, 7168, 0, 0), (3, 7168, 16, 16),
                                            (2, 65536, 0, 0)])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_bit_for_bit(T, H, pad, offset, dtype, fmt):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + H)
    flat = torch.randn(T * (H + pad) + offset, generator=g, device="cuda") * 3
    x = flat.to(TYPES[dtype])[offset:].view(T, H + pad)[:, :H]
    c = ops.mhc_ckpt_pack(x, fmt)
    _same(c, x)
    _reads_back(c)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [64, 61])
def test_edge_values(fmt, H):
    """Borders of the scale, ties of the codes, subnormals, zeros of either
    sign, and what is not finite, each in a group of its own."""
    q = ref.QMAX[fmt]
    up = torch.nextafter(torch.tensor(q), torch.tensor(1e9)).item()
    rows = []
    for e in (-149, -140, -130, -127, -126, -120, -20, 0, 1, 30, 110, 118):
        for m in (1.0, 1.5, 1.75, 1.9375, 1.984375, 1.9999999):
            rows.append([m * 2.0 ** e, -m * 2.0 ** (e - 3)])
    rows += [[q], [up], [-q], [-up], [q * 2.0 ** -126], [up * 2.0 ** -126], [0.0, -0.0], [3.4028234663852886e38]]
    ties = [k + 0.5 for k in range(-20, 20)] if fmt == "int8" else [(17 + 2 * k) * 2.0 ** (e - 4)
                                                                     for k in range(8) for e in (0, 1, -6)]
    ties += [k * 2.0 ** -10 for k in range(1, 18)] if fmt == "e4m3" else []
    rows += [[q, *ties[i:i + 25]] for i in range(0, len(ties), 25)]
    x = torch.zeros(len(rows), H, dtype=torch.float64)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r, dtype=torch.float64)
        x[i, 32:32 + len(r)] = torch.tensor(r, dtype=torch.float64)
    x = x.float().cuda()
    _same(ops.mhc_ckpt_pack(x, fmt), x)
    _reads_back(ops.mhc_ckpt_pack(x, fmt), (FP32,))
    b = x.to(BF)
    b = torch.where(torch.isinf(b), torch.zeros_like(b), b)
    _same(ops.mhc_ckpt_pack(b, fmt), b)
    bad = torch.randn(6, H, device="cuda")
    bad[1, 3], bad[2, 40], bad[3, 0], bad[4, 33] = float("nan"), float("inf"), float("-inf"), float("-nan")
    for dt in (FP32, BF, FP16):
        c = ops.mhc_ckpt_pack(bad.to(dt), fmt)
        _same(c, bad.to(dt))
        _reads_back(c)


def test_no_tokens_and_a_given_output():
    for fmt in ("e4m3", "int8"):
        c = ops.mhc_ckpt_pack(torch.empty(0, 64, dtype=BF, device="cuda"), fmt)
        assert ops.mhc_ckpt_unpack(c).shape == (0, 64)
    x = torch.randn(8, 96, device="cuda")
    c = ops.ckpt_empty(8, 96, "int8")
    assert ops.mhc_ckpt_pack(x, "int8", out=c) is c
    _same(c, x)
    out = torch.empty(8, 96, device="cuda")
    assert ops.mhc_ckpt_unpack(c, FP32, out=out) is out
    with pytest.raises(ValueError, match="format"):
        ops.mhc_ckpt_pack(x, "e4m3", out=c)
    with pytest.raises(ValueError, match="dtype"):
        ops.mhc_ckpt_unpack(c, torch.float64)
    with pytest.raises(ValueError, match="x must"):
        ops.mhc_ckpt_pack(x.double())
    with pytest.raises(ValueError, match="scales"):
        ops.Checkpoint(c.codes, c.scales[:, :2].contiguous(), "int8")
    # codes in the middle of an allocation, no more than byte aligned
    flat = torch.empty(8 * 96 + 1, dtype=torch.uint8, device="cuda")
    odd = ops.Checkpoint(flat[1:].view(8, 96), torch.empty(8 * 3 + 1, dtype=torch.uint8, device="cuda")[1:].view(8, 3),
                         "e4m3")
    ops.mhc_ckpt_pack(x, "e4m3", out=odd)
    _same(odd, x)
    _reads_back(odd)


@pytest.mark.parametrize("T,H,pad", [(1, 64, 0), (5, 520, 0), (5, 264, 8), (3, 77, 0), (4, 1000, 3), (170, 512, 0),
                                     (3, 7168, 0), (2, 16416, 0)])
@pytest.mark.parametrize("types,gate,act,scale", [("bf16", "channel", "none", "channel"),
                                                  ("bf16+", "token", "sigmoid", "one"),
                                                  ("fp16", "full", "tanh", "none"), ("fp32", "none", "none", "channel")])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_the_block_through_its_checkpoints(T, H, pad, types, gate, act, scale, fmt):
    x, d, form = make(T, H, types, gate, act, scale, pad)
    p = params(act)
    cks = {k: ops.ckpt_empty(T, H, fmt) for k in ("ckpt_y", "ckpt_residual", "ckpt_h")}
    _, ro, h, rstd = check_forward(x, form, p, **cks)
    _same(cks["ckpt_y"], x["y"])
    _same(cks["ckpt_residual"], x["residual"])
    _same(cks["ckpt_h"], h)
    values = {"y": ref.unpack(cks["ckpt_y"].codes, cks["ckpt_y"].scales, fmt),
              "residual": ref.unpack(cks["ckpt_residual"].codes, cks["ckpt_residual"].scales, fmt)}
    check_backward(x, d, form, p, cks["ckpt_y"], cks["ckpt_residual"], rstd, values)
    # one of the two held, the other as it was
    check_backward(x, d, form, p, cks["ckpt_y"], None, rstd, {"y": values["y"]})
    check_backward(x, d, form, p, None, cks["ckpt_residual"], rstd, {"residual": values["residual"]})


def test_one_checkpoint_of_three():
    x, d, form = make(4, 544, "bf16", "none", "none", "none")
    for k, src in (("ckpt_y", "y"), ("ckpt_residual", "residual"), ("ckpt_h", None)):
        c = ops.ckpt_empty(4, 544, "e4m3")
        _, _, h, _ = check_forward(x, form, params(), **{k: c})
        _same(c, h if src is None else x[src])


# ------------------------------------------------------------------ the weight gradient


def _dw_bound(d, x, T, dtype, want):
    """Products are exact in fp32. A tensor core may cut each of 17 addends 2^-23
    below the largest, every 16 tokens; the sum of magnitudes bounds the largest."""
    err = (1.1 * T + 34) * 2.0 ** -23 * (d.abs().t() @ x.abs())
    return err + ref.half_step(dtype) * (want.abs() + err) + ref.tiny(dtype)


def _check_dw(T, N, K, dt, fmt, out, pad=0, offset=0, accumulate=False, std=0.05):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + N * 7 + K)
    flat = torch.randn(T * (N + pad) + offset, generator=g, device="cuda").mul_(std).to(dt)
    d = flat[offset:].view(T, N + pad)[:, :N]
    c = ops.mhc_ckpt_pack(torch.randn(T, K, generator=g, device="cuda"), fmt)
    x = ref.unpack(c.codes, c.scales, fmt)
    want = d.double().t() @ x
    kw = {"dtype": out}
    if accumulate:
        kw = {"d_w": torch.randn(N, K, generator=g, device="cuda").to(out), "accumulate": True}
        want = want + kw["d_w"].double()
    bound = _dw_bound(d.double(), x, T, out, want)
    if accumulate:
        bound = bound + 2.0 ** -23 * want.abs()
    within(ops.mhc_ckpt_linear_dw(d, c, **kw), want, bound, "d_w")


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 32, 32), (3, 17, 45), (16, 128, 256), (64, 128, 256), (65, 129, 257),
                                   (63, 127, 255), (200, 256, 512), (333, 519, 1096), (1000, 96, 40), (129, 640, 33),
                                   (512, 1024, 512), (77, 8, 2000), (5, 2000, 8)])
@pytest.mark.parametrize("dt,fmt,out", [("bf16", "e4m3", "fp32"), ("bf16", "int8", "bf16"), ("fp16", "int8", "fp32"),
                                        ("fp16", "e4m3", "fp16")])
def test_weight_gradient(T, N, K, dt, fmt, out):
    _check_dw(T, N, K, TYPES[dt], fmt, TYPES[out])


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (16, 8), (1, 7)])
def test_weight_gradient_of_strided_rows(pad, offset):
    _check_dw(150, 200, 96, BF, "e4m3", FP32, pad, offset)


def test_weight_gradient_of_one_row_for_every_token():
    d = torch.randn(1, 136, device="cuda").to(BF).expand(70, 136)
    c = ops.mhc_ckpt_pack(torch.randn(70, 264, device="cuda"), "int8")
    x = ref.unpack(c.codes, c.scales, "int8")
    want = d.double().t() @ x
    within(ops.mhc_ckpt_linear_dw(d, c), want, _dw_bound(d.double(), x, 70, FP32, want), "d_w")


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("N,K", [(130, 288), (67, 51)])
def test_weight_gradient_added_to_what_is_there(out, N, K):
    _check_dw(90, N, K, BF, "int8", TYPES[out], accumulate=True)


def test_weight_gradient_is_exact_for_small_whole_numbers():
    """Sums below 2^24 of whole numbers: no rounding anywhere, so a product
    that is missing, doubled or misplaced shows. Long and short sums, many tiles."""
    for T, N, K in ((1, 300, 520), (100, 300, 520), (8192, 136, 264), (515, 1288, 2056)):
        g = torch.Generator(device="cuda").manual_seed(T)
        d = torch.randint(-4, 5, (T, N), generator=g, device="cuda").to(BF)
        x = torch.randint(-15, 16, (T, K), generator=g, device="cuda").float()
        c = ops.mhc_ckpt_pack(x, "int8")
        assert torch.equal(ops.mhc_ckpt_unpack(c, FP32), x)
        want = (d.double().t() @ x.double()).float()
        assert torch.equal(ops.mhc_ckpt_linear_dw(d, c), want)


@pytest.mark.parametrize("K", [1288, 1283])
def test_weight_gradient_of_many_tokens_in_one_sum(K):
    """Tiles enough that the tokens are not split: sums in several pieces, exact
    for whole numbers, and for values of one sign off by no more than the cuts of a piece."""
    T, N = 4209, 2048
    g = torch.Generator(device="cuda").manual_seed(K)
    d = torch.randint(-4, 5, (T, N), generator=g, device="cuda").to(BF)
    c = ops.mhc_ckpt_pack(torch.randint(-15, 16, (T, K), generator=g, device="cuda").float(), "int8")
    want = d.double().t() @ ops.mhc_ckpt_unpack(c, FP32).double()
    assert torch.equal(ops.mhc_ckpt_linear_dw(d, c), want.float())
    assert torch.equal(ops.mhc_ckpt_linear_dw(d, c, d_w=torch.empty(N, K, dtype=BF, device="cuda")), want.to(BF))
    d = torch.rand(T, N, generator=g, device="cuda").to(BF)
    c = ops.mhc_ckpt_pack(torch.rand(T, K, generator=g, device="cuda"), "e4m3")
    want = d.double().t() @ ref.unpack(c.codes, c.scales, "e4m3")
    # 32 products of 16 tokens to a piece of 512, each of which may cut 2^-23 of
    # the sum so far twice; then 9 pieces rounded to nearest
    bound = want * (32 * 2 * 2.0 ** -23 + 9 * 2.0 ** -24)
    assert ((ops.mhc_ckpt_linear_dw(d, c).double() - want).abs() <= bound).all()


def test_weight_gradient_of_no_tokens_and_refusals():
    c = ops.mhc_ckpt_pack(torch.empty(0, 64, dtype=BF, device="cuda"))
    d = torch.empty(0, 48, dtype=BF, device="cuda")
    assert (ops.mhc_ckpt_linear_dw(d, c) == 0).all()
    w = torch.ones(48, 64, device="cuda")
    assert (ops.mhc_ckpt_linear_dw(d, c, d_w=w, accumulate=True) == 1).all()
    c = ops.mhc_ckpt_pack(torch.randn(4, 64, device="cuda"))
    d = torch.randn(4, 48, device="cuda").to(BF)
    with pytest.raises(ValueError, match="bfloat16"):
        ops.mhc_ckpt_linear_dw(d.float(), c)
    with pytest.raises(ValueError, match="x must"):
        ops.mhc_ckpt_linear_dw(d[:3], c)
    with pytest.raises(ValueError, match="accumulate"):
        ops.mhc_ckpt_linear_dw(d, c, accumulate=True)
    with pytest.raises(ValueError, match="d_w"):
        ops.mhc_ckpt_linear_dw(d, c, d_w=w[:40])


def test_not_a_number_stays_in_its_rows_and_columns():
    x = torch.randn(40, 96, device="cuda")
    x[7, 40] = float("nan")                     # its group: columns 32 .. 63
    d = torch.randn(40, 72, device="cuda").to(BF)
    got = ops.mhc_ckpt_linear_dw(d, ops.mhc_ckpt_pack(x))
    assert torch.isnan(got[:, 32:64]).all() and torch.isfinite(got[:, :32]).all() and torch.isfinite(got[:, 64:]).all()


@pytest.mark.parametrize("T,N,K", [(300, 264, 520), (45, 31, 77)])
def test_weight_gradient_run_to_run_on_a_stream_and_captured(T, N, K):
    d = torch.randn(T, N, device="cuda").to(BF)
    c = ops.mhc_ckpt_pack(torch.randn(T, K, device="cuda"), "int8")
    want = ops.mhc_ckpt_linear_dw(d, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.mhc_ckpt_linear_dw(d, c, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.mhc_ckpt_linear_dw(d, c)
    d.copy_(torch.randn(T, N, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ops.mhc_ckpt_linear_dw(d, c))
    assert ops.mhc_get_device_status() == 0
