"""The gated residual block on the GPU: forward and backward against the
plain 64-bit forms within the bounds that tests/block_ref.py derives."""
import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = {"bf16": (BF, BF), "bf16+": (BF, FP32), "fp16": (FP16, FP16), "fp16+": (FP16, FP32),
         "fp32": (FP32, FP32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


def _rows(g, T, H, dtype, std=1.0, pad=0, offset=0):
    """[T, H] with rows `pad` further apart, `offset` elements into its storage."""
    flat = torch.randn(T * (H + pad) + offset, generator=g, device="cuda").mul_(std).to(dtype)
    return flat[offset:].view(T, H + pad)[:, :H]


def make(T, H, types="bf16", gate="channel", act="none", scale="channel", pad=0, offset=0, seed=0,
         w_dtype=FP32, gate_dtype=None):
    g = torch.Generator(device="cuda").manual_seed(1000 * T + H + seed)
    dt, rt = PAIRS[types]
    gt = gate_dtype or (dt if gate == "full" else FP32)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {"y": _rows(g, T, H, dt, 1.5, pad, offset), "residual": _rows(g, T, H, rt, 2.0, pad, offset),
         "w_post": (1 + 0.2 * rand(H)).to(w_dtype), "w_pre": (1 + 0.2 * rand(H)).to(w_dtype),
         "gate": {"none": lambda: None, "channel": lambda: rand(H).to(gt), "token": lambda: rand(T, 1).to(gt),
                  "full": lambda: _rows(g, T, H, gt, 1.0, pad, offset)}[gate](),
         "res_scale": {"none": lambda: None, "one": lambda: 0.9 + 0.1 * rand(1),
                       "channel": lambda: 0.9 + 0.1 * rand(H)}[scale]()}
    d = {"d_ro": _rows(g, T, H, rt, 0.02, pad, offset), "d_h": _rows(g, T, H, dt, 0.05, pad, offset)}
    return x, d, {"gate": gate, "scale": scale, "act": act}


def params(act="none", **kw):
    return ops.BlockParams(gate_act=act, **kw)


def within(got, want, bound, what):
    far = (got.double() - want).abs() > bound
    assert not far.any(), (what, int(far.sum()), float((got.double() - want).abs().max()))
    assert torch.isfinite(got).all(), what


def check_forward(x, form, p, out=None, **kw):
    T, H = x["y"].shape
    f = ref.block(**x, eps_post=p.eps_post, eps_pre=p.eps_pre, gate_act=form["act"],
                  weight_offset=p.weight_offset, post_norm=p.post_norm)
    ro, h, rstd = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"],
                                     p, **kw)
    b = ref.forward_bounds(f, h.dtype, ro.dtype)
    within(ro, f["ro"], b["residual_out"], "residual_out")
    within(h, f["h"], b["h"], "h")
    within(rstd, f["rstd"], b["rstd"], "rstd")
    return f, ro, h, rstd


def check_backward(x, d, form, p, y=None, residual=None, rstd=None, values=None, **kw):
    T, H = x["y"].shape
    dt, rt = x["y"].dtype, x["residual"].dtype
    if rstd is None:
        rstd = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)[2]
    f = ref.block(**{**x, **(values or {})}, eps_post=p.eps_post, eps_pre=p.eps_pre, gate_act=form["act"],
                  weight_offset=p.weight_offset, post_norm=p.post_norm)
    if not p.post_norm:
        rstd_post = torch.ones_like(rstd[:, :1])
    else:
        rstd_post = rstd[:, :1]
    # what the kernel forms residual_out from: the kept rstd
    f["n"] = f["y"] * rstd_post.double() * f["w1"]
    f["ro"] = f["a"] * f["r"] + f["g"] * f["n"]
    kept = torch.cat((rstd_post, rstd[:, 1:]), 1)
    want, size = ref.backward(f, d["d_ro"], d["d_h"], kept, form["gate"], form["scale"], form["act"], p.post_norm)
    got = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"] if y is None else y,
                                      x["residual"] if residual is None else residual, rstd, x["w_post"],
                                      x["w_pre"], x["gate"], x["res_scale"], p, **kw)
    gt = None if x["gate"] is None else x["gate"].dtype
    b = ref.backward_bounds(want, size, T, H, dt, rt, form["gate"], gt)
    for k, v in want.items():
        if (k == "d_w_post" and x["w_post"] is None) or (k == "d_w_pre" and x["w_pre"] is None):
            assert getattr(got, k) is None
            continue
        within(getattr(got, k), v, b[k], k)
    return got


# ------------------------------------------------------------------ forward and backward

SHAPES = [(1, 1), (2, 7), (3, 31), (1, 32), (5, 33), (4, 64), (2, 96), (3, 127), (1, 256), (7, 520), (2, 1000),
          (3, 1999), (4, 2048), (160, 1024), (2, 4104), (1, 7168), (9, 7168), (2, 8193), (1, 16384), (2, 16392),
          (1, 20000), (1, 65536)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("types", ["bf16", "fp32"])
def test_every_width(T, H, types):
    x, d, form = make(T, H, types, gate="full", act="sigmoid", scale="channel")
    p = params("sigmoid")
    _, _, _, rstd = check_forward(x, form, p)
    check_backward(x, d, form, p, rstd=rstd)


@pytest.mark.parametrize("types", list(PAIRS))
@pytest.mark.parametrize("gate,act", [("none", "none"), ("channel", "none"), ("channel", "tanh"),
                                      ("token", "sigmoid"), ("full", "none"), ("full", "tanh")])
@pytest.mark.parametrize("scale", ["none", "one", "channel"])
@pytest.mark.parametrize("T,H", [(5, 264), (3, 77)])
def test_every_form(T, H, types, gate, act, scale):
    x, d, form = make(T, H, types, gate, act, scale)
    p = params(act)
    _, _, _, rstd = check_forward(x, form, p)
    check_backward(x, d, form, p, rstd=rstd)


@pytest.mark.parametrize("T,H,pad,offset", [(6, 512, 8, 0), (6, 512, 3, 0), (6, 512, 0, 1), (6, 512, 8, 8),
                                            (5, 510, 2, 0), (300, 72, 1, 5)])
@pytest.mark.parametrize("types", ["bf16", "fp16+"])
def test_strides_and_offsets(T, H, pad, offset, types):
    x, d, form = make(T, H, types, "full", "sigmoid", "one", pad, offset)
    p = params("sigmoid")
    _, _, _, rstd = check_forward(x, form, p)
    check_backward(x, d, form, p, rstd=rstd)


def test_rows_and_gates_that_are_one_row():
    """Stride 0: the same row for every token."""
    x, d, form = make(9, 320, "bf16", "full", "sigmoid", "none")
    for k in ("y", "gate"):
        x[k] = x[k][:1].expand(9, 320)
    d["d_h"] = d["d_h"][:1].expand(9, 320)
    p = params("sigmoid")
    _, _, _, rstd = check_forward(x, form, p)
    check_backward(x, d, form, p, rstd=rstd)


@pytest.mark.parametrize("T", [151, 153, 305, 700])
def test_more_rows_than_blocks(T):
    for H, gate in ((256, "channel"), (1031, "token")):
        x, d, form = make(T, H, "bf16", gate, "sigmoid", "channel")
        p = params("sigmoid")
        _, _, _, rstd = check_forward(x, form, p)
        check_backward(x, d, form, p, rstd=rstd)


@pytest.mark.parametrize("T,H,types,gate,pad", [(3100, 1984, "fp32", "token", 16), (4000, 544, "bf16+", "full", 0),
                                                 (2500, 1032, "bf16", "channel", 0), (1900, 4096, "fp16", "token", 0),
                                                 (1100, 7168, "bf16", "full", 0), (1500, 2056, "bf16", "token", 3),
                                                 (2000, 1031, "fp16+", "full", 0)])
def test_many_rows_in_flight(T, H, types, gate, pad):
    """Rows staged ahead, many a block: groups of warps that share the stages go at
    their own pace, and each must find its own row in its stage every time."""
    x, d, form = make(T, H, types, gate, "sigmoid", "one", pad)
    p = params("sigmoid")
    args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
    _, ro, h, rstd = check_forward(x, form, p)
    got = check_backward(x, d, form, p, rstd=rstd)
    cold = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(12):
        cold.zero_()                                # the rows come from memory again, in no order
        again = ops.mhc_block_norm(x["y"], x["residual"], *args)
        for a, b in zip((ro, h, rstd), again):
            assert torch.equal(a, b)
        cold.zero_()
        for a, b in zip(got, ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], rstd, *args)):
            assert torch.equal(a, b)
    assert ops.mhc_get_device_status() == 0


@pytest.mark.parametrize("w_dtype", [FP32, BF, FP16])
@pytest.mark.parametrize("H", [640, 99])
def test_weight_types_offsets_and_missing_ones(w_dtype, H):
    x, d, form = make(4, H, "bf16", "channel", "none", "one", w_dtype=w_dtype, gate_dtype=BF)
    p = params(weight_offset=1.0, eps_post=1e-3, eps_pre=1e-2)
    _, _, _, rstd = check_forward(x, form, p)
    check_backward(x, d, form, p, rstd=rstd)
    x["w_post"] = None
    check_forward(x, form, p)
    check_backward(x, d, form, p)
    x["w_pre"] = None
    check_backward(x, d, form, p)
    # no norm after the block
    p = params(post_norm=False)
    check_forward(x, form, p)
    check_backward(x, d, form, p)


def test_no_gradient_of_the_stream():
    x, d, form = make(6, 512, "bf16+", "token", "tanh", "channel")
    d["d_ro"] = None
    check_backward(x, d, form, params("tanh"), residual_dtype=FP32)


def test_rows_of_zeros_and_of_large_values():
    for H in (512, 101):
        x, d, form = make(5, H, "bf16+", "channel", "none", "none")
        x["y"][1] = 0
        x["residual"][1] = 0                       # both norms of nothing: eps alone
        x["y"][2] = 0
        x["residual"][3] = 0
        x["y"][4] *= 1e15
        x["residual"][4] *= 1e-12
        p = params()
        _, ro, h, rstd = check_forward(x, form, p)
        assert (h[1] == 0).all() and (ro[1] == 0).all()
        check_backward(x, d, form, p, rstd=rstd)


def test_a_row_of_nan_or_infinity_stays_alone():
    for H in (512, 77):
        x, d, form = make(6, H, "bf16", "full", "sigmoid", "channel")
        p = params("sigmoid")
        clean = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
        bad = {k: (v.clone() if v is not None else None) for k, v in x.items()}
        bad["y"][2, 5] = float("nan")
        bad["residual"][4, 0] = float("inf")
        out = ops.mhc_block_norm(bad["y"], bad["residual"], bad["w_post"], bad["w_pre"], bad["gate"],
                                 bad["res_scale"], p)
        keep = [0, 1, 3, 5]
        for a, b in zip(clean, out):
            assert torch.equal(a[keep], b[keep])
        assert torch.isnan(out[1][2]).all()
        g0 = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], clean[2], x["w_post"],
                                         x["w_pre"], x["gate"], x["res_scale"], p)
        g1 = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], bad["y"], bad["residual"], out[2], x["w_post"],
                                         x["w_pre"], x["gate"], x["res_scale"], p)
        for k in ("d_y", "d_residual", "d_gate"):
            assert torch.equal(getattr(g0, k)[keep], getattr(g1, k)[keep]), k
        assert torch.isnan(g1.d_w_post).all()


def test_saturated_gates():
    """Far tails: the slope neither vanishes early nor turns to NaN."""
    for gate in ("channel", "token", "full"):
        for act in ("sigmoid", "tanh"):
            x, d, form = make(6, 128, "fp32", gate, act, "none")
            z = x["gate"].reshape(-1)
            vals = torch.tensor([-80.0, -30.0, -10.0, 10.0, 30.0, 0.0], device="cuda")
            z[:6] = vals
            p = params(act)
            _, _, _, rstd = check_forward(x, form, p)
            check_backward(x, d, form, p, rstd=rstd)


def test_no_tokens():
    x, d, form = make(1, 96, "bf16", "channel", "none", "one")
    e = {k: (v[:0] if k in ("y", "residual") else v) for k, v in x.items()}
    ro, h, rstd = ops.mhc_block_norm(e["y"], e["residual"], e["w_post"], e["w_pre"], e["gate"], e["res_scale"])
    assert ro.shape == h.shape == (0, 96) and rstd.shape == (0, 2)
    g = ops.mhc_block_norm_backward(d["d_ro"][:0], d["d_h"][:0], e["y"], e["residual"], rstd, e["w_post"],
                                    e["w_pre"], e["gate"], e["res_scale"])
    for k in ("d_w_post", "d_w_pre", "d_gate", "d_res_scale"):
        assert (getattr(g, k) == 0).all(), k
    z = torch.empty(0, 1, device="cuda")
    g = ops.mhc_block_norm_backward(d["d_ro"][:0], d["d_h"][:0], e["y"], e["residual"], rstd, gate=z)
    assert g.d_gate.shape == (0, 1) and g.d_w_post is None and g.d_res_scale is None


def test_in_place():
    for H in (512, 77):
        x, d, form = make(40, H, "bf16", "token", "sigmoid", "channel")
        p = params("sigmoid")
        args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
        want = ops.mhc_block_norm(x["y"], x["residual"], *args)
        r = x["residual"].contiguous().clone()
        got = ops.mhc_block_norm(x["y"], r, *args, residual_out=r)
        assert got[0] is r
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        gw = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], want[2], *args)
        dr = d["d_ro"].contiguous().clone()
        gg = ops.mhc_block_norm_backward(dr, d["d_h"], x["y"], x["residual"], want[2], *args, d_residual=dr)
        for a, b in zip(gw, gg):
            assert torch.equal(a, b)


def test_the_same_run_to_run_and_on_another_stream():
    x, d, form = make(500, 1032, "bf16", "channel", "sigmoid", "one")
    p = params("sigmoid")
    args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)

    def both(**kw):
        f = ops.mhc_block_norm(x["y"], x["residual"], *args, **kw)
        return [*f, *ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], f[2], *args, **kw)]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        got = both(stream=side if k % 2 else None)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("H", [1024, 333])
def test_captured_in_a_graph(H):
    x, d, form = make(33, H, "bf16", "full", "sigmoid", "channel")
    p = params("sigmoid")
    args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)

    def both():
        f = ops.mhc_block_norm(x["y"], x["residual"], *args)
        return [*f, *ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], f[2], *args)]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x["y"], x["residual"], d["d_ro"], d["d_h"]):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, both()):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the first, a middle and the last rows against the plain form."""
    T, H = 327_700, 6560
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(T, H, dtype=BF, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    ck = ops.ckpt_empty(T, H, "int8")
    ro, h, rstd = ops.mhc_block_norm(x, x, w, w, ckpt_y=ck)
    d = ops.mhc_block_norm_backward(x, x, ck, x, rstd, w, w)
    for at in (0, T // 2, T - 3):
        rows = x[at:at + 3]
        f = ref.block(rows, rows, w, w)
        b = ref.forward_bounds(f, BF, BF)
        within(ro[at:at + 3], f["ro"], b["residual_out"], "residual_out")
        within(h[at:at + 3], f["h"], b["h"], "h")
        codes, scales = ref.pack(rows, "int8")
        assert torch.equal(ck.codes[at:at + 3], codes) and torch.equal(ck.scales[at:at + 3], scales)
        f = ref.block(ref.unpack(codes, scales, "int8"), rows, w, w)
        f["n"] = f["y"] * rstd[at:at + 3, :1].double() * f["w1"]
        f["ro"] = f["r"] + f["n"]
        want, size = ref.backward(f, rows, rows, rstd[at:at + 3], "none", "none")
        b = ref.backward_bounds(want, size, T, H, BF, BF, "none", None)
        for k in ("d_y", "d_residual"):
            within(getattr(d, k)[at:at + 3], want[k], b[k], k)


def test_gradients_against_differences():
    """Central differences of the kernel's own forward pass. The outputs' sum is
    formed in 64 bits; a forward value is off by its bound, so a difference over
    2 e by at most the sum of the bounds over e, beside e^2 of the third derivative."""
    x, d, form = make(4, 88, "fp32", "token", "sigmoid", "channel")
    p = params("sigmoid")
    names = ("y", "residual", "w_post", "w_pre", "gate", "res_scale")

    def loss(**over):
        t = {**x, **over}
        ro, h, _ = ops.mhc_block_norm(*(t[k] for k in names), p)
        return float((ro.double() * d["d_ro"].double() + h.double() * d["d_h"].double()).sum())

    f = ref.block(**x, gate_act="sigmoid")
    b = ref.forward_bounds(f, FP32, FP32)
    noise = float((b["residual_out"] * d["d_ro"].double().abs() + b["h"] * d["d_h"].double().abs()).sum())
    rstd = ops.mhc_block_norm(*(x[k] for k in names), p)[2]
    got = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], rstd, x["w_post"], x["w_pre"],
                                      x["gate"], x["res_scale"], p)
    g = torch.Generator(device="cuda").manual_seed(5)
    e = 2.0 ** -6
    for k, grad in zip(names, got):
        v = torch.randn(x[k].shape, generator=g, device="cuda")
        v /= v.norm()

        def slope_at(step):
            return (loss(**{k: x[k] + step * v}) - loss(**{k: x[k] - step * v})) / (2 * step)

        s1, s2 = slope_at(e), slope_at(2 * e)
        # the e^2 term taken out by the two steps; what is left of it is below its own size
        best = (4 * s1 - s2) / 3
        want = float((grad.double() * v.double()).sum())
        assert abs(best - want) <= 2 * noise / e + abs(s1 - s2) + 1e-6 * abs(want), (k, best, want)


# ------------------------------------------------------------------ refusals of the binding


def test_refusals():
    x, d, form = make(4, 64, "bf16", "channel", "none", "one")
    y, r = x["y"], x["residual"]
    for args, kw, match in (((y, r[:3]), {}, "residual"), ((y, r[:, :32]), {}, "residual"),
                            ((y, r.half()), {}, "residual"), ((y.double(), r), {}, "float32"),
                            ((y.t(), r.t()), {}, "contiguous"),
                            ((y, r, x["w_post"][:3]), {}, "w_post"), ((y, r, None, x["w_post"].int()), {}, "w_pre"),
                            ((y, r, None, None, torch.zeros(3, device="cuda")), {}, "gate"),
                            ((y, r, None, None, x["gate"].half()), {}, "gate"),
                            ((y, r, None, None, None, torch.zeros(3, device="cuda")), {}, "res_scale"),
                            ((y, r, None, None, None, None, params("relu")), {}, "gate_act"),
                            ((y, r, None, None, None, None, params("tanh")), {}, "gate_act"),
                            ((y, r), {"h": r.float()}, "h must"), ((y, r), {"residual_out": r[:, :32]}, "residual_out"),
                            ((y, r), {"ckpt_y": ops.ckpt_empty(4, 32)}, "ckpt_y"),
                            ((y, r), {"ckpt_y": ops.ckpt_empty(4, 64), "ckpt_h": ops.ckpt_empty(4, 64, "int8")}, "format")):
        with pytest.raises(ValueError, match=match):
            ops.mhc_block_norm(*args, **kw)
    with pytest.raises(ops.MhcError, match="ALIAS"):
        ops.mhc_block_norm(y, r, h=y)
    with pytest.raises(ops.MhcError, match="SHAPE"):
        ops.mhc_block_norm(y, r, x["w_post"], params=params(post_norm=False))
    rstd = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError, match="rstd"):
        ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], y, r, rstd[:3])
    with pytest.raises(ValueError, match="y must"):
        ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], y.float(), r, rstd)
    with pytest.raises(ValueError, match="d_residual_out"):
        ops.mhc_block_norm_backward(d["d_ro"][:2], d["d_h"], y, r, rstd)
    with pytest.raises(ops.MhcError, match="WORKSPACE"):
        ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], y, r, rstd,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
