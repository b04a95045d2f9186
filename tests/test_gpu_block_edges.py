"""The gated residual block, the checkpoints and the weight gradient at the edges
of their range: long sums, infinities, values past fp16, one token, no tokens."""

import pytest
import torch

from manifold_constrained_hyper_gb300 import ops
from tests import block_ref as ref
from tests.test_gpu_block import BF, FP16, FP32, PAIRS, check_backward, check_forward, make, params, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from manifold_constrained_hyper_gb300 import build
    build.build()
    ops.load()


# ------------------------------------------------------------------ sums over tokens

# every way a row goes: staged on boundaries, off them (inputs alone, outputs too), from
# memory (the widest types), by the loop; with a full gate, and from checkpoints
SUMS = [(2047, 1102, "fp32", "full", 0, False), (1500, 1032, "bf16", "none", 0, False), (1500, 1032, "bf16", "token", 3, False),
        (1500, 2056, "fp16+", "channel", 0, True), (1200, 1031, "bf16+", "full", 0, True), (1300, 520, "bf16", "full", 8, True),
        (700, 7168, "fp32", "token", 0, False), (330, 8192, "fp32", "full", 0, False), (330, 7171, "fp32", "none", 0, False),
        (700, 8200, "bf16", "channel", 0, False), (700, 8203, "bf16", "none", 0, True), (4000, 64, "fp16", "none", 0, False)]


def _whole(g, T, H, dtype, lo, hi, pad=0):
    t = torch.randint(lo, hi, (T, H + pad), generator=g, device="cuda").to(dtype)
    return t[:, :H] if pad else t


@pytest.mark.parametrize("T,H,types,gate,pad,held", SUMS)
@pytest.mark.parametrize("scale", ["one", "channel"])
def test_sums_over_tokens_are_exact_for_whole_numbers(T, H, types, gate, pad, held, scale):
    """With d_h = 0 and whole numbers everywhere, D is d_residual_out and every term is a whole
    number. A column's sums stay below 2^24 and have to be exact; a single scale's sum passes
    2^24 by far: its thread's terms of a row are exact, and what joins them holds 48 bits, so
    that it is off by its own rounding alone."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    dt, rt = PAIRS[types]
    gt = dt if gate == "full" else FP32
    y, r = _whole(g, T, H, dt, -2, 3, pad), _whole(g, T, H, rt, 1, 128, pad)
    d_ro, d_h = _whole(g, T, H, rt, 1, 64, pad), torch.zeros(T, H, dtype=dt, device="cuda")
    w_post, w_pre = (_whole(g, 1, H, FP32, 1, 3)[0] for _ in range(2))
    z = {"none": lambda: None, "channel": lambda: _whole(g, 1, H, gt, -1, 2)[0], "token": lambda: _whole(g, T, 1, gt, -1, 2),
         "full": lambda: _whole(g, T, H, gt, -1, 2)}[gate]()
    a = torch.full((1,), 2.0, device="cuda") if scale == "one" else _whole(g, 1, H, FP32, 1, 3)[0]
    rstd = torch.ones(T, 2, device="cuda")
    args = (rstd, w_post, w_pre, z, a, params())
    f = {"y": ops.mhc_ckpt_pack(y, "int8") if held else y, "residual": ops.mhc_ckpt_pack(r, "int8") if held else r}
    got = ops.mhc_block_norm_backward(d_ro, d_h, f["y"], f["residual"], *args, residual_dtype=rt)
    Y, R, D = y.double(), r.double(), d_ro.double()
    gz = 1.0 if z is None else z.double()
    assert torch.equal(got.d_w_post, (gz * D * Y).sum(0).float())
    ds = R * D
    assert torch.equal(got.d_res_scale, (ds.sum(0) if scale == "channel" else ds.sum().reshape(1)).float())
    if z is not None and gate != "full":
        dg = Y * w_post.double() * D
        assert torch.equal(got.d_gate, (dg.sum(0) if gate == "channel" else dg.sum(1, keepdim=True)).float())
    # d_w_pre needs no D: whole numbers of d_h, ro = a r + g y w_post
    r = _whole(g, T, H, rt, -3, 4, pad)
    d_h = _whole(g, T, H, dt, -3, 4, pad)
    ro = a.double() * r.double() + gz * Y * w_post.double()
    got = ops.mhc_block_norm_backward(None, d_h, f["y"], ops.mhc_ckpt_pack(r, "int8") if held else r, *args, residual_dtype=rt)
    assert torch.equal(got.d_w_pre, (d_h.double() * ro).sum(0).float())


@pytest.mark.parametrize("T,H,types,gate,pad,held", SUMS)
def test_single_scale_gradient_of_a_stream(T, H, types, gate, pad, held):
    """A gradient with a part along the stream, as a loss's has: the sum is of the size of its
    magnitudes. Each D passes two row sums (2 steps(H) roundings); then a thread adds at most 16
    columns of a row, or a column of at most T / 152 + 1 rows, and the rest holds 48 bits."""
    x, d, form = make(T, H, types, gate, "sigmoid" if gate != "none" else "none", "one", pad)
    p = params(form["act"])
    d["d_ro"].add_((0.05 * x["residual"].float()).to(d["d_ro"].dtype))
    rstd = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)[2]
    y, r, values = x["y"], x["residual"], {}
    if held:
        y, r = ops.mhc_ckpt_pack(y, "e4m3"), ops.mhc_ckpt_pack(r, "e4m3")
        values = {"y": ref.unpack(y.codes, y.scales, "e4m3"), "residual": ref.unpack(r.codes, r.scales, "e4m3")}
    f = ref.block(**{**x, **values}, gate_act=form["act"])
    f["n"] = f["y"] * rstd[:, :1].double() * f["w1"]
    f["ro"] = f["a"] * f["r"] + f["g"] * f["n"]
    want, size = ref.backward(f, d["d_ro"], d["d_h"], rstd, gate, "one", form["act"])
    got = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], y, r, rstd, x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
    bound = (2 * ref.steps(H) + 16 + T / 152 + 1) * ref.EPS * size["d_res_scale"] + ref.EPS * want["d_res_scale"].abs()
    assert bound < 1e-3 * want["d_res_scale"].abs()             # a sum that is missing a part shows
    within(got.d_res_scale, want["d_res_scale"], bound, "d_res_scale")


# ------------------------------------------------------------------ the widest rows, many a block


@pytest.mark.parametrize("T,H,types,gate,scale,pad", [(400, 7168, "fp32", "token", "one", 0), (400, 7168, "fp32", "full", "channel", 0),
                                                      (400, 8192, "fp32", "full", "one", 0), (400, 8192, "fp32", "none", "none", 3),
                                                      (400, 7168, "fp32", "full", "one", 3), (400, 8184, "bf16+", "full", "channel", 0),
                                                      (320, 8191, "fp32", "token", "channel", 0), (400, 5600, "fp32", "full", "none", 0)])
@pytest.mark.parametrize("held", [False, True])
def test_rows_of_which_two_do_not_fit_shared_memory(T, H, types, gate, scale, pad, held):
    x, d, form = make(T, H, types, gate, "none" if gate == "none" else "sigmoid", scale, pad)
    p = params(form["act"])
    cks = {k: ops.ckpt_empty(T, H, "int8") for k in ("ckpt_y", "ckpt_residual")} if held else {}
    _, _, _, rstd = check_forward(x, form, p, **cks)
    if not held:
        return check_backward(x, d, form, p, rstd=rstd)
    values = {k[5:]: ref.unpack(c.codes, c.scales, "int8") for k, c in cks.items()}
    for k, c in cks.items():
        codes, scales = ref.pack(x[k[5:]], "int8")
        assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales)
    check_backward(x, d, form, p, cks["ckpt_y"], cks["ckpt_residual"], rstd, values)


# ------------------------------------------------------------------ values past fp16


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [64, 77])
def test_finite_values_stay_finite_in_fp16(fmt, H):
    """What a checkpoint of fp16's largest values stands for may be 65536: read back as the
    largest fp16 value, and so are a wider stream's values past it."""
    x = torch.zeros(6, H, device="cuda")
    x[0, 3], x[1, 40], x[2, :] = 65504.0, -65504.0, torch.linspace(62000, 65504, H, device="cuda")
    x[3, 5], x[4, H - 1], x[5, 0] = 1e6, -3e38, 65519.0
    for t in (x.clamp(-65504, 65504).half(), x):
        c = ops.mhc_ckpt_pack(t, fmt)
        want = ref.unpack(c.codes, c.scales, fmt).clamp(-65504.0, 65504.0).half()
        assert torch.equal(ops.mhc_ckpt_unpack(c, FP16), want)
    x[1, 0] = float("nan")
    got = ops.mhc_ckpt_unpack(ops.mhc_ckpt_pack(x, fmt), FP16)
    assert torch.isnan(got[1, :32]).all() and torch.isfinite(got[1, 32:]).all() and torch.isfinite(got[0]).all()


@pytest.mark.parametrize("fmt,h", [("e4m3", 7), ("int8", 9)])
@pytest.mark.parametrize("T,N,K,pad", [(70, 40, 96, 0), (333, 264, 200, 3), (1300, 136, 264, 0), (45, 31, 77, 1),
                                       (2100, 2048, 1288, 0), (2100, 2048, 1288, 8), (1, 64, 64, 0), (40001, 24, 72, 0)])
def test_fp16_weight_gradient_of_any_range(fmt, h, T, N, K, pad):
    """x in fp16 shares a power of two in 32 columns, whose largest scale 2^k becomes 2^h there:
    at the ends of fp16's range, past it and below it the products are what they are elsewhere.
    What lies 2^(h + 24) below a column's scale is rounded, by 2^(k - h - 25) at most."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    d = (0.05 * torch.randn(T, N + pad, generator=g, device="cuda")).half()[:, :N]
    x = torch.randn(T, K, generator=g, device="cuda")
    top = x.clamp(-1, 1) * 65504
    top[T // 2, 0], top[0, K - 1] = 65504.0, -65504.0
    wide = x * torch.exp2(torch.randint(-100, 100, (1, K), generator=g, device="cuda").float())
    loud = x * torch.exp2(torch.randint(-8, 12, (T, 1), generator=g, device="cuda").float())
    for v in (top.half(), wide, loud.bfloat16(), x * 2.0 ** -60):
        c = ops.mhc_ckpt_pack(v, fmt)
        held = ref.unpack(c.codes, c.scales, fmt)
        want = d.double().t() @ held
        k = (c.scales.max(0).values.double() - 127).repeat_interleave(32)[:K]
        for out in (FP32, BF):
            err = (1.1 * T + 34) * 2.0 ** -23 * (d.double().abs().t() @ held.abs())
            err = err + torch.exp2(k - h - 25) * d.double().abs().sum(0)[:, None]
            bound = err + ref.half_step(out) * (want.abs() + err) + ref.tiny(out)
            within(ops.mhc_ckpt_linear_dw(d, c, dtype=out), want, bound, "d_w")
    w = torch.randn(N, K, generator=g, device="cuda")
    c = ops.mhc_ckpt_pack(top, fmt)
    held = ref.unpack(c.codes, c.scales, fmt)
    want = d.double().t() @ held + w.double()
    err = (1.1 * T + 36) * 2.0 ** -23 * (d.double().abs().t() @ held.abs() + w.double().abs())
    within(ops.mhc_ckpt_linear_dw(d, c, d_w=w.clone(), accumulate=True), want, err, "d_w")


def test_fp16_weight_gradient_of_a_group_that_is_not_a_number():
    x = torch.randn(40, 96, device="cuda")
    x[7, 40] = float("inf")                     # its group: columns 32 .. 63
    d = torch.randn(40, 72, device="cuda").half()
    got = ops.mhc_ckpt_linear_dw(d, ops.mhc_ckpt_pack(x))
    assert torch.isnan(got[:, 32:64]).all() and torch.isfinite(got[:, :32]).all() and torch.isfinite(got[:, 64:]).all()
    x[:, 32:64] = float("nan")                  # no scale at all in these columns
    got = ops.mhc_ckpt_linear_dw(d, ops.mhc_ckpt_pack(x))
    assert torch.isnan(got[:, 32:64]).all() and torch.isfinite(got[:, :32]).all() and torch.isfinite(got[:, 64:]).all()


# ------------------------------------------------------------------ infinities

ROWS = [(6, 264, 0), (400, 1032, 0), (400, 1032, 3), (6, 77, 0), (400, 333, 0), (4, 8200, 0), (4, 8203, 0), (400, 72, 0)]


def _same_kind(got, want, what):
    """NaN and the infinities where they are in `want`, which is in 64 bits."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), what
    assert torch.equal(got.double()[inf], want[inf]), what


@pytest.mark.parametrize("T,H,pad", ROWS)
@pytest.mark.parametrize("types", ["bf16", "fp32"])
@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("held", [False, True])
def test_an_infinity_does_the_same_in_every_column(T, H, pad, types, post_norm, held):
    for name, gate, scale in (("residual", "none", "none"), ("residual", "full", "channel"), ("y", "channel", "one")):
        x, _, form = make(T, H, types, gate, "none", scale, pad)
        if gate == "channel":
            x["gate"] = x["gate"].abs() + 0.5
        for i, c in enumerate((0, H // 2, H - 9, H - 1)):
            x[name][i % T, c] = float("inf")
        if not post_norm:
            x["w_post"] = None
        kw = {"ckpt_h": ops.ckpt_empty(T, H, "int8")} if held else {}
        ro, h, rstd = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"],
                                         params(post_norm=post_norm), **kw)
        f = ref.block(**x, post_norm=post_norm)
        _same_kind(ro, f["ro"], (name, "residual_out"))
        _same_kind(rstd, f["rstd"], (name, "rstd"))
        _same_kind(h, f["h"], (name, "h"))
        bad = ~torch.isfinite(f["ro"]).all(1)
        assert (h[bad][torch.isfinite(h[bad])] == 0).all()
        if held:
            codes, scales = ref.pack(h, "int8")
            assert torch.equal(kw["ckpt_h"].scales, scales) and torch.equal(kw["ckpt_h"].codes, codes)


@pytest.mark.parametrize("T,H,pad", ROWS)
@pytest.mark.parametrize("types", ["bf16", "fp32"])
@pytest.mark.parametrize("gate,scale,held", [("none", "none", False), ("full", "channel", False), ("full", "one", False),
                                             ("token", "channel", True), ("none", "one", True)])
def test_a_gradient_s_infinity_does_the_same_in_every_column(T, H, pad, types, gate, scale, held):
    """An infinite gradient of residual_out leaves its row's other d_residual alone and makes
    d_y infinite; one of h makes the row's d_residual infinite."""
    for name, which in (("d_ro", ("d_residual", "d_y")), ("d_h", ("d_residual",))):
        x, d, form = make(T, H, types, gate, "none" if gate == "none" else "sigmoid", scale, pad)
        p = params(form["act"])
        rstd = ops.mhc_block_norm(x["y"], x["residual"], x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)[2]
        for i, c in enumerate((0, H // 2, H - 9, H - 1)):
            # nothing else in this row's sum is infinite, and nothing at its place is zero
            x["y"][i % T, c], x["residual"][i % T, c], x["w_post"][c], x["w_pre"][c] = 1.0, 1.0, 1.0, 1.0
            if gate == "full":
                x["gate"][i % T, c] = 1.0
            d[name][i % T, c] = float("inf")
        y, r, values = x["y"], x["residual"], {}
        if held:
            y, r = ops.mhc_ckpt_pack(y, "int8"), ops.mhc_ckpt_pack(r, "int8")
            values = {"y": ref.unpack(y.codes, y.scales, "int8"), "residual": ref.unpack(r.codes, r.scales, "int8")}
        f = ref.block(**{**x, **values}, gate_act=form["act"])
        f["n"] = f["y"] * rstd[:, :1].double() * f["w1"]
        f["ro"] = f["a"] * f["r"] + f["g"] * f["n"]
        want, _ = ref.backward(f, d["d_ro"], d["d_h"], rstd, gate, scale, form["act"])
        got = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], y, r, rstd, x["w_post"], x["w_pre"], x["gate"],
                                          x["res_scale"], p)
        for k in which:
            # a checkpoint's zero times an infinity is NaN in both
            _same_kind(getattr(got, k), want[k], (name, k))


# ------------------------------------------------------------------ one token, no tokens


@pytest.mark.parametrize("H", [512, 77])
def test_one_token_in_place_in_wider_rows(H):
    """One row has no stride: a slice of wider rows is updated where it lies."""
    for types in ("bf16", "bf16+"):
        x, d, form = make(1, H, types, "token", "sigmoid", "channel")
        p = params("sigmoid")
        args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
        want = ops.mhc_block_norm(x["y"], x["residual"], *args)
        wide = torch.zeros(3, H + 24, dtype=x["residual"].dtype, device="cuda")
        r = wide[:1, :H]
        r.copy_(x["residual"])
        got = ops.mhc_block_norm(x["y"], r, *args, residual_out=r)
        assert got[0] is r and all(torch.equal(a, b) for a, b in zip(want, got))
        gw = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], want[2], *args)
        dr = wide[1:2, :H]
        dr.copy_(d["d_ro"])
        gg = ops.mhc_block_norm_backward(dr, d["d_h"], x["y"], x["residual"], want[2], *args, d_residual=dr)
        assert all(torch.equal(a, b) for a, b in zip(gw, gg))
        assert (wide[2] == 0).all() and (wide[:2, H:] == 0).all()
    with pytest.raises(ops.MhcError, match="ALIAS"):
        ops.mhc_block_norm(x["y"], wide[:1, :H], *args, residual_out=wide[:1, 4:H + 4])


def test_no_tokens_read_nothing():
    """Sums over no tokens are zeros whatever the weights and the gate hold, a gate that is
    not there among them."""
    from tests.test_block_cpu import _back, _block
    H = 96
    grads = {k: torch.full((H,), 7.0, device="cuda") for k in ("dw1", "dw2", "dg", "ds")}
    w = torch.full((H,), float("nan"), device="cuda")
    gate = torch.full((H,), float("inf"), device="cuda")
    for g in (None, gate.data_ptr()):
        for act in (0, 1):
            for t in grads.values():
                t.fill_(7.0)
            b = _block(tokens=0, hidden=H, w_post=w.data_ptr(), w_pre=w.data_ptr(), gate=g, gate_act=act, res_scale=None)
            torch.cuda.synchronize()
            assert _back(ops.load(), b, dr=None, dh=None, y=None, r=None, rstd=None, dy=None, dres=None, ws=None, wsb=0,
                         **{k: t.data_ptr() for k, t in grads.items()}) == 0
            torch.cuda.synchronize()
            for k, t in grads.items():
                assert (t == 0).all(), (k, g, act)


# ------------------------------------------------------------------ what the binding gives and takes


def test_outputs_have_storages_of_their_own():
    """What is kept of a small call holds nothing else, and what is freed frees nothing else."""
    x, d, form = make(8, 256, "bf16", "full", "sigmoid", "one")
    p = params("sigmoid")
    args = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
    out = ops.mhc_block_norm(x["y"], x["residual"], *args)
    for t in out:
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
    g = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], out[2], *args)
    for t in (g.d_y, g.d_residual, g.d_gate):
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
    # the fp32 gradients of the parameters alone are together
    assert g.d_w_post.untyped_storage().nbytes() < 3 * 256 * 4 + 3 * 256
    c = ops.mhc_ckpt_pack(x["y"])
    d_w = ops.mhc_ckpt_linear_dw(d["d_h"], c)
    assert d_w.storage_offset() == 0 and d_w.untyped_storage().nbytes() == d_w.numel() * 4


def test_gradients_do_not_go_missing():
    """No call records a history: tensors whose gradients are being recorded are refused where
    these would end without a word."""
    x, d, form = make(4, 64, "bf16", "full", "sigmoid", "one")
    p = params("sigmoid")
    names = ("y", "residual", "w_post", "w_pre", "gate", "res_scale")
    want = ops.mhc_block_norm(*(x[k] for k in names), p)
    for k in names:
        t = {**x, k: x[k].detach().clone().requires_grad_()}
        with pytest.raises(ValueError, match="grad"):
            ops.mhc_block_norm(*(t[n] for n in names), p)
        with torch.no_grad():
            got = ops.mhc_block_norm(*(t[n] for n in names), p)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    rest = (x["w_post"], x["w_pre"], x["gate"], x["res_scale"], p)
    for k in ("d_ro", "d_h"):
        t = {**d, k: d[k].clone().requires_grad_()}
        with pytest.raises(ValueError, match="grad"):
            ops.mhc_block_norm_backward(t["d_ro"], t["d_h"], x["y"], x["residual"], want[2], *rest)
    # of the forward pass's own inputs the gradients are what is asked for
    w = x["w_post"].clone().requires_grad_()
    ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], want[2], w, *rest[1:])
    c = ops.mhc_ckpt_pack(x["y"])
    with pytest.raises(ValueError, match="grad"):
        ops.mhc_ckpt_linear_dw(d["d_h"].clone().requires_grad_(), c)
    with torch.no_grad():
        ops.mhc_ckpt_linear_dw(d["d_h"].clone().requires_grad_(), c)

    class Block(torch.autograd.Function):
        """The pair as a user wraps it."""

        @staticmethod
        def forward(ctx, y, r, w_post, w_pre, gate, scale):
            ro, h, rstd = ops.mhc_block_norm(y, r, w_post, w_pre, gate, scale, p)
            ctx.save_for_backward(y, r, rstd, w_post, w_pre, gate, scale)
            return ro, h

        @staticmethod
        def backward(ctx, d_ro, d_h):
            y, r, rstd, *rest = ctx.saved_tensors
            return tuple(ops.mhc_block_norm_backward(d_ro, d_h, y, r, rstd, *rest, p))

    t = {k: x[k].detach().clone().requires_grad_() for k in names}
    ro, h = Block.apply(*(t[k] for k in names))
    torch.autograd.backward((ro, h), (d["d_ro"], d["d_h"]))
    for k, v in zip(names, ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], want[2], *rest)):
        assert torch.equal(t[k].grad, v.to(x[k].dtype)), k


def test_a_workspace_is_device_bytes():
    """Refused before anything is launched: the workspace's address goes to the kernels."""
    x, d, form = make(4, 64, "bf16", "none", "none", "none")
    rstd = torch.ones(4, 2, device="cuda")
    n = ops.block_norm_backward_workspace_bytes(4, 64)
    c = ops.mhc_ckpt_pack(x["y"])
    m = ops.ckpt_linear_dw_workspace_bytes(4, 64, 64)
    for bad in (lambda k: torch.empty(k, dtype=torch.uint8), lambda k: torch.empty(2 * k, dtype=torch.uint8, device="cuda")[::2],
                lambda k: torch.empty(k, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], rstd, workspace=bad(n))
        with pytest.raises(ValueError, match="workspace"):
            ops.mhc_ckpt_linear_dw(d["d_h"], c, workspace=bad(m))
    want = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], rstd)
    got = ops.mhc_block_norm_backward(d["d_ro"], d["d_h"], x["y"], x["residual"], rstd,
                                      workspace=torch.empty(n // 4 + 1, device="cuda"))
    assert torch.equal(want.d_y, got.d_y)


def test_an_allocation_that_fails_raises_torch_s_error():
    """More than the device holds: what a program that shrinks its batch catches."""
    with pytest.raises(torch.cuda.OutOfMemoryError):
        ops.ckpt_empty(1 << 25, 65536)
    x = torch.randn(4, 64, device="cuda")
    assert ops.mhc_ckpt_unpack(ops.mhc_ckpt_pack(x, "int8"), FP32).shape == x.shape
