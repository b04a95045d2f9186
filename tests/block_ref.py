"""Plain 64-bit forms of the gated residual block, its backward pass and the
8-bit checkpoints, and how far a 32-bit evaluation may be from them.

EPS is half a step of fp32 relative to a value. A sum of H values by a block
of threads is off by at most (values per thread + 10 for the tree) EPS times
the sum of magnitudes; `steps` below counts that and the handful of products
around it. An output's own rounding is half a step of its type."""
import torch

EPS = 2.0 ** -24
GROUP = 32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def steps(H):
    """Roundings on the way of one term through a row's sum and the products
    around it: a thread adds at most max(64, H / 512) values, the tree at most
    10 more, and the terms and what they multiply are rounded some 20 times."""
    return 30 + max(64, H / 512)


def tiny(dtype):
    """Half of the least subnormal."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def act(z, name):
    if name == "sigmoid":
        return torch.sigmoid(z)
    if name == "tanh":
        return torch.tanh(z)
    return z


def slope(z, name):
    if name == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    if name == "tanh":
        return 1 / torch.cosh(z) ** 2
    return torch.ones_like(z)


def block(y, residual, w_post=None, w_pre=None, gate=None, res_scale=None, *, eps_post=1e-6,
          eps_pre=1e-6, gate_act="none", weight_offset=0.0, post_norm=True):
    """Everything of the forward pass, in 64 bits."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    y, r = d(y), d(residual)
    one = torch.ones(1, dtype=torch.float64, device=y.device)
    w1 = one if w_post is None else d(w_post) + weight_offset
    w2 = one if w_pre is None else d(w_pre) + weight_offset
    a = one if res_scale is None else d(res_scale)
    z = None if gate is None else d(gate)
    g = one if z is None else act(z, gate_act)
    rstd1 = (y.square().mean(1, keepdim=True) + eps_post).rsqrt() if post_norm \
        else torch.ones(y.shape[0], 1, dtype=torch.float64, device=y.device)
    n = y * rstd1 * w1
    ro = a * r + g * n
    rstd2 = (ro.square().mean(1, keepdim=True) + eps_pre).rsqrt()
    return {"y": y, "r": r, "w1": w1, "w2": w2, "a": a, "z": z, "g": g, "n": n, "ro": ro,
            "h": ro * rstd2 * w2, "rstd": torch.cat((rstd1, rstd2), 1),
            "size": (a * r).abs() + (g * n).abs(), "eps_pre": eps_pre}


def forward_bounds(f, dtype, r_dtype):
    """How far residual_out, h and rstd may be."""
    H = f["y"].shape[1]
    C = steps(H) * EPS
    dro = C * f["size"]
    ro, rstd2 = f["ro"], f["rstd"][:, 1:]
    # of rstd_pre, relative: half of that of the mean square
    rel2 = (ro.abs() * dro).sum(1, keepdim=True) / (ro.square().sum(1, keepdim=True) + H * f["eps_pre"]) + C
    h = f["h"]
    return {"residual_out": dro + half_step(r_dtype) * (ro.abs() + dro) + tiny(r_dtype),
            "h": (dro * rstd2 * f["w2"].abs() + (rel2 + C) * h.abs()) * (1 + half_step(dtype))
            + half_step(dtype) * h.abs() + tiny(dtype),
            "rstd": torch.cat((C * f["rstd"][:, :1], (rel2 + C) * rstd2), 1)}


def backward(f, d_ro, d_h, rstd, gate_form, scale_form, gate_act="none", post_norm=True):
    """Gradients of the block whose forward pass `f` holds (y, r: the values
    the backward pass reads, which may be a checkpoint's; rstd: as kept)."""
    y, r, g, w1, w2, a = (f[k] for k in ("y", "r", "g", "w1", "w2", "a"))
    T, H = y.shape
    rstd1, rstd2 = rstd[:, :1].double(), rstd[:, 1:].double()
    dh = d_h.double()
    df = torch.zeros_like(y) if d_ro is None else d_ro.double()
    u = y * rstd1
    n = u * w1
    ro = a * r + g * n
    dv = dh * w2
    q = rstd2 ** 3 * (dv * ro).mean(1, keepdim=True)
    D = df + rstd2 * dv - q * ro
    dn = g * D * w1
    d_y = rstd1 * dn
    if post_norm:
        d_y = d_y - y * rstd1 ** 3 * (dn * y).mean(1, keepdim=True)
    out = {"d_y": d_y, "d_residual": a * D, "d_w_post": (g * D * u).sum(0),
           "d_w_pre": (dh * ro * rstd2).sum(0)}
    # the same sums over magnitudes: what an error of one part in 2^24 of every
    # step would come to
    A = (a * r).abs() + (g * n).abs()
    Q = rstd2 ** 3 * (dv.abs() * A).mean(1, keepdim=True)
    B = df.abs() + rstd2 * dv.abs() + Q * A
    gw = (g * w1).abs()
    size = {"d_y": rstd1 * gw * B, "d_residual": a.abs() * B, "d_w_post": (g.abs() * B * u.abs()).sum(0),
            "d_w_pre": (dh.abs() * A * rstd2).sum(0)}
    if post_norm:
        size["d_y"] = size["d_y"] + y.abs() * rstd1 ** 3 * (gw * B * y.abs()).mean(1, keepdim=True)
    if gate_form != "none":
        s = slope(f["z"], gate_act)
        dg, Bg = n * D, n.abs() * B
        if gate_form == "channel":
            dg, Bg = dg.sum(0), Bg.sum(0)
        elif gate_form == "token":
            dg, Bg = dg.sum(1, keepdim=True), Bg.sum(1, keepdim=True)
        out["d_gate"], size["d_gate"] = s * dg, s.abs() * Bg
    if scale_form != "none":
        ds, Bs = (r * D).sum(0), (r.abs() * B).sum(0)
        if scale_form == "one":
            ds, Bs = ds.sum().reshape(1), Bs.sum().reshape(1)
        out["d_res_scale"], size["d_res_scale"] = ds, Bs
    return out, size


def backward_bounds(out, size, T, H, dtype, r_dtype, gate_form, gate_dtype):
    """Each term passes two row sums' steps; a sum over tokens adds at most T
    more, the single scale's at most T * (values per thread) + 20 more."""
    C = 2 * steps(H)
    b = {}
    for k, v in out.items():
        if k == "d_y":
            extra, t = 0, dtype
        elif k == "d_residual":
            extra, t = 0, r_dtype
        elif k == "d_gate" and gate_form == "full":
            extra, t = 0, gate_dtype
        elif k == "d_gate" and gate_form == "token":
            extra, t = 0, torch.float32
        elif k == "d_res_scale":
            extra, t = T * max(64, H / 512) + 20, torch.float32
        else:
            extra, t = T, torch.float32
        err = (C + extra) * EPS * size[k]
        b[k] = err + half_step(t) * (v.abs() + err) + tiny(t)
    return b


# ---------------------------------------------------------------- checkpoints

QMAX = {"e4m3": 448.0, "int8": 127.0}


def pack(x, fmt):
    """Codes and scale bytes, by comparing with the format's grid in 64 bits."""
    T, H = x.shape
    n = -(-H // GROUP)
    v = torch.zeros(T, n * GROUP, dtype=torch.float64, device=x.device)
    v[:, :H] = x.double()
    v = v.reshape(T, n, GROUP)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    m = v.abs().amax(2)
    k = torch.full_like(m, -126.0)
    while True:
        up = m > QMAX[fmt] * torch.exp2(k)
        if not up.any():
            break
        k = torch.where(up, k + 1, k)
    s = v / torch.exp2(k)[:, :, None]
    if fmt == "int8":
        codes = torch.round(s).to(torch.int8).view(torch.uint8)
    else:
        # every finite e4m3 magnitude, and the nearest of them, ties to the even code
        grid = torch.tensor([(i & 7) * 2.0 ** -9 if i < 8 else (1 + (i & 7) / 8) * 2.0 ** ((i >> 3) - 7)
                             for i in range(127)], dtype=torch.float64, device=x.device)
        a = s.abs()
        hi = torch.searchsorted(grid, a.contiguous()).clamp_max(126)
        lo = (hi - 1).clamp_min(0)
        dl, dh = a - grid[lo], grid[hi] - a
        code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        code = torch.where(torch.signbit(s), code + 128, code)
        codes = code.to(torch.uint8)
    codes = torch.where(bad[:, :, None], torch.zeros_like(codes), codes)
    scales = torch.where(bad, torch.full_like(k, 255.0), k + 127).to(torch.uint8)
    return codes.reshape(T, -1)[:, :H].contiguous(), scales


def unpack(codes, scales, fmt):
    """The values, in 64 bits."""
    T, H = codes.shape
    c = codes.long()
    if fmt == "int8":
        v = torch.where(c > 127, c - 256, c).double()
    else:
        m, e = (c & 7).double(), ((c >> 3) & 15).double()
        v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
        v = torch.where(c > 127, -v, v)
    unit = torch.exp2(scales.double() - 127)
    unit = torch.where(scales == 255, torch.full_like(unit, float("nan")), unit)
    return v * unit.repeat_interleave(GROUP, 1)[:, :H]
