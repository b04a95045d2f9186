"""The training and serving operators of a gated, sandwich-normed residual
block, case by case: the block boundary and its backward pass, 8-bit
activation checkpoints, and the weight gradient read from a checkpoint.

    n = y * rstd1 * w_post                  rstd1 = 1 / sqrt(mean(y^2) + eps)
    residual_out = scale * residual + act(gate) * n
    h = residual_out * rstd2 * w_pre        rstd2 = 1 / sqrt(mean(residual_out^2) + eps)

A checkpoint holds a row in groups of 32 values: with m the largest magnitude
of the group and Q the format's largest value (448 for e4m3, 127 for int8),
k is the least integer, at least -126, with m <= Q * 2^k, and each value is
held as x * 2^-k rounded to the format (nearest, ties to even).
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 32
QMAX = {"e4m3": 448.0, "int8": 127.0}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases


def _block(name, op, T, H, type="bf16", res="bf16", gate="channel", act="none", scale="none",
           pad=0, fmt="none"):
    return {"name": name, "op": op, "T": T, "H": H, "type": type, "res": res, "gate": gate,
            "act": act, "scale": scale, "pad": pad, "fmt": fmt}


def listed():
    return [
        # one token of a decode loop: latency alone
        _block("norm_1x7168", "norm", 1, 7168, scale="channel"),
        # a ragged prompt of an odd width, read from rows that lie three values further apart
        _block("norm_1021x1999_odd", "norm", 1021, 1999, type="fp16", res="fp16", gate="token",
               act="sigmoid", scale="one", pad=3),
        # a long prompt with an output gate of its own for every value
        _block("norm_8192x7168_gated", "norm", 8192, 7168, gate="full", act="sigmoid"),
        # the backward pass of a short sequence
        _block("back_512x7168", "back", 512, 7168, scale="channel"),
        # single precision, a width that no vector load divides
        _block("back_2047x1102_fp32", "back", 2047, 1102, type="fp32", res="fp32", gate="full",
               act="tanh", scale="one"),
        # a training step's boundary, forward and backward, between them only 8-bit checkpoints;
        # the residual stream kept in single precision
        _block("step_4096x4096_e4m3", "step", 4096, 4096, res="fp32", gate="token", act="sigmoid",
               scale="one", fmt="e4m3"),
        # the same at the largest size, the stream in bf16
        _block("step_8192x7168_int8", "step", 8192, 7168, scale="channel", fmt="int8"),
        # activations of a small batch into a checkpoint and back
        {"name": "ckpt_64x2048_int8", "op": "ckpt", "T": 64, "H": 2048, "type": "fp16",
         "fmt": "int8", "pad": 0},
        # and of a large one
        {"name": "ckpt_8192x7168_e4m3", "op": "ckpt", "T": 8192, "H": 7168, "type": "bf16",
         "fmt": "e4m3", "pad": 0},
        # a small projection's weight gradient, nothing a multiple of a tile
        {"name": "dw_333x519x1096", "op": "dw", "T": 333, "N": 519, "K": 1096, "type": "bf16",
         "fmt": "int8", "out": "fp32"},
        # an ordinary one
        {"name": "dw_4096x2048x2048", "op": "dw", "T": 4096, "N": 2048, "K": 2048, "type": "fp16",
         "fmt": "e4m3", "out": "fp32"},
        # the largest: a long sequence into a wide projection
        {"name": "dw_8192x7168x4096", "op": "dw", "T": 8192, "N": 7168, "K": 4096, "type": "bf16",
         "fmt": "e4m3", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width in [lo, hi]: of whole groups, of whole vectors, or any."""
    step = rng.choice((32, 32, 8, 1))
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "back", "back", "step", "ckpt", "dw", "dw"))
    if op == "dw":
        while True:
            T, N, K = _log(rng, 1, 8192), _width(rng, 32, 7168), _width(rng, 32, 7168)
            if T * N * K <= 8192 * 7168 * 4096:
                break
        return {"op": op, "T": T, "N": N, "K": K, "type": rng.choice(("bf16", "bf16", "fp16")),
                "fmt": rng.choice(("e4m3", "int8")), "out": rng.choice(("fp32", "bf16"))}
    T, H = _log(rng, 1, 8192), _width(rng, 32, 7168)
    if op == "ckpt":
        return {"op": op, "T": T, "H": H, "type": rng.choice(("bf16", "fp16", "fp32")),
                "fmt": rng.choice(("e4m3", "int8")), "pad": rng.choice((0, 0, 3, 16))}
    type, res = rng.choice((("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                            ("fp32", "fp32")))
    gate = rng.choice(("none", "channel", "token", "full"))
    return {"op": op, "T": T, "H": H, "type": type, "res": res, "gate": gate,
            "act": "none" if gate == "none" else rng.choice(("none", "sigmoid", "tanh")),
            "scale": rng.choice(("none", "one", "channel")), "pad": rng.choice((0, 0, 3, 16)),
            "fmt": rng.choice(("e4m3", "int8")) if op == "step" else "none"}


def work(case):
    op, T = case["op"], case["T"]
    if op == "dw":
        N, K = case["N"], case["K"]
        return {"bytes": T * N * 2 + T * (K + -(-K // GROUP)) + N * K * SIZE[case["out"]],
                "flops": 2 * T * N * K}
    H = case["H"]
    n, e = T * H, SIZE[case["type"]]
    held = n + T * -(-H // GROUP)                      # codes and scales of one checkpoint
    if op == "ckpt":
        return {"bytes": 2 * (n * e + held), "flops": 4 * n}
    r = SIZE[case["res"]]
    g = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": n * e}[case["gate"]]
    a = {"none": 0, "one": 4, "channel": 4 * H}[case["scale"]]
    norm = n * (2 * e + 2 * r) + 8 * T + 8 * H + g + a
    back = n * (2 * e + 2 * r) + 8 * T + 16 * H + 2 * g + 2 * a
    if op == "norm":
        return {"bytes": norm, "flops": 10 * n}
    if op == "back":
        return {"bytes": back + n * (e + r), "flops": 25 * n}
    # the step: the checkpoints of y and residual written by the one half and read by the other
    return {"bytes": norm + back + 4 * held, "flops": 40 * n}


# ------------------------------------------------------------------ inputs


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _rows(g, T, H, dtype, pad=0, std=1.0):
    """[T, H] values, rows `pad` further apart than they are long."""
    t = torch.randn(T, H + pad, generator=g, device=g.device)
    t = t.mul_(std).to(dtype)
    return t[:, :H] if pad else t


def _activations(g, T, H, dtype, pad=0):
    """A stream as networks have it: rows of different size and a few channels far above the rest."""
    t = torch.randn(T, H + pad, generator=g, device=g.device)
    t *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=g.device))
    loud = torch.rand(H + pad, generator=g, device=g.device) < 0.01
    t *= torch.where(loud, 20.0, 1.0)
    t = t.to(dtype)
    return t[:, :H] if pad else t


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    T, op = case["T"], case["op"]
    s = {"case": case}
    if op == "dw":
        s["d_out"] = _rows(g, T, case["N"], TYPES[case["type"]], std=0.05)
        x = _activations(g, T, case["K"], torch.bfloat16)
        s["codes"], s["scales"] = _pack(x, case["fmt"])   # as the forward pass left them
        if own:
            from manifold_constrained_hyper_gb300 import ops
            s["ckpt"] = ops.Checkpoint(s["codes"], s["scales"], case["fmt"])
        return s
    H, dt, pad = case["H"], TYPES[case["type"]], case["pad"]
    if op == "ckpt":
        s["x"] = _activations(g, T, H, dt, pad)
        return s
    rt = TYPES[case["res"]]
    rand = lambda *shape: torch.randn(*shape, generator=g, device=g.device)  # noqa: E731
    s["y"] = _rows(g, T, H, dt, pad, std=1.5)
    s["residual"] = _activations(g, T, H, rt, pad)
    s["w_post"] = 1 + 0.1 * rand(H)
    s["w_pre"] = 1 + 0.1 * rand(H)
    s["gate"] = {"none": lambda: None, "channel": lambda: 0.5 + 0.2 * rand(H),
                 "token": lambda: rand(T, 1), "full": lambda: _rows(g, T, H, dt)}[case["gate"]]()
    s["scale"] = {"none": lambda: None, "one": lambda: 0.9 + 0.05 * rand(1),
                  "channel": lambda: 0.9 + 0.05 * rand(H)}[case["scale"]]()
    if op != "norm":
        s["d_residual_out"] = _rows(g, T, H, rt, pad, std=0.02)
        s["d_h"] = _rows(g, T, H, dt, pad, std=0.05)
    if op == "back":
        # what the forward pass kept beside its inputs
        s["rstd"] = _norm(s["y"], s["residual"], s["w_post"], s["w_pre"], s["gate"], s["scale"],
                          case["act"])[2]
    if own:
        from manifold_constrained_hyper_gb300 import ops
        s["params"] = ops.BlockParams(eps_post=EPS, eps_pre=EPS, gate_act=case["act"])
    return s


# ------------------------------------------------------------------ plain forms


def _act(z, act):
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "tanh":
        return torch.tanh(z)
    return z


def _d_act(z, act):
    g = _act(z, act)
    if act == "sigmoid":
        return g * (1 - g)
    if act == "tanh":
        return 1 - g * g
    return torch.ones_like(z)


def _norm(y, residual, w_post, w_pre, gate, scale, act):
    yf, rf = y.float(), residual.float()
    rstd1 = 1 / torch.sqrt(yf.square().mean(1, keepdim=True) + EPS)
    n = yf * rstd1 * w_post
    if gate is not None:
        n = n * _act(gate.float(), act)
    ro = n + (rf if scale is None else rf * scale)
    rstd2 = 1 / torch.sqrt(ro.square().mean(1, keepdim=True) + EPS)
    h = ro * rstd2 * w_pre
    return ro.to(residual.dtype), h.to(y.dtype), torch.cat((rstd1, rstd2), 1)


def _back(d_ro, d_h, y, residual, rstd, w_post, w_pre, gate, scale, act):
    yf, rf, df, dh = y.float(), residual.float(), d_ro.float(), d_h.float()
    H = yf.shape[1]
    rstd1, rstd2 = rstd[:, :1], rstd[:, 1:]
    g = None if gate is None else _act(gate.float(), act)
    yn = yf * rstd1
    n = yn * w_post
    ro = (n if g is None else n * g) + (rf if scale is None else rf * scale)
    dn2 = dh * w_pre
    c2 = (dn2 * ro).sum(1, keepdim=True)
    D = df + rstd2 * dn2 - ro * (rstd2 ** 3 * c2 / H)
    out = {"d_residual": (D if scale is None else D * scale).to(d_ro.dtype)}
    gD = D if g is None else D * g
    dn1 = gD * w_post
    c1 = (dn1 * yf).sum(1, keepdim=True)
    out["d_y"] = (rstd1 * dn1 - yf * (rstd1 ** 3 * c1 / H)).to(d_h.dtype)
    out["d_w_post"] = (gD * yn).sum(0)
    out["d_w_pre"] = (dh * ro * rstd2).sum(0)
    if gate is not None:
        dg = n * D
        if gate.dim() == 1:
            out["d_gate"] = dg.sum(0) * _d_act(gate.float(), act)
        elif gate.shape[1] == 1 and H > 1:
            out["d_gate"] = dg.sum(1, keepdim=True) * _d_act(gate.float(), act)
        else:
            out["d_gate"] = (dg * _d_act(gate.float(), act)).to(gate.dtype)
    if scale is not None:
        ds = rf * D
        out["d_scale"] = ds.sum(0) if scale.numel() == H and H > 1 else ds.sum().reshape(1)
    return out


def _groups(x):
    T, H = x.shape
    n = -(-H // GROUP)
    f = x.float()
    if n * GROUP != H:
        f = torch.cat((f, f.new_zeros(T, n * GROUP - H)), 1)
    return f.reshape(T, n, GROUP)


def _pack(x, fmt):
    """Codes [T, H] and scales [T, groups], both as bytes."""
    f = _groups(x)
    m, ex = torch.frexp(f.abs().amax(2))
    # Q = top * 2^e with top in [0.5, 1): m * 2^ex <= Q * 2^k
    top, e = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)
    k = (ex - e + (m > top)).clamp_min(-126)
    v = torch.ldexp(f, -k[:, :, None]).reshape(x.shape[0], -1)[:, :x.shape[1]]
    codes = v.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(v).to(torch.int8)
    return codes.contiguous().view(torch.uint8), (k + 127).to(torch.uint8)


def _unpack(codes, scales, fmt):
    v = _groups(codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8))
    v = torch.ldexp(v, scales[:, :, None].int() - 127)
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


# ------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "ckpt":
        codes, scales = _pack(s["x"], c["fmt"])
        return _unpack(codes, scales, c["fmt"]).to(s["x"].dtype)
    if c["op"] == "dw":
        x = _unpack(s["codes"], s["scales"], c["fmt"])
        return (s["d_out"].float().t() @ x).to(TYPES[c["out"]])
    block = (s["w_post"], s["w_pre"], s["gate"], s["scale"], c["act"])
    if c["op"] == "back":
        return _back(s["d_residual_out"], s["d_h"], s["y"], s["residual"], s["rstd"], *block)
    ro, h, rstd = _norm(s["y"], s["residual"], *block)
    if c["op"] == "norm":
        return {"residual_out": ro, "h": h, "rstd": rstd}
    y = _unpack(*_pack(s["y"], c["fmt"]), c["fmt"])
    residual = _unpack(*_pack(s["residual"], c["fmt"]), c["fmt"])
    out = _back(s["d_residual_out"], s["d_h"], y, residual, rstd, *block)
    return {"residual_out": ro, "h": h, **out}


def _run_own(s):
    from manifold_constrained_hyper_gb300 import ops
    c = s["case"]
    if c["op"] == "ckpt":
        return ops.mhc_ckpt_unpack(ops.mhc_ckpt_pack(s["x"], c["fmt"]), s["x"].dtype)
    if c["op"] == "dw":
        return ops.mhc_ckpt_linear_dw(s["d_out"], s["ckpt"], dtype=TYPES[c["out"]])
    block = (s["w_post"], s["w_pre"], s["gate"], s["scale"], s["params"])
    if c["op"] == "norm":
        ro, h, rstd = ops.mhc_block_norm(s["y"], s["residual"], *block)
        return {"residual_out": ro, "h": h, "rstd": rstd}
    if c["op"] == "back":
        d = ops.mhc_block_norm_backward(s["d_residual_out"], s["d_h"], s["y"], s["residual"],
                                        s["rstd"], *block)
        return _named(d)
    T, H = s["y"].shape
    y8, r8 = (ops.ckpt_empty(T, H, c["fmt"], s["y"].device) for _ in range(2))
    ro, h, rstd = ops.mhc_block_norm(s["y"], s["residual"], *block, ckpt_y=y8, ckpt_residual=r8)
    d = ops.mhc_block_norm_backward(s["d_residual_out"], s["d_h"], y8, r8, rstd, *block)
    return {"residual_out": ro, "h": h, **_named(d)}


def _named(d):
    out = {"d_residual": d.d_residual, "d_y": d.d_y, "d_w_post": d.d_w_post, "d_w_pre": d.d_w_pre}
    if d.d_gate is not None:
        out["d_gate"] = d.d_gate
    if d.d_res_scale is not None:
        out["d_scale"] = d.d_res_scale
    return out


# ------------------------------------------------------------------ in 64 bits


def _held64(x, fmt):
    """What a checkpoint of `x` stands for, found by comparing with the formats' grids."""
    T, H = x.shape
    out = torch.empty(T, H, dtype=torch.float64, device=x.device)
    for a in range(0, H, GROUP):
        v = x[:, a:a + GROUP].double()
        m = v.abs().max(1, keepdim=True).values
        k = torch.floor(torch.log2(torch.clamp(m, min=2.0 ** -200) / QMAX[fmt])) - 1
        for _ in range(3):
            k = torch.where(m > QMAX[fmt] * torch.exp2(k), k + 1, k)
        unit = torch.exp2(torch.clamp(k, min=-126.0))
        v = v / unit
        if fmt == "e4m3":
            # three bits below the leading one, or below that of 2^-6
            low = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -6)))
            step = torch.exp2(low - 3)
        else:
            step = torch.ones_like(v)
        out[:, a:a + GROUP] = torch.round(v / step) * step * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ckpt":
        return _held64(s["x"], case["fmt"])
    if op == "dw":
        T, K = s["codes"].shape
        x = (s["codes"].view(torch.float8_e4m3fn).float().double() if case["fmt"] == "e4m3"
             else s["codes"].view(torch.int8).double())
        unit = torch.exp2(s["scales"].double() - 127)
        x = x * unit.repeat_interleave(GROUP, 1)[:, :K]
        out = torch.empty(case["N"], K, dtype=torch.float64, device=x.device)
        for a in range(0, case["N"], 1024):
            out[a:a + 1024] = s["d_out"][:, a:a + 1024].double().t() @ x
        return out
    y, r = s["y"].double(), s["residual"].double()
    T, H = y.shape
    w1, w2 = s["w_post"].double(), s["w_pre"].double()
    a = torch.ones(1, dtype=torch.float64, device=y.device) if s["scale"] is None else s["scale"].double()
    z = None if s["gate"] is None else s["gate"].double()
    if z is None:
        g, slope = torch.ones(1, 1, dtype=torch.float64, device=y.device), None
    elif case["act"] == "sigmoid":
        g = torch.sigmoid(z)
        slope = torch.sigmoid(z) * torch.sigmoid(-z)
    elif case["act"] == "tanh":
        g = torch.tanh(z)
        slope = 1 / torch.cosh(z) ** 2
    else:
        g, slope = z, torch.ones_like(z)
    e1 = (y.pow(2).sum(1, keepdim=True) / H + EPS).rsqrt()
    ro = a * r + g * (y * e1 * w1)
    e2 = (ro.pow(2).sum(1, keepdim=True) / H + EPS).rsqrt()
    first = {"residual_out": ro, "h": ro * e2 * w2}
    if op == "norm":
        return {**first, "rstd": torch.cat((e1, e2), 1)}
    if op == "back":
        first = {}
    else:
        y, r = _held64(s["y"], case["fmt"]), _held64(s["residual"], case["fmt"])
        ro = a * r + g * (y * e1 * w1)
    u = y * e1                                  # normed rows, as kept
    v = ro * e2
    dh = s["d_h"].double()
    dv = dh * w2
    D = s["d_residual_out"].double() + e2 * (dv - v * (dv * v).sum(1, keepdim=True) / H)
    du = g * D * w1
    out = {"d_residual": a * D, "d_y": e1 * (du - u * (du * u).sum(1, keepdim=True) / H),
           "d_w_post": (g * D * u).sum(0), "d_w_pre": (dh * v).sum(0)}
    if z is not None:
        dg = D * u * w1
        if case["gate"] == "channel":
            out["d_gate"] = slope * dg.sum(0)
        elif case["gate"] == "token":
            out["d_gate"] = slope * dg.sum(1, keepdim=True)
        else:
            out["d_gate"] = slope * dg
    if case["scale"] != "none":
        out["d_scale"] = (r * D).sum(0) if case["scale"] == "channel" else (r * D).sum().reshape(1)
    return {**first, **out}
