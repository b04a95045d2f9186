"""The operators around a layer's weights, case by case: layer norm and its
backward pass, the product with bias, activation and residual in its epilogue,
its two gradients, and the orthogonalised update of a weight.

    layer norm:  out = (x - mean) * rstd * w + b     rstd = 1 / sqrt(mean((x - mean)^2) + eps)
    linear:      z = x w^T + bias,  out = act(z) + residual
    backward:    d_x = (d_out w) * act'(z of the layer below)
                 d_w = d_out^T x,  d_bias = sum over tokens of d_out
    orthogonalised update: X = G / (|G| + eps) (the Frobenius norm), then a number of times
                 A = X X^T,  X <- (a I + b A + c A A) X
"""
import math

import torch

own = False

LN_EPS = 1e-5
NS_EPS = 1e-7
NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")
MOST_PRODUCTS = 8192 * 4096 * 7168
MOST_NS = 5 * (3 * 4096 * 4096 * 7168 + 4096 ** 3)


# ------------------------------------------------------------------ cases


def _ln(name, op, T, H, type="bf16", out="same", affine=True, res=False, pad=0):
    return {"name": name, "op": op, "T": T, "H": H, "type": type, "out": out, "affine": affine,
            "res": res, "pad": pad}


def _lin(name, T, K, N, type="bf16", bias="none", act="none", res="none", z=False, pad=0):
    return {"name": name, "op": "lin", "T": T, "K": K, "N": N, "type": type, "bias": bias,
            "act": act, "res": res, "z": z, "pad": pad}


def _back(name, T, N, K, type="bf16", act="none", bias=False, out="fp32", pad=0):
    return {"name": name, "op": "back", "T": T, "N": N, "K": K, "type": type, "act": act,
            "bias": bias, "out": out, "pad": pad}


def _ns(name, B, M, N, type="fp32", out="bf16"):
    return {"name": name, "op": "ns", "B": B, "M": M, "N": N, "type": type, "out": out}


def listed():
    return [
        # one token of a decode loop: latency alone
        _ln("norm_1x7168", "norm", 1, 7168),
        # a long prompt; the residual stream kept in single precision, what is read from it in bf16
        _ln("norm_8192x7168_fp32", "norm", 8192, 7168, type="fp32", out="bf16"),
        # single precision, a width that no vector load divides
        _ln("norm_back_2047x1102_fp32", "norm_back", 2047, 1102, type="fp32"),
        # a training step, the gradient that goes around the norm added in
        _ln("norm_back_4096x4096", "norm_back", 4096, 4096, res=True),
        # the projection back to the residual stream, one token of a decode loop
        _lin("linear_1x7168x4096", 1, 7168, 4096, bias="same", res="same"),
        # a ragged prompt between odd widths, rows that lie apart
        _lin("linear_333x519x1096", 333, 519, 1096, type="fp16", bias="fp32", act="gelu", z=True,
             pad=3),
        # the largest: a long sequence into a wide hidden layer, what backward needs kept
        _lin("linear_8192x4096x7168", 8192, 4096, 7168, bias="fp32", act="gelu_tanh", z=True),
        # both gradients of a short sequence between odd widths
        _back("linear_back_777x1000x2046", 777, 1000, 2046, type="fp16", act="silu", bias=True),
        # and of a long one
        _back("linear_back_8192x4096x4096", 8192, 4096, 4096, act="relu2", bias=True, out="bf16"),
        # the heads of a small model, all at once
        _ns("update_6x128x500", 6, 128, 500),
        # an ordinary weight, more rows than columns
        _ns("update_2048x1024", 1, 2048, 1024),
        # the largest weight
        _ns("update_4096x7168", 1, 4096, 7168, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width in [lo, hi]: of whole vectors, of whole tiles, or any."""
    step = rng.choice((64, 32, 8, 1))
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm_back", "lin", "lin", "lin", "back", "back", "ns", "ns"))
    if op in ("norm", "norm_back"):
        type, out = rng.choice((("bf16", "same"), ("fp16", "same"), ("fp32", "same"), ("fp32", "bf16"),
                                ("fp32", "fp16")))
        return {"op": op, "T": _log(rng, 1, 8192), "H": _width(rng, 32, 7168), "type": type, "out": out,
                "affine": rng.random() < 0.8, "res": op == "norm_back" and rng.random() < 0.5,
                "pad": rng.choice((0, 0, 3, 16))}
    if op == "ns":
        while True:
            B, M, N = rng.choice((1, 1, 1, _log(rng, 2, 64))), _width(rng, 32, 7168), _width(rng, 32, 7168)
            p, q = min(M, N), max(M, N)
            if B * NS_STEPS * (3 * p * p * q + p ** 3) <= MOST_NS:
                break
        return {"op": op, "B": B, "M": M, "N": N, "type": rng.choice(("fp32", "bf16", "fp16")),
                "out": rng.choice(("bf16", "bf16", "fp16"))}
    while True:
        T, K, N = _log(rng, 1, 8192), _width(rng, 32, 7168), _width(rng, 32, 7168)
        if T * K * N * (2 if op == "back" else 1) <= MOST_PRODUCTS:
            break
    c = {"op": op, "T": T, "K": K, "N": N, "type": rng.choice(("bf16", "bf16", "fp16")),
         "act": rng.choice(ACTS), "pad": rng.choice((0, 0, 3, 16))}
    if op == "back":
        return {**c, "bias": rng.random() < 0.5, "out": rng.choice(("fp32", "bf16"))}
    return {**c, "bias": rng.choice(("none", "fp32", "same")), "res": rng.choice(("none", "same", "fp32")),
            "z": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        n, e = case["T"] * case["H"], SIZE[case["type"]]
        o = e if case["out"] == "same" else SIZE[case["out"]]
        par = 8 * case["H"] if case["affine"] else 0
        if op == "norm":
            return {"bytes": n * (e + o) + 8 * case["T"] + par, "flops": 8 * n}
        # d_out and x, the gradient around the norm, the weight and its gradients
        return {"bytes": n * (o + 2 * e + (e if case["res"] else 0)) + 8 * case["T"] + par // 2 * 3,
                "flops": 14 * n}
    if op == "ns":
        p, q = min(case["M"], case["N"]), max(case["M"], case["N"])
        # the first two products of a step are symmetric: half of each is enough
        return {"bytes": case["B"] * p * q * (SIZE[case["type"]] + SIZE[case["out"]]),
                "flops": case["B"] * NS_STEPS * (3 * p * p * q + p ** 3)}
    T, K, N, e = case["T"], case["K"], case["N"], SIZE[case["type"]]
    if op == "lin":
        r = {"none": 0, "same": e, "fp32": 4}[case["res"]]
        b = {"none": 0, "same": e, "fp32": 4}[case["bias"]]
        return {"bytes": (T * K + N * K) * e + T * N * (r + (r or e) + (e if case["z"] else 0)) + b * N,
                "flops": 2 * T * N * K}
    z = e if case["act"] != "none" else 0
    return {"bytes": (T * N + N * K + 2 * T * K) * e + T * K * z + N * K * SIZE[case["out"]]
            + (4 * N if case["bias"] else 0), "flops": 4 * T * N * K}


# ------------------------------------------------------------------ inputs


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _rows(g, T, H, dtype, pad=0, std=1.0):
    """[T, H] values, rows `pad` further apart than they are long."""
    t = torch.randn(T, H + pad, generator=g, device=g.device)
    t = t.mul_(std).to(dtype)
    return t[:, :H] if pad else t


def _activations(g, T, H, dtype, pad=0):
    """A stream as networks have it: rows of different size and off zero, a few channels far above the rest."""
    t = torch.randn(T, H + pad, generator=g, device=g.device)
    t += 0.5 * torch.randn(T, 1, generator=g, device=g.device)
    t *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=g.device))
    loud = torch.rand(H + pad, generator=g, device=g.device) < 0.01
    t *= torch.where(loud, 20.0, 1.0)
    t = t.to(dtype)
    return t[:, :H] if pad else t


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    rand = lambda *shape: torch.randn(*shape, generator=g, device=g.device)  # noqa: E731
    if op == "ns":
        # momentum as training leaves it: a few strong directions over a floor
        B, M, N = case["B"], case["M"], case["N"]
        r = min(M, N, 32)
        u = rand(B, M, r) * torch.exp2(-0.25 * torch.arange(r, device=g.device))
        s["g"] = (1e-3 * (u @ rand(B, r, N) + 0.5 * rand(B, M, N))).to(TYPES[case["type"]])
        if B == 1:
            s["g"] = s["g"][0]
        return s
    T, pad = case["T"], case["pad"]
    dt = TYPES[case["type"]]
    if op in ("norm", "norm_back"):
        H = case["H"]
        ot = dt if case["out"] == "same" else TYPES[case["out"]]
        s["x"] = _activations(g, T, H, dt, pad)
        s["w"] = 1 + 0.1 * rand(H) if case["affine"] else None
        s["b"] = 0.1 * rand(H) if case["affine"] else None
        s["out_type"] = ot
        if op == "norm_back":
            s["d_out"] = _rows(g, T, H, ot, pad, std=0.05)
            s["d_residual"] = _rows(g, T, H, dt, pad, std=0.05) if case["res"] else None
            s["stats"] = _norm(s["x"], None, None, ot)[1]     # what the forward pass kept
        return s
    K, N = case["K"], case["N"]
    s["w"] = _rows(g, N, K, dt, std=K ** -0.5)
    if op == "lin":
        s["x"] = _rows(g, T, K, dt, pad)
        s["bias"] = {"none": lambda: None, "fp32": lambda: 0.2 * rand(N),
                     "same": lambda: (0.2 * rand(N)).to(dt)}[case["bias"]]()
        s["residual"] = {"none": lambda: None, "fp32": lambda: _activations(g, T, N, torch.float32, pad),
                         "same": lambda: _activations(g, T, N, dt, pad)}[case["res"]]()
        return s
    s["d_out"] = _rows(g, T, N, dt, pad, std=0.05)
    s["x"] = _rows(g, T, K, dt, pad)
    s["z"] = _rows(g, T, K, dt, pad) if case["act"] != "none" else None
    return s


# ------------------------------------------------------------------ plain forms


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "relu2":
        return torch.where(z > 0, z * z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _d_act(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return torch.where(z > 0, 2 * z, torch.zeros_like(z))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _norm(x, w, b, out_type):
    f = x.float()
    mean = f.mean(1, keepdim=True)
    c = f - mean
    rstd = 1 / torch.sqrt(c.square().mean(1, keepdim=True) + LN_EPS)
    h = c * rstd
    if w is not None:
        h = h * w
    if b is not None:
        h = h + b
    return h.to(out_type), torch.cat((mean, rstd), 1)


def _norm_back(d_out, x, stats, w, d_residual):
    f, d = x.float(), d_out.float()
    mean, rstd = stats[:, :1], stats[:, 1:]
    h = (f - mean) * rstd
    dh = d if w is None else d * w
    dx = rstd * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
    if d_residual is not None:
        dx = dx + d_residual.float()
    out = {"d_x": dx.to(x.dtype)}
    if w is not None:
        out["d_w"], out["d_b"] = (d * h).sum(0), d.sum(0)
    return out


def _orthogonal(g, out_type):
    a, b, c = NS_COEFFS
    X = g.float()
    X = X / (torch.sqrt(X.square().sum((-2, -1), keepdim=True)) + NS_EPS)
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.transpose(-2, -1)
    for _ in range(NS_STEPS):
        A = X @ X.transpose(-2, -1)
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.transpose(-2, -1) if tall else X).to(out_type).contiguous()


# ------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        out, stats = _norm(s["x"], s["w"], s["b"], s["out_type"])
        return {"out": out, "stats": stats}
    if c["op"] == "norm_back":
        return _norm_back(s["d_out"], s["x"], s["stats"], s["w"], s["d_residual"])
    if c["op"] == "ns":
        return _orthogonal(s["g"], TYPES[c["out"]])
    if c["op"] == "lin":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _act(z, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        out = out.to(s["x"].dtype if s["residual"] is None else s["residual"].dtype)
        return {"out": out, "z": z.to(s["x"].dtype)} if c["z"] else {"out": out}
    d = s["d_out"].float()
    dx = d @ s["w"].float()
    if s["z"] is not None:
        dx = dx * _d_act(s["z"].float(), c["act"])
    out = {"d_x": dx.to(s["x"].dtype), "d_w": (d.t() @ s["x"].float()).to(TYPES[c["out"]])}
    if c["bias"]:
        out["d_bias"] = d.sum(0)
    return out


def _run_own(s):
    from manifold_constrained_hyper_gb300 import ops
    c = s["case"]
    if c["op"] == "norm":
        out, stats = ops.mhc_layer_norm(s["x"], s["w"], s["b"], LN_EPS, dtype=s["out_type"])
        return {"out": out, "stats": stats}
    if c["op"] == "norm_back":
        d = ops.mhc_layer_norm_backward(s["d_out"], s["x"], s["stats"], s["w"], bias=c["affine"],
                                        d_residual=s["d_residual"])
        out = {"d_x": d.d_x}
        if c["affine"]:
            out["d_w"], out["d_b"] = d.d_w, d.d_b
        return out
    if c["op"] == "ns":
        return ops.mhc_orthogonalize(s["g"], NS_STEPS, NS_COEFFS, NS_EPS, dtype=TYPES[c["out"]])
    if c["op"] == "lin":
        if c["z"]:
            out, z = ops.mhc_linear(s["x"], s["w"], s["bias"], s["residual"], c["act"], keep_z=True)
            return {"out": out, "z": z}
        return {"out": ops.mhc_linear(s["x"], s["w"], s["bias"], s["residual"], c["act"])}
    out = {"d_x": ops.mhc_linear_dx(s["d_out"], s["w"], s["z"], c["act"])}
    if c["bias"]:
        out["d_w"], out["d_bias"] = ops.mhc_linear_dw(s["d_out"], s["x"], dtype=TYPES[c["out"]], bias=True)
    else:
        out["d_w"] = ops.mhc_linear_dw(s["d_out"], s["x"], dtype=TYPES[c["out"]])
    return out


# ------------------------------------------------------------------ in 64 bits


def _act64(z, act):
    """act(z) and its slope."""
    zero, one = torch.zeros_like(z), torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, zero)
    if act == "relu2":
        return z.clamp_min(0) ** 2, 2 * z.clamp_min(0)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        phi = torch.special.erfc(z * -(0.5 ** 0.5)) / 2
        return z * phi, phi + z * torch.exp(z * z * -0.5) * (2 * math.pi) ** -0.5
    # 0.5 (1 + tanh u) is the sigmoid of 2u
    u = (8 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(u)
    return z * p, p + z * p * torch.sigmoid(-u) * (8 / math.pi) ** 0.5 * (1 + 0.134145 * z * z)


def _product64(a, b):
    """a b for two matrices of few bits, in bands."""
    out = torch.empty(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
    b = b.double()
    for i in range(0, a.shape[0], 1024):
        out[i:i + 1024] = a[i:i + 1024].double() @ b
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + LN_EPS).rsqrt()
        out = (x - mean) * rstd
        if case["affine"]:
            out = torch.addcmul(s["b"].double(), out, s["w"].double())
        return {"out": out, "stats": torch.cat((mean, rstd), 1)}
    if op == "norm_back":
        x, d = s["x"].double(), s["d_out"].double()
        T, H = x.shape
        mean, rstd = s["stats"].double().unbind(1)
        n = (x - mean[:, None]) * rstd[:, None]
        e = d * s["w"].double() if case["affine"] else d
        # the projection away from the row of ones and the normed row
        s1, s2 = e.sum(1), torch.einsum("th,th->t", e, n)
        dx = (e - (s1[:, None] + n * s2[:, None]) / H) * rstd[:, None]
        if s["d_residual"] is not None:
            dx += s["d_residual"].double()
        out = {"d_x": dx}
        if case["affine"]:
            out["d_w"], out["d_b"] = torch.einsum("th,th->h", d, n), d.sum(0)
        return out
    if op == "ns":
        G = s["g"].double()
        p, q = sorted(G.shape[-2:])
        wide = G.shape[-2] == p
        G = G / (torch.linalg.vector_norm(G, dim=(-2, -1), keepdim=True) + NS_EPS)
        # every X is P times the first one, P a polynomial in its Gram matrix
        S = G @ G.mT if wide else G.mT @ G
        unit = torch.eye(p, dtype=G.dtype, device=G.device)
        P = unit.expand_as(S)
        for _ in range(NS_STEPS):
            A = S @ (P @ P)
            P = (NS_COEFFS[0] * unit + A @ (NS_COEFFS[1] * unit + NS_COEFFS[2] * A)) @ P
        return P @ G if wide else G @ P
    if op == "lin":
        z = _product64(s["x"], s["w"].t())
        if s["bias"] is not None:
            z += s["bias"].double()
        out = _act64(z, case["act"])[0]
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return {"out": out, "z": z} if case["z"] else {"out": out}
    dx = _product64(s["d_out"], s["w"])
    if s["z"] is not None:
        dx *= _act64(s["z"].double(), case["act"])[1]
    out = {"d_x": dx, "d_w": _product64(s["d_out"].t(), s["x"])}
    if case["bias"]:
        out["d_bias"] = s["d_out"].double().sum(0)
    return out
