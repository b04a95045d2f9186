"""Layer norm, the projections with their epilogue and the orthogonalised
update in 64 bits, and how far fp32 sums and a rounding at the end may be from them."""
import math

import torch

U = 2.0 ** -24                                     # half a step of fp32
ACTS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


def half_step(t, value):
    """Half a step of type t at `value` (and of its smallest values)."""
    f = torch.finfo(t)
    return value.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def act(z, name):
    """act(z), act'(z), and the size of what an fp32 evaluation of either may be off by, in units of
    2^-23: 8 roundings and approximations of 2 ulp, and 4 times the exponent's argument, whose
    rounding the exponential passes on as it is."""
    if name == "none":
        return z, torch.ones_like(z), 0 * z, 0 * z
    if name == "relu":
        return z.clamp_min(0), (z > 0).double(), 0 * z, 0 * z
    if name == "relu2":
        return z.clamp_min(0) ** 2, 2 * z.clamp_min(0), z.clamp_min(0) ** 2, 2 * z.clamp_min(0)
    if name == "gelu":
        p = torch.special.erfc(-z / math.sqrt(2)) / 2
        d = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        a = 8 + 4 * z * z
        return z * p, p + d, (z * p).abs() * a, (p + d.abs()) * a
    u = z if name == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    du = torch.ones_like(z) if name == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
    p, q = torch.sigmoid(u), torch.sigmoid(-u)
    a = 8 + 4 * u.abs()
    return z * p, p + z * p * q * du, (z * p).abs() * a, (p + (z * p * q * du).abs()) * a


def product_error(a, b, pieces=64):
    """How far the tensor cores' a b^T may be from it: an instruction adds 16 products to a sum and cuts
    what the addition shifts out, at most 2^-22 of the largest magnitudes in it; a sum takes at
    most 4 x 64 of them, the pieces are added in fp32."""
    k = a.shape[1]
    n = 4 * min(-(-k // 64), 64) + pieces
    return n * 2.0 ** -22 * (a.abs() @ b.abs().t())


def linear(x, w, bias, residual, name):
    x, w = x.double(), w.double()
    z = x @ w.t()
    ez = product_error(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * (z.abs() + bias.double().abs())
    out, slope, ea, _ = act(z, name)
    # the activations are steeper than 1.13 nowhere but relu squared, by 2 |z|
    steep = 2 * (z.abs() + ez) if name == "relu2" else 1.13
    eo = steep * ez + 2 * U * ea
    if residual is not None:
        out = out + residual.double()
        eo = eo + U * (out.abs() + eo)
    return out, z, eo, ez


def linear_dx(d, w, z, name):
    d, w = d.double(), w.double()
    p, e = d @ w, product_error(d, w.t().contiguous())
    if name == "none":
        return p, e
    _, slope, _, es = act(z.double(), name)
    return p * slope, e * (slope.abs() + 2 * U * es) + p.abs() * 2 * U * es + U * (p * slope).abs()


def layer_norm(x, w, b, eps):
    """out, stats and how far each may be: row sums are trees of at most 48 additions deep."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    D = 48 * U
    em = D * x.abs().mean(1, keepdim=True)
    ec = em + U * c.abs()
    evar = (2 * ec * c.abs() + ec * ec).mean(1, keepdim=True) + D * var
    er = rstd * (0.5 * evar / (var + eps) + 4 * U)
    h = c * rstd
    eh = ec * rstd + c.abs() * er + 2 * U * h.abs()
    w = torch.ones_like(x[0]) if w is None else w.double()
    b = torch.zeros_like(x[0]) if b is None else b.double()
    out = h * w + b
    return out, torch.cat((mean, rstd), 1), eh * w.abs() + 2 * U * (out.abs() + (h * w).abs()), torch.cat((em, er), 1)


def layer_norm_backward(d, x, stats, w, d_residual):
    d, x, stats = d.double(), x.double(), stats.double()
    T, H = x.shape
    mean, rstd = stats[:, :1], stats[:, 1:]
    h = (x - mean) * rstd
    eh = 3 * U * h.abs()                               # two roundings, of x - mean and of the product
    w = torch.ones_like(x[0]) if w is None else w.double()
    e = d * w
    m1, m2 = e.mean(1, keepdim=True), (e * h).mean(1, keepdim=True)
    D = 48 * U
    em1 = D * e.abs().mean(1, keepdim=True)
    em2 = D * (e * h).abs().mean(1, keepdim=True) + (e.abs() * eh).mean(1, keepdim=True)
    inner = e - m1 - h * m2
    dx = rstd * inner
    edx = rstd * (4 * U * (e.abs() + m1.abs() + (h * m2).abs()) + em1 + h.abs() * em2 + eh * m2.abs())
    if d_residual is not None:
        dx = dx + d_residual.double()
        edx = edx + 2 * U * dx.abs()
    # a sum over tokens has at most T additions, and 64 where its parts meet
    n = (T + 64) * U
    return {"d_x": (dx, edx), "d_w": ((d * h).sum(0), n * (d * h).abs().sum(0) + (d.abs() * eh).sum(0)),
            "d_b": (d.sum(0), n * d.abs().sum(0))}


def orthogonalize(g, steps, coeffs, eps, noise=None):
    """In 64 bits. noise(value, terms, last): what a product's result is off by, added where given; last:
    what the last step reads."""
    a, b, c = coeffs
    off = noise if noise is not None else (lambda v, terms, last: 0)
    X = g.double()
    X = X / (torch.linalg.vector_norm(X, dim=(-2, -1), keepdim=True) + eps)
    X = X + off(X, X.abs(), steps == 1)
    wide = X.shape[-2] <= X.shape[-1]
    for k in range(steps):
        last = k == steps - 1
        Y = X if wide else X.mT
        A = Y @ Y.mT
        A = A + off(A, Y.abs() @ Y.abs().mT, last)
        P = a * torch.eye(A.shape[-1], dtype=A.dtype, device=A.device) + b * A + c * (A @ A)
        P = P + off(P, P.abs() + abs(b) * A.abs() + abs(c) * (A.abs() @ A.abs()), last)
        Y = P @ Y
        if not last:
            Y = Y + off(Y, P.abs() @ (X if wide else X.mT).abs(), k == steps - 2)
        X = Y if wide else Y.mT
    return X


def orthogonalize_error(g, steps, coeffs, eps, out_type):
    """The result and how far a run on the tensor cores may be from it. Each product is off by 2^-21 of
    the sizes of its terms (two fp16 parts hold 22 bits, what is left out of the product of two
    pairs is of that size too) and by what the additions cut: each of the 12 instructions for 64 of the summed axis
    leaves out between 0 and 2^-23 of the sum, which adds up to 2^-24 of it for each, towards zero, and varies by the root of
    their number; what the last step of a bf16 result reads is rounded to
    fp16, 2^-11 of itself, which on the diagonal A has b / 2c beside it; all of random sign, carried through
    the steps in 64 bits, three times. What comes out is a sum of many independent terms: the largest of N such values lies
    near sqrt(2 ln N) root mean squares (5.5 for three million, where four were not enough), and one
    more makes it rare; or four times an element's own largest sample; and the rounding at the end."""
    want = orthogonalize(g, steps, coeffs, eps)
    k = max(g.shape[-2:])
    n = 12 * -(-k // 64)
    size, drift = 2.0 ** -21 + 2.0 ** -23 * math.sqrt(n), n * 2.0 ** -24
    shift = abs(coeffs[1] / (2 * coeffs[2])) if coeffs[2] else 0.0
    worst = torch.zeros_like(want)
    for seed in range(3):
        r = torch.Generator(device=g.device).manual_seed(seed)

        def noise(v, terms, last):
            s = torch.randint(0, 2, v.shape, generator=r, device=v.device, dtype=torch.int8).double() * 2 - 1
            tol = size * terms
            if last and out_type == torch.bfloat16:
                held = v.abs()
                if v.shape[-1] == v.shape[-2]:
                    held = held + shift * torch.eye(v.shape[-1], dtype=v.dtype, device=v.device)
                tol = tol + held * 2.0 ** -11
            return s * tol - drift * v
        worst = torch.maximum(worst, (orthogonalize(g, steps, coeffs, eps, noise) - want).abs())
    # worst is the largest of three samples: its root mean square is above one sample's
    floor = worst.square().mean((-2, -1), keepdim=True).sqrt()
    most = 1 + math.sqrt(2 * math.log(max(g.numel(), 2)))
    return want, torch.maximum(4 * worst, most * floor) + half_step(out_type, want)


def within(got, want, error, t=None):
    """Every element of got within `error` and the half step of its own type."""
    t = t or got.dtype
    off = (got.double() - want).abs()
    tol = error + half_step(t, want.abs() + error)
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), got.numel(), float((off / tol).max()), bad.nonzero()[:4].tolist())
