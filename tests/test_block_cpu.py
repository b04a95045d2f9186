"""What of the gated residual block and the 8-bit checkpoints needs no GPU:
the 64-bit forms' gradients against differences, the entry points' refusals
(before any device work), and the workspace sizes."""
import ctypes
import os
import struct
import subprocess

import pytest
import torch

from manifold_constrained_hyper_gb300 import build as mbuild
from manifold_constrained_hyper_gb300 import ops
from tests import block_ref as ref


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return ops.load()


GATES = {"none": None, "channel": (5,), "token": (3, 1), "full": (3, 5)}


@pytest.mark.parametrize("gate_form,act", [("none", "none"), ("channel", "tanh"), ("token", "sigmoid"),
                                           ("full", "none"), ("full", "sigmoid")])
@pytest.mark.parametrize("scale_form", ["none", "one", "channel"])
@pytest.mark.parametrize("post_norm", [True, False])
def test_the_plain_gradients_against_differences(gate_form, act, scale_form, post_norm):
    g = torch.Generator().manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    y, r = rand(3, 5), rand(3, 5)
    w1, w2 = (1 + 0.1 * rand(5) if post_norm else None), 1 + 0.1 * rand(5)
    gate = None if gate_form == "none" else rand(*GATES[gate_form])
    scale = {"none": None, "one": rand(1), "channel": rand(5)}[scale_form]
    A, B = rand(3, 5), rand(3, 5)
    kw = {"gate_act": act, "post_norm": post_norm, "weight_offset": 0.25}

    def loss(**over):
        t = {"y": y, "residual": r, "w_post": w1, "w_pre": w2, "gate": gate, "res_scale": scale, **over}
        f = ref.block(**t, **kw)
        return (A * f["ro"] + B * f["h"]).sum()

    f = ref.block(y, r, w1, w2, gate, scale, **kw)
    out, _ = ref.backward(f, A, B, f["rstd"], gate_form, scale_form, act, post_norm)
    names = {"d_y": ("y", y), "d_residual": ("residual", r), "d_w_post": ("w_post", w1),
             "d_w_pre": ("w_pre", w2), "d_gate": ("gate", gate), "d_res_scale": ("res_scale", scale)}
    for k, d in out.items():
        name, x = names[k]
        if x is None:
            continue
        for at in range(x.numel()):
            e = torch.zeros(x.numel(), dtype=torch.float64)
            e[at] = 1e-5
            e = e.reshape(x.shape)
            diff = (loss(**{name: x + e}) - loss(**{name: x - e})) / 2e-5
            # the differences' own error: (1e-5)^2 of the third derivative, 1e-16 / 1e-5 of the loss
            assert abs(float(diff) - float(d.reshape(-1)[at])) < 1e-7 * (1 + abs(float(diff))), (k, at)


def test_the_plain_checkpoint_round_trip():
    x = torch.randn(7, 77, dtype=torch.float64) * 3
    for fmt, rel, absolute in (("e4m3", 2.0 ** -4, 2.0 ** -10), ("int8", 0.0, 0.5)):
        codes, scales = ref.pack(x, fmt)
        unit = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :77]
        assert ((ref.unpack(codes, scales, fmt) - x).abs() <= rel * x.abs() + absolute * unit).all()
    # Q 2^k itself keeps k, the next value above takes k + 1
    top = torch.tensor([[448.0] + [0.0] * 31, [448.0000001] + [0.0] * 31], dtype=torch.float64)
    assert ref.pack(top, "e4m3")[1].flatten().tolist() == [127, 128]


# mhc_block and mhc_ckpt of include/mhc.h
_BLOCK = struct.Struct("@qiiiPPiiPiiiqPifffi4x")
_CKPT = struct.Struct("@PP")
A = 0x100000           # an aligned address that is never read


def _P(v):
    return ctypes.c_void_p(v)


def _ckpt(codes, scales):
    return _CKPT.pack(codes or 0, scales or 0)


def _block(**over):
    v = dict(tokens=4, hidden=64, dtype=1, residual_dtype=1, w_post=A * 1, w_pre=A * 2, w_post_dtype=0,
             w_pre_dtype=0, gate=A * 3, gate_dtype=0, gate_form=1, gate_act=0, gate_stride=64,
             res_scale=A * 4, scale_form=2, eps_post=1e-6, eps_pre=1e-6, weight_offset=0.0, post_norm=1)
    v.update(over)
    return _BLOCK.pack(*(0 if x is None else x for x in v.values()))


def _norm(lib, b, y=A * 5, ys=64, r=A * 6, rs=64, ro=A * 7, h=A * 8, rstd=A * 9, fmt=0, cy=None, cr=None, ch=None):
    return lib.mhc_block_norm(b, _P(y), ys, _P(r), rs, _P(ro), _P(h), _P(rstd), fmt, cy, cr, ch, None)


def test_the_packed_structures_are_the_compiler_s(tmp_path):
    fields = ("tokens hidden dtype residual_dtype w_post w_pre w_post_dtype w_pre_dtype gate gate_dtype gate_form "
              "gate_act gate_stride res_scale scale_form eps_post eps_pre weight_offset post_norm").split()
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "layout.c"
    src.write_text('#include "mhc.h"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(mhc_block, {f}));' for f in fields)
                   + 'printf("%zu %zu", sizeof(mhc_block), sizeof(mhc_ckpt)); return 0; }')
    subprocess.run(["gcc", "-I", include, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "layout")]).split()]
    codes = "qiiiPPiiPiiiqPifffi"
    want = [struct.calcsize("@" + codes[:i] + "0" + codes[i]) for i in range(len(codes))]
    assert got == want + [_BLOCK.size, _CKPT.size]


def test_refusals_of_the_block(lib):
    assert _norm(lib, None) == 1
    assert _norm(lib, _block(tokens=-1)) == 3
    for H in (0, -5, 65537):
        assert _norm(lib, _block(hidden=H)) == 4
    for bad in (dict(dtype=3), dict(dtype=1, residual_dtype=2), dict(dtype=0, residual_dtype=1),
                dict(w_post_dtype=7), dict(w_pre_dtype=-1), dict(gate_form=4), dict(gate_form=-1),
                dict(gate_act=3), dict(scale_form=3), dict(eps_post=-1.0), dict(eps_pre=float("nan")),
                dict(weight_offset=float("inf")), dict(post_norm=0), dict(gate_dtype=2),
                dict(gate_form=3, gate_stride=-64), dict(gate_form=0), dict(gate_form=0, gate=None, gate_act=1),
                dict(scale_form=0), dict(tokens=1 << 60)):
        assert _norm(lib, _block(**bad)) == 3, bad
    assert _norm(lib, _block(gate=None)) == 1
    assert _norm(lib, _block(res_scale=None)) == 1
    for k in ("y", "r", "ro", "h"):
        assert _norm(lib, _block(), **{k: None}) == 1, k
    assert _norm(lib, _block(), ys=-64) == 3
    assert _norm(lib, _block(), rs=-1) == 3
    assert _norm(lib, _block(), ys=1 << 62) == 3
    # an element type's own alignment, no more
    for k, odd in (("y", A * 5 + 1), ("h", A * 8 + 1), ("rstd", A * 9 + 2), ("r", A * 6 + 1)):
        assert _norm(lib, _block(), **{k: odd}) == 2, k
    assert _norm(lib, _block(w_post=A + 2)) == 2
    assert _norm(lib, _block(res_scale=A * 4 + 2)) == 2
    # outputs over inputs and over one another; T == 0 is a no-op
    assert _norm(lib, _block(), h=A * 5) == 5
    assert _norm(lib, _block(), h=A * 7 + 64) == 5
    assert _norm(lib, _block(), ro=A * 6 + 2) == 5
    assert _norm(lib, _block(), ro=A * 6, rs=128) == 5
    assert _norm(lib, _block(gate_form=3), h=A * 3) == 5
    assert _norm(lib, _block(), h=A * 2) == 5
    assert _norm(lib, _block(tokens=0, gate=None, res_scale=None), y=None, r=None, ro=None, h=None) == 0
    # checkpoints: format, missing parts, overlap
    ck = _ckpt(A * 10, A * 11)
    assert _norm(lib, _block(), fmt=0, cy=ck) == 3
    assert _norm(lib, _block(), fmt=3, cr=ck) == 3
    assert _norm(lib, _block(), fmt=1, ch=_ckpt(A * 10, None)) == 1
    assert _norm(lib, _block(), fmt=1, cy=ck, cr=ck) == 5
    assert _norm(lib, _block(), fmt=2, cy=_ckpt(A * 7 + 8, A * 11)) == 5


def _back(lib, b, dr=A * 20, drs=64, dh=A * 21, dhs=64, y=A * 22, ys=64, r=A * 23, rs=64, fmt=0, cy=None, cr=None,
          rstd=A * 24, dy=A * 25, dres=A * 26, dw1=A * 27, dw2=A * 28, dg=A * 29, ds=A * 30, ws=A * 31,
          wsb=1 << 19):
    return lib.mhc_block_norm_backward(b, _P(dr), drs, _P(dh), dhs, _P(y), ys, _P(r), rs, fmt, cy, cr, _P(rstd),
                                       _P(dy), _P(dres), _P(dw1), _P(dw2), _P(dg), _P(ds), _P(ws), wsb, None)


def test_refusals_of_the_backward_pass(lib):
    assert _back(lib, None) == 1
    assert _back(lib, _block(hidden=0)) == 4
    for k in ("dh", "y", "r", "rstd", "dy", "dres", "ws"):
        assert _back(lib, _block(), **{k: None}) == 1, k
    for k in ("drs", "dhs", "ys", "rs"):
        assert _back(lib, _block(), **{k: -1}) == 3, k
    assert _back(lib, _block(), wsb=16) == 8
    ck = _ckpt(A * 40, A * 41)
    assert _back(lib, _block(), fmt=1, cy=ck) == 3                    # y and its checkpoint
    assert _back(lib, _block(), fmt=0, cy=ck, y=None) == 3
    assert _back(lib, _block(), fmt=1, cy=_ckpt(None, A * 41), y=None) == 1
    # gradients of what is not there
    assert _back(lib, _block(w_post=None)) == 3
    assert _back(lib, _block(w_pre=None)) == 3
    assert _back(lib, _block(gate_form=0, gate=None)) == 3
    assert _back(lib, _block(scale_form=0, res_scale=None)) == 3
    for k, odd in (("dy", A * 25 + 1), ("dw1", A * 27 + 2), ("dg", A * 29 + 2), ("ws", A * 31 + 8), ("rstd", A * 24 + 1)):
        assert _back(lib, _block(), **{k: odd}) == 2, k
    assert _back(lib, _block(), dy=A * 22) == 5
    assert _back(lib, _block(), dres=A * 20, drs=128) == 5
    assert _back(lib, _block(), dres=A * 20 + 2) == 5
    assert _back(lib, _block(), dw1=A * 28) == 5
    assert _back(lib, _block(), ws=A * 24 - 64) == 5
    assert _back(lib, _block(), fmt=1, cr=_ckpt(A * 26, A * 41), r=None) == 5


def test_refusals_of_the_checkpoints(lib):
    ck = _ckpt(A * 2, A * 3)
    ok = [_P(A), 64, 1, 4, 64, 1]
    assert lib.mhc_ckpt_pack(*ok[:3], -1, 64, 1, ck, None) == 3
    assert lib.mhc_ckpt_pack(_P(A), -1, 1, 4, 64, 1, ck, None) == 3
    assert lib.mhc_ckpt_pack(_P(A), 64, 5, 4, 64, 1, ck, None) == 3
    assert lib.mhc_ckpt_pack(_P(A), 64, 1, 4, 64, 0, ck, None) == 3
    assert lib.mhc_ckpt_pack(_P(A), 64, 1, 4, 0, 1, ck, None) == 4
    assert lib.mhc_ckpt_pack(_P(A), 64, 1, 4, 65537, 1, ck, None) == 4
    assert lib.mhc_ckpt_pack(None, 64, 1, 4, 64, 1, ck, None) == 1
    assert lib.mhc_ckpt_pack(*ok, None, None) == 1
    assert lib.mhc_ckpt_pack(*ok, _ckpt(A * 2, None), None) == 1
    assert lib.mhc_ckpt_pack(_P(A + 1), 64, 1, 4, 64, 1, ck, None) == 2
    assert lib.mhc_ckpt_pack(*ok, _ckpt(A + 16, A * 3), None) == 5
    assert lib.mhc_ckpt_pack(None, 64, 1, 0, 64, 1, None, None) == 0
    un = [ck, 1, 4, 64, 1]
    assert lib.mhc_ckpt_unpack(ck, 0, 4, 64, 1, _P(A), None) == 3
    assert lib.mhc_ckpt_unpack(ck, 1, -4, 64, 1, _P(A), None) == 3
    assert lib.mhc_ckpt_unpack(ck, 1, 4, 64, 9, _P(A), None) == 3
    assert lib.mhc_ckpt_unpack(ck, 1, 4, 0, 1, _P(A), None) == 4
    assert lib.mhc_ckpt_unpack(*un, None, None) == 1
    assert lib.mhc_ckpt_unpack(None, 1, 4, 64, 1, _P(A), None) == 1
    assert lib.mhc_ckpt_unpack(*un, _P(A + 1), None) == 2
    assert lib.mhc_ckpt_unpack(*un, _P(A * 2), None) == 5
    assert lib.mhc_ckpt_unpack(None, 1, 0, 64, 1, None, None) == 0


def test_refusals_of_the_weight_gradient(lib):
    ck = _ckpt(A * 2, A * 3)

    def dw(d=A, s=64, t=1, x=ck, fmt=1, T=4, n=64, k=32, w=A * 4, wt=0, acc=0, ws=A * 5, wsb=1 << 19):
        return lib.mhc_ckpt_linear_dw(_P(d), s, t, x, fmt, T, n, k, _P(w), wt, acc, _P(ws), wsb, None)

    assert dw(T=-1) == 3
    assert dw(s=-64) == 3
    assert dw(fmt=0) == 3
    assert dw(wt=4) == 3
    assert dw(t=0) == 4                       # an fp32 gradient
    for bad in (dict(n=0), dict(k=0), dict(n=65537), dict(k=65537)):
        assert dw(**bad) == 4, bad
    for bad in (dict(d=None), dict(x=None), dict(w=None), dict(x=_ckpt(None, A))):
        assert dw(**bad) == 1, bad
    assert dw(d=A + 1) == 2
    assert dw(w=A * 4 + 2) == 2
    assert dw(ws=A * 5 + 8) == 2
    assert dw(w=A * 2) == 5
    assert dw(w=A + 128) == 5
    assert dw(T=0, acc=1, d=None, x=None) == 0


def test_workspace_sizes(lib):
    assert ops.block_norm_backward_workspace_bytes(0, 64) == 0
    assert ops.block_norm_backward_workspace_bytes(4, 0) == 0
    assert ops.block_norm_backward_workspace_bytes(4, 64) >= 4 * 2 * 64 * 4
    # no more than the most CTAs' sums however many tokens
    assert ops.block_norm_backward_workspace_bytes(1 << 20, 64) == ops.block_norm_backward_workspace_bytes(1 << 30, 64)
    assert ops.ckpt_linear_dw_workspace_bytes(0, 64, 64) == 0


def test_the_binding_refuses_on_the_host(lib):
    y = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.mhc_block_norm(y, y)
    with pytest.raises(ValueError, match="CUDA"):
        ops.mhc_ckpt_pack(y)
    with pytest.raises(ValueError, match="format"):
        ops.Checkpoint(y, y, "e5m2")
    with pytest.raises(ValueError, match="codes"):
        ops.Checkpoint(y, y, "e4m3")
