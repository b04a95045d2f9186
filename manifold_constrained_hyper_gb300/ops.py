"""Thin ctypes binding of libmhc.so (include/mhc.h).

Argument marshalling only: every step of the boundary runs in the library's
CUDA kernels. Tensors are torch CUDA tensors (bf16 tensors travel as their
bit patterns); outputs are allocated with torch when not given; the call is
enqueued on torch's current stream. There is no fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct
from contextlib import nullcontext
from dataclasses import dataclass
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmhc.so")
_lib = None

MHC_F32, MHC_BF16, MHC_F16 = 0, 1, 2
STATUS_NAMES = {0: "MHC_OK", 1: "MHC_ERR_NULL", 2: "MHC_ERR_ALIGN", 3: "MHC_ERR_SHAPE",
                4: "MHC_ERR_UNSUPPORTED", 5: "MHC_ERR_ALIAS", 6: "MHC_ERR_CUDA",
                7: "MHC_ERR_DEVICE_TIMEOUT", 8: "MHC_ERR_WORKSPACE"}

# every entry point include/mhc.h declares
EXPORTS = ("mhc_weight_bytes", "mhc_prepare_weight", "mhc_post", "mhc_workspace_bytes",
           "mhc_pre", "mhc_boundary_fused", "mhc_get_device_status", "mhc_last_timeout_site",
           "mhc_status_string", "mhc_set_wait_timeout_ns", "mhc_debug_unarmed_wait",
           "mhc_plan", "mhc_debug_record_between", "mhc_boundary_fused_noalloc",
           "mhc_debug_rcp_check", "mhc_pre_split_k", "mhc_debug_coef_check", "mhc_plan_cluster",
           "mhc_debug_set_decode_path", "mhc_debug_set_pdl", "mhc_debug_delayed_copy",
           "mhc_debug_launch_count", "mhc_block_norm", "mhc_block_norm_backward",
           "mhc_block_norm_backward_workspace_bytes", "mhc_ckpt_pack", "mhc_ckpt_unpack",
           "mhc_ckpt_linear_dw", "mhc_ckpt_linear_dw_workspace_bytes")


class MhcError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


class _Params(ctypes.Structure):
    _fields_ = [("hc_norm_eps", ctypes.c_float), ("hc_pre_eps", ctypes.c_float),
                ("hc_post_mult", ctypes.c_float), ("sinkhorn_eps", ctypes.c_float),
                ("norm_eps", ctypes.c_float), ("sinkhorn_iters", ctypes.c_int),
                ("batch_invariant", ctypes.c_int)]


# mhc_block and mhc_ckpt of include/mhc.h, packed by hand: a third of what
# filling a ctypes structure costs
_BLOCK = struct.Struct("@qiiiPPiiPiiiqPifffi4x")
_CKPT = struct.Struct("@PP")


@dataclass
class Params:
    hc_norm_eps: float = 1e-6
    hc_pre_eps: float = 1e-6
    hc_post_mult: float = 2.0
    sinkhorn_eps: float = 1e-6
    norm_eps: float = 1e-6
    sinkhorn_iters: int = 20
    batch_invariant: bool = False

    def c(self) -> _Params:
        return _Params(self.hc_norm_eps, self.hc_pre_eps, self.hc_post_mult,
                       self.sinkhorn_eps, self.norm_eps, int(self.sinkhorn_iters),
                       int(bool(self.batch_invariant)))


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libmhc.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    PP = ctypes.POINTER(_Params)
    PB = PC = P                    # structures as bytes
    sig = {
        "mhc_weight_bytes": (sz, [i32]),
        "mhc_prepare_weight": (i32, [P, i32, P, P]),
        "mhc_post": (i32, [P, P, P, P, P, i64, i32, P]),
        "mhc_workspace_bytes": (sz, [i64, i32]),
        "mhc_pre": (i32, [P, P, P, P, P, i32, PP, i64, i32, P, P, P, P, P, sz, P]),
        "mhc_boundary_fused": (i32, [P, P, P, P, P, P, P, P, P, i32, PP, i64, i32,
                                     P, P, P, P, P, P, sz, P]),
        "mhc_boundary_fused_noalloc": (i32, [P, P, P, P, P, P, P, P, P, i32, PP, i64, i32,
                                             P, P, P, P, P, P]),
        "mhc_get_device_status": (i32, [P]),
        "mhc_last_timeout_site": (i32, []),
        "mhc_status_string": (ctypes.c_char_p, [i32]),
        "mhc_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
        "mhc_debug_unarmed_wait": (i32, [P]),
        "mhc_debug_record_between": (None, [P]),
        "mhc_debug_rcp_check": (i32, [ctypes.c_uint32, ctypes.c_uint64, P, P]),
        "mhc_debug_coef_check": (i32, [P, P, P, PP, i32, i64, P, P, P]),
        "mhc_pre_split_k": (i32, [P, P, P, i32, P, P, P, i32, PP, i64, i32, P, P, P, P, P]),
        "mhc_plan": (i32, [i64, i32, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
        "mhc_plan_cluster": (i32, [i64, i32, ctypes.POINTER(ctypes.c_int)]),
        "mhc_debug_set_decode_path": (None, [i32]),
        "mhc_debug_set_pdl": (None, [i32]),
        "mhc_debug_delayed_copy": (i32, [P, P, i64, ctypes.c_uint32, P]),
        "mhc_debug_launch_count": (ctypes.c_uint64, []),
        "mhc_block_norm": (i32, [PB, P, i64, P, i64, P, P, P, i32, PC, PC, PC, P]),
        "mhc_block_norm_backward_workspace_bytes": (sz, [i64, i32]),
        "mhc_block_norm_backward": (i32, [PB, P, i64, P, i64, P, i64, P, i64, i32, PC, PC, P, P, P,
                                          P, P, P, P, P, sz, P]),
        "mhc_ckpt_pack": (i32, [P, i64, i32, i64, i32, i32, PC, P]),
        "mhc_ckpt_unpack": (i32, [PC, i32, i64, i32, i32, P, P]),
        "mhc_ckpt_linear_dw_workspace_bytes": (sz, [i64, i32, i32, i32]),
        "mhc_ckpt_linear_dw": (i32, [P, i64, i32, PC, i32, i64, i32, i32, P, i32, i32, P, sz, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(code: int, where: str):
    if code != 0:
        raise MhcError(code, where)


def _p(t):
    # plain ints: the argtypes convert them (cheaper than c_void_p objects)
    return None if t is None else t.data_ptr()


# The current stream's raw handle without building a Stream object (the
# public call costs several microseconds per call on some hosts).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, device=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        idx = device.index if device is not None and device.index is not None \
            else torch.cuda.current_device()
        return _raw_stream(idx)
    return torch.cuda.current_stream().cuda_stream


_DEFAULT_PARAMS_C = None


def _params_c(params):
    """ctypes struct of `params`; the default one is built once."""
    global _DEFAULT_PARAMS_C
    if params is not None:
        return params.c()
    if _DEFAULT_PARAMS_C is None:
        _DEFAULT_PARAMS_C = Params().c()
    return _DEFAULT_PARAMS_C


def _bf16(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    return t


def _f32(t: torch.Tensor, name: str):
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA float32 tensor")
    return t


def weight_bytes(hidden: int) -> int:
    return int(load().mhc_weight_bytes(hidden))


def workspace_bytes(tokens: int, hidden: int) -> int:
    return int(load().mhc_workspace_bytes(tokens, hidden))


def plan(tokens: int, hidden: int):
    s, w = ctypes.c_int(), ctypes.c_int()
    _check(load().mhc_plan(tokens, hidden, ctypes.byref(s), ctypes.byref(w)), "mhc_plan")
    return s.value, w.value


def plan_cluster(tokens: int, hidden: int) -> int:
    """Cluster size of a shifted call of (tokens, hidden) on the current
    device, or 0 when it takes the slice-parallel streaming kernel."""
    c = ctypes.c_int()
    _check(load().mhc_plan_cluster(tokens, hidden, ctypes.byref(c)), "mhc_plan_cluster")
    return c.value


def mhc_debug_set_decode_path(path: int):
    """0 (the default): the cluster kernel where it is the faster path; 1:
    every later shifted call takes the slice-parallel streaming kernel; 2:
    the cluster kernel wherever it can run."""
    load().mhc_debug_set_decode_path(int(path))


def mhc_debug_set_pdl(enable: bool):
    """Launch the boundary kernels as programmatic dependents (the default)
    or as plain stream kernels."""
    load().mhc_debug_set_pdl(int(bool(enable)))


def mhc_debug_launch_count() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().mhc_debug_launch_count())


def mhc_debug_delayed_copy(src, dst, delay_ns: int, stream=None):
    """dst <- src (bf16, same size) by a kernel that lets the next kernel on
    the stream start at once and writes only after delay_ns."""
    _bf16(src, "src"), _bf16(dst, "dst")
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have the same size")
    _check(load().mhc_debug_delayed_copy(_p(src), _p(dst), src.numel(), int(delay_ns),
                                         _stream(stream, src.device)), "mhc_debug_delayed_copy")


def mhc_prepare_weight(fn: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """fn [24, 4H] fp32 -> prepared mixer (uint8, mhc_weight_bytes(H) bytes)."""
    _f32(fn, "fn")
    H = fn.shape[1] // 4
    if out is None:
        out = torch.empty(weight_bytes(H), dtype=torch.uint8, device=fn.device)
    _check(load().mhc_prepare_weight(_p(fn), H, _p(out), _stream(stream)), "mhc_prepare_weight")
    return out


def mhc_post(x, residual, post, comb, out=None, stream=None):
    """Residual update: returns residual_out [T, 4, H] bf16 (may be residual)."""
    _bf16(x, "x"), _bf16(residual, "residual"), _f32(post, "post"), _f32(comb, "comb")
    T, n, H = residual.shape
    if out is None:
        out = torch.empty_like(residual)
    _check(load().mhc_post(_p(x), _p(residual), _p(post), _p(comb), _p(out), T, H,
                           _stream(stream)), "mhc_post")
    return out


def _outs(T, H, dev, layer_input, pre_out, post_out, comb_out, workspace):
    if layer_input is None:
        layer_input = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if pre_out is None:
        pre_out = torch.empty(T, 4, dtype=torch.float32, device=dev)
    if post_out is None:
        post_out = torch.empty(T, 4, dtype=torch.float32, device=dev)
    if comb_out is None:
        comb_out = torch.empty(T, 4, 4, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(workspace_bytes(T, H), 16), dtype=torch.uint8, device=dev)
    return layer_input, pre_out, post_out, comb_out, workspace


def _nw(norm_w):
    if norm_w is None:
        return None, MHC_F32
    if norm_w.dtype == torch.bfloat16:
        return norm_w, MHC_BF16
    return _f32(norm_w, "norm_w"), MHC_F32


def mhc_pre(residual, weight, scale, base, norm_w=None, params: Params | None = None, *,
            layer_input=None, pre_out=None, post_out=None, comb_out=None, workspace=None,
            stream=None):
    """Unshifted pre: returns (layer_input, pre, post, comb)."""
    _bf16(residual, "residual")
    T, n, H = residual.shape
    li, pr, po, cb, ws = _outs(T, H, residual.device, layer_input, pre_out, post_out,
                               comb_out, workspace)
    nw, nwt = _nw(norm_w)
    p = _params_c(params)
    _check(load().mhc_pre(_p(residual), _p(weight), _p(scale), _p(base), _p(nw), nwt,
                          ctypes.byref(p), T, H, _p(li), _p(pr), _p(po), _p(cb), _p(ws),
                          ws.numel() * ws.element_size(), _stream(stream, residual.device)), "mhc_pre")
    return li, pr, po, cb


def mhc_pre_split_k(residual, dot_mix, sqrsum, scale, base, norm_w=None,
                    params: Params | None = None, *, layer_input=None, pre_out=None,
                    post_out=None, comb_out=None, stream=None):
    """Unshifted pre from split-K partial mixes dot_mix [S, T, 24] and partial
    sums of squares sqrsum [S, T]: returns (layer_input, pre, post, comb)."""
    _bf16(residual, "residual"), _f32(dot_mix, "dot_mix"), _f32(sqrsum, "sqrsum")
    T, n, H = residual.shape
    S = dot_mix.shape[0]
    if tuple(dot_mix.shape) != (S, T, 24) or tuple(sqrsum.shape) != (S, T):
        raise ValueError("dot_mix must be [S, T, 24] and sqrsum [S, T]")
    dev = residual.device
    li = layer_input if layer_input is not None else torch.empty(T, H, dtype=torch.bfloat16,
                                                                 device=dev)
    pr = pre_out if pre_out is not None else torch.empty(T, 4, device=dev)
    po = post_out if post_out is not None else torch.empty(T, 4, device=dev)
    cb = comb_out if comb_out is not None else torch.empty(T, 4, 4, device=dev)
    nw, nwt = _nw(norm_w)
    p = _params_c(params)
    _check(load().mhc_pre_split_k(_p(residual), _p(dot_mix), _p(sqrsum), S, _p(scale), _p(base),
                                  _p(nw), nwt, ctypes.byref(p), T, H, _p(li), _p(pr), _p(po),
                                  _p(cb), _stream(stream, residual.device)), "mhc_pre_split_k")
    return li, pr, po, cb


def mhc_boundary_fused(x, residual, post, comb, weight, scale, base, norm_w=None, pre_lag=None,
                       params: Params | None = None, *, residual_out=None, layer_input=None,
                       pre_out=None, post_out=None, comb_out=None, workspace=None, stream=None):
    """Fused post + pre boundary (shifted when pre_lag is given). Returns
    (residual_out, layer_input, pre, post, comb)."""
    _bf16(x, "x"), _bf16(residual, "residual"), _f32(post, "post"), _f32(comb, "comb")
    if pre_lag is not None:
        _f32(pre_lag, "pre_lag")
    T, n, H = residual.shape
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    li, pr, po, cb, ws = _outs(T, H, residual.device, layer_input, pre_out, post_out,
                               comb_out, workspace)
    nw, nwt = _nw(norm_w)
    p = _params_c(params)
    _check(load().mhc_boundary_fused(
        _p(x), _p(residual), _p(post), _p(comb), _p(pre_lag), _p(weight), _p(scale), _p(base),
        _p(nw), nwt, ctypes.byref(p), T, H, _p(residual_out), _p(li), _p(pr), _p(po), _p(cb),
        _p(ws), ws.numel() * ws.element_size(), _stream(stream, residual.device)), "mhc_boundary_fused")
    return residual_out, li, pr, po, cb


def mhc_boundary_fused_noalloc(x, residual, post, comb, weight, scale, base, norm_w=None,
                               pre_lag=None, params: Params | None = None, *,
                               residual_out=None, layer_input=None, pre_out=None,
                               post_out=None, comb_out=None, stream=None):
    """mhc_boundary_fused whose scratch is the library's fixed device array
    (for callers that cannot allocate device memory). Outputs not given are
    allocated here with torch; pass them all to allocate nothing."""
    _bf16(x, "x"), _bf16(residual, "residual"), _f32(post, "post"), _f32(comb, "comb")
    if pre_lag is not None:
        _f32(pre_lag, "pre_lag")
    T, n, H = residual.shape
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    dev = residual.device
    li = layer_input if layer_input is not None else torch.empty(T, H, dtype=torch.bfloat16,
                                                                 device=dev)
    pr = pre_out if pre_out is not None else torch.empty(T, 4, device=dev)
    po = post_out if post_out is not None else torch.empty(T, 4, device=dev)
    cb = comb_out if comb_out is not None else torch.empty(T, 4, 4, device=dev)
    nw, nwt = _nw(norm_w)
    p = _params_c(params)
    _check(load().mhc_boundary_fused_noalloc(
        _p(x), _p(residual), _p(post), _p(comb), _p(pre_lag), _p(weight), _p(scale), _p(base),
        _p(nw), nwt, ctypes.byref(p), T, H, _p(residual_out), _p(li), _p(pr), _p(po), _p(cb),
        _stream(stream, residual.device)), "mhc_boundary_fused_noalloc")
    return residual_out, li, pr, po, cb


def mhc_get_device_status(stream=None) -> int:
    return int(load().mhc_get_device_status(_stream(stream)))


def mhc_last_timeout_site() -> int:
    return int(load().mhc_last_timeout_site())


def mhc_set_wait_timeout_ns(ns: int):
    load().mhc_set_wait_timeout_ns(int(ns))


def mhc_debug_unarmed_wait(stream=None):
    _check(load().mhc_debug_unarmed_wait(_stream(stream)), "mhc_debug_unarmed_wait")


def mhc_debug_coef_check(values, scale, base, hidden: int, params: Params | None = None,
                         stream=None):
    """Coefficients of the tokens of `values` [n, 25] (fp32, CUDA) formed by
    the one-thread and the 16-lane routines: returns (out_thread, out_lanes),
    each [n, 24] (pre 4, post 4, comb 16)."""
    for t in (values, scale, base):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("values, scale and base must be contiguous CUDA float32 tensors")
    n = values.shape[0]
    p = _params_c(params)
    a = torch.empty(n, 24, dtype=torch.float32, device=values.device)
    b = torch.empty(n, 24, dtype=torch.float32, device=values.device)
    _check(load().mhc_debug_coef_check(_p(values), _p(scale), _p(base), ctypes.byref(p),
                                       int(hidden), n, _p(a), _p(b), _stream(stream)),
           "mhc_debug_coef_check")
    return a, b


def mhc_debug_rcp_check(first_bits: int, count: int, stream=None):
    """(number of bit patterns in [first_bits, first_bits + count) whose
    library reciprocal differs from the correctly rounded one, smallest such
    pattern or None)."""
    s = stream if stream is not None else torch.cuda.current_stream()
    res = torch.tensor([0, -1], dtype=torch.int64, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    _check(load().mhc_debug_rcp_check(first_bits, count, ctypes.c_void_p(res.data_ptr()),
                                      _stream(s)), "mhc_debug_rcp_check")
    s.synchronize()
    n, first = (int(v) for v in res.cpu().tolist())
    return n, (None if n == 0 else first & 0xFFFFFFFF)


def mhc_debug_record_between(event):
    """Record `event` (torch.cuda.Event) between the streaming and finishing
    kernels of this thread's next mhc_pre / mhc_boundary_fused call."""
    load().mhc_debug_record_between(ctypes.c_void_p(event.cuda_event) if event else None)


def mhc_status_string(code: int) -> str:
    return load().mhc_status_string(int(code)).decode()


# ---------------------------------------------------------------------------
# Gated residual block, its backward pass, and 8-bit activation checkpoints

_DTYPES = {torch.float32: MHC_F32, torch.bfloat16: MHC_BF16, torch.float16: MHC_F16}
_GATE_NONE, _GATE_CHANNEL, _GATE_TOKEN, _GATE_FULL = 0, 1, 2, 3
_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}
_SCALE_NONE, _SCALE_ONE, _SCALE_CHANNEL = 0, 1, 2
_FORMATS = {"e4m3": 1, "int8": 2}
CKPT_GROUP = 32


@dataclass
class BlockParams:
    """What shapes a gated residual block beside its tensors. gate_act: "none",
    "sigmoid" or "tanh", applied to the gate. weight_offset is added to both
    norms' weights (1 where they are kept as w - 1). post_norm False leaves the
    norm of the block's output out."""
    eps_post: float = 1e-6
    eps_pre: float = 1e-6
    gate_act: str = "none"
    weight_offset: float = 0.0
    post_norm: bool = True


_DEFAULT_BLOCK_PARAMS = BlockParams()


class Checkpoint:
    """An activation [T, H] kept in 8 bits: codes [T, H] and scales
    [T, ceil(H / 32)], uint8 and contiguous, in fmt "e4m3" or "int8"."""

    __slots__ = ("codes", "scales", "fmt")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: str):
        if fmt not in _FORMATS:
            raise ValueError(f"checkpoint format must be one of {sorted(_FORMATS)}: got {fmt!r}")
        for t, name in ((codes, "codes"), (scales, "scales")):
            if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous 2-D CUDA uint8 tensor")
        T, H = codes.shape
        if tuple(scales.shape) != (T, -(-H // CKPT_GROUP)) or scales.device != codes.device:
            raise ValueError(f"scales must be [{T}, {-(-H // CKPT_GROUP)}] on the codes' device: "
                             f"got {tuple(scales.shape)}")
        self.codes, self.scales, self.fmt = codes, scales, fmt

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device

    def _c(self):
        return _CKPT.pack(self.codes.data_ptr(), self.scales.data_ptr())


class BlockGrads(NamedTuple):
    """Gradients of mhc_block_norm's inputs; None where there is no such input."""
    d_y: torch.Tensor
    d_residual: torch.Tensor
    d_w_post: torch.Tensor | None
    d_w_pre: torch.Tensor | None
    d_gate: torch.Tensor | None
    d_res_scale: torch.Tensor | None


_NOWHERE_ELSE = nullcontext()


def _on(stream):
    """Where outputs and workspaces of a call on `stream` are allocated: there."""
    return torch.cuda.stream(stream) if stream is not None else _NOWHERE_ELSE


def ckpt_empty(tokens: int, hidden: int, fmt: str = "e4m3", device="cuda") -> Checkpoint:
    """A checkpoint to be written."""
    if fmt not in _FORMATS:
        raise ValueError(f"checkpoint format must be one of {sorted(_FORMATS)}: got {fmt!r}")
    c = Checkpoint.__new__(Checkpoint)
    c.codes = torch.empty((tokens, hidden), dtype=torch.uint8, device=device)
    c.scales = torch.empty((tokens, -(-hidden // CKPT_GROUP)), dtype=torch.uint8, device=device)
    c.fmt = fmt
    return c


def _matrix(t, name, shape, dtype, device):
    """A CUDA tensor `shape` = [T, H] of `dtype` whose rows are contiguous: its row stride."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return shape[1]
        if shape[1] == 1 or t.stride(1) == 1:
            return t.stride(0)
    raise ValueError(f"{name} must be a {list(shape)} {dtype} tensor on {device} with contiguous "
                     f"rows: got {list(t.shape)} {t.dtype} on {t.device}")


def _whole(t, name, shape, dtype, device):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor on {device}: "
                         f"got {list(t.shape)} {t.dtype} on {t.device}")
    return t


def _out(t, name, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None \
        else _whole(t, name, shape, dtype, device)


def _held(c, name, shape, device):
    if c.codes.shape != shape or c.codes.device != device:
        raise ValueError(f"{name} must be a {list(shape)} checkpoint on {device}: got "
                         f"{list(c.codes.shape)} on {c.codes.device}")
    return c._c()


def _format(*cks):
    """The one format of the checkpoints given (0: none given)."""
    fmt = None
    for c in cks:
        if c is not None:
            if fmt is not None and c.fmt != fmt:
                raise ValueError("the checkpoints of a call must have one format")
            fmt = c.fmt
    return _FORMATS[fmt] if fmt is not None else 0


def _weight(w, name, H, device):
    if w is None:
        return 0, MHC_F32
    t = _DTYPES.get(w.dtype)
    if t is None or w.shape != (H,) or not w.is_contiguous() or w.device != device:
        raise ValueError(f"{name} must be a contiguous [{H}] float tensor on {device}: got "
                         f"{list(w.shape)} {w.dtype} on {w.device}")
    return w.data_ptr(), t


def _block_c(shape, dtype, r_dtype, device, w_post, w_pre, gate, res_scale, params):
    """The C struct of a block from its tensors, as bytes, and the gate's form (its
    and the scale's are told by their shapes)."""
    p = params if params is not None else _DEFAULT_BLOCK_PARAMS
    T, H = shape
    t = _DTYPES.get(dtype)
    if t is None or (r_dtype is not dtype and r_dtype is not torch.float32):
        raise ValueError(f"y must be float32, bfloat16 or float16 and residual the same or "
                         f"float32: got {dtype} and {r_dtype}")
    wp, wpt = _weight(w_post, "w_post", H, device)
    wq, wqt = _weight(w_pre, "w_pre", H, device)
    act = _ACTS.get(p.gate_act)
    if act is None or (act and gate is None):
        raise ValueError(f"gate_act must be one of {sorted(_ACTS)}, and \"none\" without a gate: "
                         f"got {p.gate_act!r}")
    form, gate_p, gate_t, gate_stride = _GATE_NONE, 0, MHC_F32, 0
    if gate is not None:
        gate_t = _DTYPES.get(gate.dtype)
        gs = gate.shape
        if (gate_t != t and gate_t != MHC_F32) or gate.device != device:
            raise ValueError(f"gate must be {dtype} or float32 on {device}: got {gate.dtype} on "
                             f"{gate.device}")
        if gs == (H,) and (gate.is_contiguous() or H == 1):
            form = _GATE_CHANNEL
        elif gs == (T, 1):
            form, gate_stride = _GATE_TOKEN, gate.stride(0)
        elif gs == shape and gate.stride(1) == 1:
            form, gate_stride = _GATE_FULL, gate.stride(0)
        else:
            raise ValueError(f"gate must be [{H}], [{T}, 1] or [{T}, {H}] with contiguous rows: "
                             f"got {list(gs)}")
        gate_p = gate.data_ptr()
    scale_form, scale_p = _SCALE_NONE, 0
    if res_scale is not None:
        n = res_scale.numel()
        if res_scale.dtype is not torch.float32 or res_scale.dim() > 1 or (n != 1 and n != H) \
                or not res_scale.is_contiguous() or res_scale.device != device:
            raise ValueError(f"res_scale must be a contiguous [1] or [{H}] float32 tensor on "
                             f"{device}: got {list(res_scale.shape)} {res_scale.dtype} on "
                             f"{res_scale.device}")
        scale_form, scale_p = (_SCALE_ONE if n == 1 else _SCALE_CHANNEL), res_scale.data_ptr()
    return _BLOCK.pack(T, H, t, MHC_F32 if r_dtype is torch.float32 else t, wp, wq, wpt, wqt, gate_p,
                       gate_t, form, act, gate_stride, scale_p, scale_form, p.eps_post, p.eps_pre,
                       p.weight_offset, 1 if p.post_norm else 0), form


def _cuda_2d(t, name):
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    return shape, t.device


def mhc_block_norm(y, residual, w_post=None, w_pre=None, gate=None, res_scale=None,
                   params: BlockParams | None = None, *, residual_out=None, h=None, rstd=None,
                   ckpt_y: Checkpoint | None = None, ckpt_residual: Checkpoint | None = None,
                   ckpt_h: Checkpoint | None = None, stream=None):
    """The gated residual block's boundary:

        n = y * rstd_post * w_post
        residual_out = res_scale * residual + act(gate) * n
        h = residual_out * rstd_pre * w_pre

    y [T, H] (float32, bfloat16 or float16) and residual [T, H] (the same or
    float32) may be strided rows; w_post, w_pre [H]; gate [H], [T, 1] or
    [T, H], of y's type or float32; res_scale [1] or [H] float32; each may be
    None. ckpt_y, ckpt_residual and ckpt_h are checkpoints to write of y,
    residual and h in the same pass. Returns (residual_out, h, rstd), rstd
    [T, 2] being what mhc_block_norm_backward needs beside y and residual.
    residual_out may be the residual itself."""
    shape, dev = _cuda_2d(y, "y")
    dtype, r_dtype = y.dtype, residual.dtype
    ys = _matrix(y, "y", shape, dtype, dev)
    rs = _matrix(residual, "residual", shape, r_dtype, dev)
    b, _ = _block_c(shape, dtype, r_dtype, dev, w_post, w_pre, gate, res_scale, params)
    fmt, cy, cr, ch = 0, None, None, None
    if ckpt_y is not None or ckpt_residual is not None or ckpt_h is not None:
        fmt = _format(ckpt_y, ckpt_residual, ckpt_h)
        cy = None if ckpt_y is None else _held(ckpt_y, "ckpt_y", shape, dev)
        cr = None if ckpt_residual is None else _held(ckpt_residual, "ckpt_residual", shape, dev)
        ch = None if ckpt_h is None else _held(ckpt_h, "ckpt_h", shape, dev)
    with _on(stream):
        residual_out = _out(residual_out, "residual_out", shape, r_dtype, dev)
        h = _out(h, "h", shape, dtype, dev)
        rstd = _out(rstd, "rstd", (shape[0], 2), torch.float32, dev)
    code = (_lib or load()).mhc_block_norm(b, y.data_ptr(), ys, residual.data_ptr(), rs,
                                           residual_out.data_ptr(), h.data_ptr(), rstd.data_ptr(),
                                           fmt, cy, cr, ch, _stream(stream, dev))
    if code:
        raise MhcError(code, "mhc_block_norm")
    return residual_out, h, rstd


def block_norm_backward_workspace_bytes(tokens: int, hidden: int) -> int:
    return int(load().mhc_block_norm_backward_workspace_bytes(tokens, hidden))


def mhc_block_norm_backward(d_residual_out, d_h, y, residual, rstd, w_post=None, w_pre=None,
                            gate=None, res_scale=None, params: BlockParams | None = None, *,
                            residual_dtype=None, d_y=None, d_residual=None, workspace=None,
                            stream=None) -> BlockGrads:
    """Gradients of mhc_block_norm's inputs from those of residual_out (None:
    zero) and h. y and residual are the inputs or Checkpoints of them; rstd,
    the weights, the gate, the scale and params as in the forward call.
    residual_dtype (d_residual_out's, else d_h's, unless given) is needed only
    where neither d_residual_out nor the residual itself tells it. The
    gradients of weights, of a [H] or [T, 1] gate and of res_scale are float32
    (those of [H] rows of one allocation); d_residual may be d_residual_out itself."""
    shape, dev = _cuda_2d(d_h, "d_h")
    T, H = shape
    dtype = d_h.dtype
    dhs = _matrix(d_h, "d_h", shape, dtype, dev)
    if residual_dtype is None:
        residual_dtype = d_residual_out.dtype if d_residual_out is not None \
            else residual.dtype if isinstance(residual, torch.Tensor) else dtype
    drs = 0 if d_residual_out is None else _matrix(d_residual_out, "d_residual_out", shape,
                                                   residual_dtype, dev)
    b, form = _block_c(shape, dtype, residual_dtype, dev, w_post, w_pre, gate, res_scale, params)
    cy = cr = yp = rp = None
    ys = rs = fmt = 0
    if isinstance(y, Checkpoint):
        cy, fmt = _held(y, "y", shape, dev), _FORMATS[y.fmt]
    else:
        yp, ys = y.data_ptr(), _matrix(y, "y", shape, dtype, dev)
    if isinstance(residual, Checkpoint):
        cr = _held(residual, "residual", shape, dev)
        fmt = _format(residual, y if cy is not None else None)
    else:
        rp, rs = residual.data_ptr(), _matrix(residual, "residual", shape, residual_dtype, dev)
    _whole(rstd, "rstd", (T, 2), torch.float32, dev)
    lib = _lib or load()
    f32 = torch.float32
    channel = form == _GATE_CHANNEL
    per_channel = res_scale is not None and res_scale.numel() != 1
    d_w_post = d_w_pre = d_gate = d_scale = None
    with _on(stream):
        d_y = _out(d_y, "d_y", shape, dtype, dev)
        d_residual = _out(d_residual, "d_residual", shape, residual_dtype, dev)
        rows = (w_post is not None) + (w_pre is not None) + channel + per_channel
        if rows:
            own = iter(torch.empty((rows, H), dtype=f32, device=dev).unbind(0))
            if w_post is not None:
                d_w_post = next(own)
            if w_pre is not None:
                d_w_pre = next(own)
            if channel:
                d_gate = next(own)
            if per_channel:
                d_scale = next(own)
        if gate is not None and not channel:
            d_gate = torch.empty(gate.shape, dtype=gate.dtype if form == _GATE_FULL else f32,
                                 device=dev)
        if res_scale is not None and not per_channel:
            d_scale = torch.empty(res_scale.shape, dtype=f32, device=dev)
        if workspace is None:
            need = lib.mhc_block_norm_backward_workspace_bytes(T, H)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    code = lib.mhc_block_norm_backward(
        b, _p(d_residual_out), drs, d_h.data_ptr(), dhs, yp, ys, rp, rs, fmt, cy, cr,
        rstd.data_ptr(), d_y.data_ptr(), d_residual.data_ptr(), _p(d_w_post), _p(d_w_pre),
        _p(d_gate), _p(d_scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if code:
        raise MhcError(code, "mhc_block_norm_backward")
    return BlockGrads(d_y, d_residual, d_w_post, d_w_pre, d_gate, d_scale)


def mhc_ckpt_pack(x, fmt: str = "e4m3", *, out: Checkpoint | None = None, stream=None) -> Checkpoint:
    """x [T, H] (float32, bfloat16 or float16, rows may be strided) kept in 8 bits."""
    shape, dev = _cuda_2d(x, "x")
    t = _DTYPES.get(x.dtype)
    if t is None:
        raise ValueError(f"x must be float32, bfloat16 or float16: got {x.dtype}")
    s = _matrix(x, "x", shape, x.dtype, dev)
    T, H = shape
    if out is None:
        with _on(stream):
            out = ckpt_empty(T, H, fmt, dev)
        c = out._c()
    else:
        if out.fmt != fmt:
            raise ValueError(f"out has the format {out.fmt!r}, not {fmt!r}")
        c = _held(out, "out", shape, dev)
    code = (_lib or load()).mhc_ckpt_pack(x.data_ptr(), s, t, T, H, _FORMATS[fmt], c,
                                          _stream(stream, dev))
    if code:
        raise MhcError(code, "mhc_ckpt_pack")
    return out


def mhc_ckpt_unpack(ckpt: Checkpoint, dtype=torch.bfloat16, *, out=None, stream=None):
    """The values [T, H] that a checkpoint stands for, in `dtype`."""
    t = _DTYPES.get(dtype)
    if t is None:
        raise ValueError(f"dtype must be float32, bfloat16 or float16: got {dtype}")
    shape = ckpt.codes.shape
    dev = ckpt.codes.device
    with _on(stream):
        out = _out(out, "out", shape, dtype, dev)
    code = (_lib or load()).mhc_ckpt_unpack(ckpt._c(), _FORMATS[ckpt.fmt], shape[0], shape[1], t,
                                            out.data_ptr(), _stream(stream, dev))
    if code:
        raise MhcError(code, "mhc_ckpt_unpack")
    return out


def ckpt_linear_dw_workspace_bytes(tokens: int, n: int, k: int, aligned: bool = True) -> int:
    """aligned: d_out's address and row stride (at least n) are multiples of 16 bytes."""
    return int(load().mhc_ckpt_linear_dw_workspace_bytes(tokens, n, k, int(aligned)))


def mhc_ckpt_linear_dw(d_out, x: Checkpoint, *, d_w=None, dtype=torch.float32,
                       accumulate: bool = False, workspace=None, stream=None):
    """d_w [N, K] = d_out^T x, the weight gradient of out = x W^T, from d_out
    [T, N] (bfloat16 or float16, rows may be strided) and the checkpoint of
    x [T, K]. accumulate adds to the d_w given."""
    shape, dev = _cuda_2d(d_out, "d_out")
    t_in = d_out.dtype
    if t_in is not torch.bfloat16 and t_in is not torch.float16:
        raise ValueError(f"d_out must be bfloat16 or float16: got {t_in}")
    s = _matrix(d_out, "d_out", shape, t_in, dev)
    T, N = shape
    K = x.codes.shape[1]
    c = _held(x, "x", (T, K), dev)
    if d_w is not None:
        dtype = d_w.dtype
    elif accumulate:
        raise ValueError("accumulate needs the d_w to add to")
    t = _DTYPES.get(dtype)
    if t is None:
        raise ValueError(f"d_w must be float32, bfloat16 or float16: got {dtype}")
    lib = _lib or load()
    dp = d_out.data_ptr()
    with _on(stream):
        d_w = _out(d_w, "d_w", (N, K), dtype, dev)
        if workspace is None:
            aligned = dp % 16 == 0 and ((s % 8 == 0 and N <= s < 1 << 38) or T == 1)
            need = lib.mhc_ckpt_linear_dw_workspace_bytes(T, N, K, aligned)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib.mhc_ckpt_linear_dw(dp, s, _DTYPES[t_in], c, _FORMATS[x.fmt], T, N, K,
                                  d_w.data_ptr(), t, 1 if accumulate else 0, _p(workspace), ws_bytes,
                                  _stream(stream, dev))
    if code:
        raise MhcError(code, "mhc_ckpt_linear_dw")
    return d_w
