"""Thin binding of libmhc.so (include/mhc.h): ctypes, and for the gated residual
block, the checkpoints and the weight gradient the C++ of csrc/binding.cpp.

Argument marshalling only: every step of the boundary runs in the library's
CUDA kernels. Tensors are torch CUDA tensors (bf16 tensors travel as their
bit patterns); outputs are allocated with torch when not given; the call is
enqueued on torch's current stream. There is no fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
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
    PB = PC = P                    # structures, by address
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
_FORMATS = {"e4m3": 1, "int8": 2}
CKPT_GROUP = 32
_fast = None


def load_binding():
    """The C++ binding (raises if it has not been built), over load()'s library."""
    global _fast
    if _fast is None:
        lib = load()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the C++ binding is missing: build it with `python -c 'import "
                               "__graft_entry__ as g; g.build()'`") from e
        _binding.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
            "mhc_block_norm", "mhc_block_norm_backward", "mhc_block_norm_backward_workspace_bytes",
            "mhc_ckpt_pack", "mhc_ckpt_unpack", "mhc_ckpt_linear_dw",
            "mhc_ckpt_linear_dw_workspace_bytes")), MhcError)
        _fast = _binding
    return _fast


def _at(stream, call, *args):
    """call(*args) with `stream` as torch's current one: its outputs and workspace are
    allocated there too."""
    if stream is None:
        return call(*args)
    with torch.cuda.stream(stream):
        return call(*args)


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


class BlockGrads(NamedTuple):
    """Gradients of mhc_block_norm's inputs; None where there is no such input."""
    d_y: torch.Tensor
    d_residual: torch.Tensor
    d_w_post: torch.Tensor | None
    d_w_pre: torch.Tensor | None
    d_gate: torch.Tensor | None
    d_res_scale: torch.Tensor | None


def _held(codes, scales, fmt) -> Checkpoint:
    c = Checkpoint.__new__(Checkpoint)
    c.codes, c.scales, c.fmt = codes, scales, fmt
    return c


def _format_number(fmt):
    n = _FORMATS.get(fmt)
    if n is None:
        raise ValueError(f"checkpoint format must be one of {sorted(_FORMATS)}: got {fmt!r}")
    return n


def ckpt_empty(tokens: int, hidden: int, fmt: str = "e4m3", device="cuda") -> Checkpoint:
    """A checkpoint to be written."""
    _format_number(fmt)
    d = device if isinstance(device, torch.device) else torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"a checkpoint lies on a CUDA device: got {d}")
    return _held(*(_fast or load_binding()).ckpt_empty(tokens, hidden, -1 if d.index is None else d.index), fmt)


def _format(*cks):
    """The one format of the checkpoints given (0: none given)."""
    fmt = None
    for c in cks:
        if c is not None:
            if fmt is not None and c.fmt != fmt:
                raise ValueError("the checkpoints of a call must have one format")
            fmt = c.fmt
    return _FORMATS[fmt] if fmt is not None else 0


def _parts(c):
    return (None, None) if c is None else (c.codes, c.scales)


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
    residual_out may be the residual itself. No history is recorded: while
    gradients are, tensors that require them are refused (wrap the two
    directions in a torch.autograd.Function, or call under no_grad)."""
    f = (_fast or load_binding()).block_norm
    p = _DEFAULT_BLOCK_PARAMS if params is None else params
    if ckpt_y is None and ckpt_residual is None and ckpt_h is None:
        return _at(stream, f, y, residual, w_post, w_pre, gate, res_scale, p, residual_out, h, rstd,
                   0, None, None, None, None, None, None)
    return _at(stream, f, y, residual, w_post, w_pre, gate, res_scale, p, residual_out, h, rstd,
               _format(ckpt_y, ckpt_residual, ckpt_h), *_parts(ckpt_y), *_parts(ckpt_residual),
               *_parts(ckpt_h))


def block_norm_backward_workspace_bytes(tokens: int, hidden: int) -> int:
    return int(load().mhc_block_norm_backward_workspace_bytes(tokens, hidden))


def mhc_block_norm_backward(d_residual_out, d_h, y, residual, rstd, w_post=None, w_pre=None,
                            gate=None, res_scale=None, params: BlockParams | None = None, *,
                            residual_dtype=None, d_y=None, d_residual=None, workspace=None,
                            stream=None) -> BlockGrads:
    """Gradients of mhc_block_norm's inputs from those of residual_out (None:
    zero) and h. y and residual are the inputs or Checkpoints of them; rstd,
    the weights, the gate, the scale and params as in the forward call.
    residual_dtype (d_residual_out's, else the residual's, else d_h's, unless
    given) is needed only where none of them tells it. The gradients of
    weights, of a [H] or [T, 1] gate and of res_scale are float32 (always parts
    of one allocation); d_residual may be d_residual_out itself. Not
    differentiable itself: gradients of outputs that require grad are refused
    while gradients are recorded."""
    f = (_fast or load_binding()).block_norm_backward
    p = _DEFAULT_BLOCK_PARAMS if params is None else params
    typed = None if residual_dtype is None else torch.empty(0, dtype=residual_dtype)
    cy = y if isinstance(y, Checkpoint) else None
    cr = residual if isinstance(residual, Checkpoint) else None
    if cy is None and cr is None:
        return BlockGrads._make(_at(stream, f, d_residual_out, d_h, y, residual, rstd, w_post, w_pre, gate,
                                    res_scale, p, typed, d_y, d_residual, workspace, 0, None, None, None, None))
    return BlockGrads._make(_at(
        stream, f, d_residual_out, d_h, y if cy is None else None, residual if cr is None else None,
        rstd, w_post, w_pre, gate, res_scale, p, typed, d_y, d_residual, workspace, _format(cy, cr),
        *_parts(cy), *_parts(cr)))


def mhc_ckpt_pack(x, fmt: str = "e4m3", *, out: Checkpoint | None = None, stream=None) -> Checkpoint:
    """x [T, H] (float32, bfloat16 or float16, rows may be strided) kept in 8 bits:
    its values, as of a detached tensor."""
    f = (_fast or load_binding()).ckpt_pack
    if out is None:
        return _held(*_at(stream, f, x, _format_number(fmt), None, None), fmt)
    if out.fmt != fmt:
        raise ValueError(f"out has the format {out.fmt!r}, not {fmt!r}")
    _at(stream, f, x, _format_number(fmt), out.codes, out.scales)
    return out


def _dtype_number(dtype, name):
    t = _DTYPES.get(dtype)
    if t is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16: got {dtype}")
    return t


def mhc_ckpt_unpack(ckpt: Checkpoint, dtype=torch.bfloat16, *, out=None, stream=None):
    """The values [T, H] that a checkpoint stands for, in `dtype` (float16: at most its
    largest finite value)."""
    return _at(stream, (_fast or load_binding()).ckpt_unpack, ckpt.codes, ckpt.scales,
               _FORMATS[ckpt.fmt], _dtype_number(dtype, "dtype"), out)


def ckpt_linear_dw_workspace_bytes(tokens: int, n: int, k: int, aligned: bool = True) -> int:
    """aligned: d_out's address and row stride (at least n) are multiples of 16 bytes."""
    return int(load().mhc_ckpt_linear_dw_workspace_bytes(tokens, n, k, int(aligned)))


def mhc_ckpt_linear_dw(d_out, x: Checkpoint, *, d_w=None, dtype=torch.float32,
                       accumulate: bool = False, workspace=None, stream=None):
    """d_w [N, K] = d_out^T x, the weight gradient of out = x W^T, from d_out
    [T, N] (bfloat16 or float16, rows may be strided) and the checkpoint of
    x [T, K]. accumulate adds to the d_w given. A d_out that requires grad is
    refused while gradients are recorded."""
    if d_w is not None:
        dtype = d_w.dtype
    elif accumulate:
        raise ValueError("accumulate needs the d_w to add to")
    return _at(stream, (_fast or load_binding()).ckpt_linear_dw, d_out, x.codes, x.scales,
               _FORMATS[x.fmt], d_w, _dtype_number(dtype, "d_w"), accumulate, workspace)
