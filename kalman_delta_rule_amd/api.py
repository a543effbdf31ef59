"""Python binding of the KDN C ABI (``include/kdn.h``) over torch tensors.

Same entry-point names as the C library.  This layer only checks tensor
metadata, allocates outputs / workspace with torch (device memory) and passes
raw pointers plus torch's current HIP stream; every step of the method runs
in the library's kernels.  Layouts: activations [B,T,H,D], state [B,H,dk,dv],
variances [B,H,dk] (Diagonal) or [B,H] (Isotropic).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import (KDN_BF16, KDN_CLEAR_TAIL, KDN_DIAG, KDN_F32, KDN_ISO, KDN_MATH_BF16,  # noqa: F401
                   KDN_OUT_F32, KdnError)


def _io_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDN_BF16
    if t.dtype == torch.float32:
        return KDN_F32
    raise TypeError("q, k, v must be bfloat16 or float32, got %s" % t.dtype)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, shape, dtype, device) -> None:
    # the usual case in one go: single-token calls are bound by these checks
    if (type(t) is torch.Tensor and t.dtype == dtype and t.shape == shape
            and t.is_contiguous() and t.device == device):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _math_flag(math: Optional[str]) -> int:
    """Contraction precision of the bf16 forward: None (the library's
    default: split-operand products for Diagonal, single bf16 products for
    Isotropic) or "bf16" (single bf16 products)."""
    if math is None:
        return 0
    if math == "bf16":
        return KDN_MATH_BF16
    raise ValueError("math must be None or 'bf16', got %r" % (math,))


# torch's own accessor of a device's current stream handle: current_stream()
# builds a Stream object around it, 1.9 us of a 10 us single-token call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _launch(dev, fn, *args) -> None:
    """fn(*args, stream) on dev, whichever device is current."""
    if _current_device() == dev.index:
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st != 0:
        _lib.check(st)


def _head_vec(t, name, H, dev):
    if t is not None:
        _need(t, name, (H,), torch.float32, dev)
    return t


def _fwd(variant: int, q, k, v, alpha, omega, r, S0, var0, mu, o, S_T, var_T,
         ext: bool = False, mu_h=None, c0_h=None, beta_eff=None, sequence_parallel=True,
         math=None, o_dtype=None, prepare=False):
    """Checks the tensors, allocates what is missing, and launches the
    forward (or, with ``prepare``, returns (outputs, launch) where launch()
    repeats the call on the same tensors and stream without re-checking)."""
    L = _lib.lib()
    if q.dim() != 4:
        raise ValueError("q must be [B,T,H,dk]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    io = _io_code(q)
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(alpha, "alpha", (B, T, H, dk), torch.float32, dev)
    wshape = (B, T, H, dk) if variant == KDN_DIAG else (B, T, H)
    _need(omega, "omega", wshape, torch.float32, dev)
    _need(r, "r", (B, T, H), torch.float32, dev)
    vshape = (B, H, dk) if variant == KDN_DIAG else (B, H)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if var0 is not None:
        _need(var0, "p0" if variant == KDN_DIAG else "b0", vshape, torch.float32, dev)
    o_dtype = q.dtype if o_dtype is None else o_dtype
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=o_dtype, device=dev)
    _need(o, "o", (B, T, H, dv), o_dtype, dev)
    if S_T is None:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    _need(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    if var_T is None:
        var_T = torch.empty(vshape, dtype=torch.float32, device=dev)
    _need(var_T, "var_T", vshape, torch.float32, dev)
    mu = float(dk if mu is None else mu)
    io |= _math_flag(math)
    if o_dtype != q.dtype:
        if not (q.dtype == torch.bfloat16 and o_dtype == torch.float32):
            raise TypeError("o may differ from q's dtype only as fp32 with bf16 inputs")
        io |= KDN_OUT_F32
    # with the workspace, shapes with few heads and long sequences run sequence-parallel
    ws_bytes = L.kdn_fwd_workspace_size(variant, B, T, H, dk, dv, io) if sequence_parallel else 0
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    if ext:
        _head_vec(mu_h, "mu_h", H, dev)
        _head_vec(c0_h, "c0_h", H, dev)
        if beta_eff is not None:
            _need(beta_eff, "beta_eff", (B, T, H), torch.float32, dev)
        fn = L.kdn_fwd_ex
        args = (variant, B, T, H, dk, dv, io, mu, _ptr(mu_h), _ptr(q), _ptr(k), _ptr(v),
                _ptr(alpha), _ptr(omega), _ptr(r), _ptr(S0), _ptr(var0), _ptr(c0_h), _ptr(o),
                _ptr(S_T), _ptr(var_T), _ptr(beta_eff), _ptr(ws), ws_bytes)
    else:
        fn = L.kdn_diag_fwd if variant == KDN_DIAG else L.kdn_iso_fwd
        args = (B, T, H, dk, dv, io, mu, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(omega),
                _ptr(r), _ptr(S0), _ptr(var0), _ptr(o), _ptr(S_T), _ptr(var_T), _ptr(ws),
                ws_bytes)
    stream = _stream(dev)
    keep = (q, k, v, alpha, omega, r, S0, var0, o, S_T, var_T, mu_h, c0_h, beta_eff, ws)

    def launch():
        _lib.check(fn(*args, stream))
        return keep  # the tensors stay alive as long as the launcher does

    if prepare:
        return (o, S_T, var_T), launch
    with torch.cuda.device(dev):
        launch()
    return o, S_T, var_T


def kdn_diag_fwd(q, k, v, alpha, omega, r, S0=None, p0=None, mu=None, o=None, S_T=None,
                 p_T=None, math=None, o_dtype=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Diagonal KDN forward.  Returns (o [B,T,H,dv], S_T [B,H,dk,dv], p_T [B,H,dk]).
    With bf16 q/k/v the contractions run split-operand products (near fp32)
    unless math="bf16" asks for single bf16 products; o_dtype=torch.float32
    then writes o in fp32."""
    return _fwd(KDN_DIAG, q, k, v, alpha, omega, r, S0, p0, mu, o, S_T, p_T, math=math,
                o_dtype=o_dtype)


def fwd_launcher(variant: str, q, k, v, alpha, omega, r, S0=None, var0=None, mu=None,
                 o=None, S_T=None, var_T=None, math=None, o_dtype=None):
    """Check the arguments once and return ((o, S_T, var_T), launch): each
    launch() runs the same forward (kdn_diag_fwd / kdn_iso_fwd) on the same
    tensors and on the stream that was current here, without re-checking or
    allocating (a workspace the shape needs is allocated once, now)."""
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    return _fwd(var, q, k, v, alpha, omega, r, S0, var0, mu, o, S_T, var_T, math=math,
                o_dtype=o_dtype, prepare=True)


def kdn_iso_fwd(q, k, v, alpha, omega, r, S0=None, b0=None, mu=None, o=None, S_T=None,
                b_T=None, math=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Isotropic KDN forward.  Returns (o [B,T,H,dv], S_T [B,H,dk,dv], b_T [B,H])."""
    return _fwd(KDN_ISO, q, k, v, alpha, omega, r, S0, b0, mu, o, S_T, b_T, math=math)


def kdn_fwd_ex(variant: str, q, k, v, alpha, omega, r, S0=None, var0=None, mu=None,
               mu_h=None, c0_h=None, want_beta_eff: bool = False, o=None, S_T=None,
               var_T=None, sequence_parallel: bool = True, math=None, o_dtype=None):
    """Forward with per-head mu_h [H] and c0_h [H] (both optional) and the
    effective write strength.  Returns (o, S_T, var_T, beta_eff [B,T,H] or
    None).  sequence_parallel=False withholds the workspace, so that shapes the
    library would split over the sequence run the serial walk instead."""
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    beta = None
    if want_beta_eff:
        B, T, H, _ = q.shape
        beta = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    o, S_T, var_T = _fwd(var, q, k, v, alpha, omega, r, S0, var0, mu, o, S_T, var_T,
                         ext=True, mu_h=mu_h, c0_h=c0_h, beta_eff=beta,
                         sequence_parallel=sequence_parallel, math=math, o_dtype=o_dtype)
    return o, S_T, var_T, beta


def kdn_dense_fwd(q, k, v, alpha, omega, r, S0=None, P0=None, want_beta_eff: bool = False,
                  o=None, S_T=None, P_T=None):
    """Exact dense-covariance Kalman memory with diag(alpha) / diag(omega)
    gates, for small d_k.  Returns (o [B,T,H,dv], S_T [B,H,dk,dv],
    P_T [B,H,dk,dk], beta_eff [B,T,H] or None)."""
    L = _lib.lib()
    if q.dim() != 4:
        raise ValueError("q must be [B,T,H,dk]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    io = _io_code(q)
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(alpha, "alpha", (B, T, H, dk), torch.float32, dev)
    _need(omega, "omega", (B, T, H, dk), torch.float32, dev)
    _need(r, "r", (B, T, H), torch.float32, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if P0 is not None:
        _need(P0, "P0", (B, H, dk, dk), torch.float32, dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    _need(o, "o", (B, T, H, dv), q.dtype, dev)
    if S_T is None:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if P_T is None:
        P_T = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev)
    _need(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    _need(P_T, "P_T", (B, H, dk, dk), torch.float32, dev)
    beta = torch.empty((B, T, H), dtype=torch.float32, device=dev) if want_beta_eff else None
    with torch.cuda.device(dev):
        st = L.kdn_dense_fwd(B, T, H, dk, dv, io, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                             _ptr(omega), _ptr(r), _ptr(S0), _ptr(P0), _ptr(o), _ptr(S_T),
                             _ptr(P_T), _ptr(beta), _stream(dev))
    _lib.check(st)
    return o, S_T, P_T, beta


def kdn_fwd_preact(variant: str, q, k, v, a_pre, w_pre, r_pre, r_min: float = 0.01, S0=None,
                   var0=None, mu=None, mu_h=None, c0_h=None, want_beta_eff: bool = False,
                   o=None, S_T=None, var_T=None, workspace=None, math=None):
    """Forward from the gates' pre-activations (alpha = sigmoid(a_pre),
    omega = softplus(w_pre), r = r_min + softplus(r_pre)); pre-activations in
    the io dtype of q.  Returns (o, S_T, var_T, beta_eff or None)."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    if q.dim() != 4:
        raise ValueError("q must be [B,T,H,dk]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    io = _io_code(q)
    iso = var == KDN_ISO
    f32 = torch.float32
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(a_pre, "a_pre", (B, T, H, dk), q.dtype, dev)
    _need(w_pre, "w_pre", (B, T, H) if iso else (B, T, H, dk), q.dtype, dev)
    _need(r_pre, "r_pre", (B, T, H), q.dtype, dev)
    var_shape = (B, H) if iso else (B, H, dk)
    for t, n, shp in ((S0, "S0", (B, H, dk, dv)), (var0, "var0", var_shape),
                      (mu_h, "mu_h", (H,)), (c0_h, "c0_h", (H,))):
        if t is not None:
            _need(t, n, shp, f32, dev)
    mu = float(dk if mu is None else mu)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    if S_T is None:
        S_T = torch.empty((B, H, dk, dv), dtype=f32, device=dev)
    if var_T is None:
        var_T = torch.empty(var_shape, dtype=f32, device=dev)
    beta = torch.empty((B, T, H), dtype=f32, device=dev) if want_beta_eff else None
    need = int(L.kdn_fwd_preact_workspace_size(var, B, T, H, dk))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = L.kdn_fwd_preact(var, B, T, H, dk, dv, io | _math_flag(math), mu, _ptr(mu_h),
                              _ptr(q), _ptr(k), _ptr(v),
                              _ptr(a_pre), _ptr(w_pre), _ptr(r_pre), float(r_min), _ptr(S0),
                              _ptr(var0), _ptr(c0_h), _ptr(o), _ptr(S_T), _ptr(var_T),
                              _ptr(beta), _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(st)
    return o, S_T, var_T, beta


def kdn_gates_from_preact(variant: str, a_pre, w_pre, r_pre, r_min: float = 0.01):
    """The gates (alpha, omega, r), fp32, from their pre-activations, with the
    arithmetic the forward from pre-activations uses (kdn_fwd_ex on these
    gates equals kdn_fwd_preact bit for bit)."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    if a_pre.dim() != 4:
        raise ValueError("a_pre must be [B,T,H,dk]")
    B, T, H, dk = a_pre.shape
    dev = a_pre.device
    io = _io_code(a_pre)
    iso = var == KDN_ISO
    _need(w_pre, "w_pre", (B, T, H) if iso else (B, T, H, dk), a_pre.dtype, dev)
    _need(r_pre, "r_pre", (B, T, H), a_pre.dtype, dev)
    f32 = torch.float32
    alpha = torch.empty((B, T, H, dk), dtype=f32, device=dev)
    omega = torch.empty(tuple(w_pre.shape), dtype=f32, device=dev)
    r = torch.empty((B, T, H), dtype=f32, device=dev)
    with torch.cuda.device(dev):
        st = L.kdn_gates_from_preact(var, B, T, H, dk, io, _ptr(a_pre), _ptr(w_pre), _ptr(r_pre),
                                     float(r_min), _ptr(alpha), _ptr(omega), _ptr(r), _stream(dev))
    _lib.check(st)
    return alpha, omega, r


def kdn_bwd(variant: str, q, k, v, alpha, omega, r, d_o, S0=None, var0=None, mu=None,
            mu_h=None, c0_h=None, dS_T=None, dvar_T=None, want_state_grads: bool = True,
            workspace=None) -> dict:
    """Backward pass of the forward given by the same arguments (see kdn_fwd_ex)
    for dL/do = d_o, dL/dS_T = dS_T and dL/dvar_T = dvar_T (both optional).
    Returns a dict with dq, dk, dv (io dtype), dalpha, domega, dr (fp32) and,
    with ``want_state_grads``, dS0, dvar0 and dmu [B,H] (fp32).  A given
    ``workspace`` (uint8) is passed as it is: the library requires its base
    size and splits the sequence (bf16 io, few heads) only when it holds all
    of kdn_bwd_workspace_size; without one, that size is allocated."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    if q.dim() != 4:
        raise ValueError("q must be [B,T,H,dk]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    io = _io_code(q)
    iso = var == KDN_ISO
    var_shape = (B, H) if iso else (B, H, dk)
    f32 = torch.float32
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(d_o, "d_o", (B, T, H, dv), q.dtype, dev)
    _need(alpha, "alpha", (B, T, H, dk), f32, dev)
    _need(omega, "omega", (B, T, H) if iso else (B, T, H, dk), f32, dev)
    _need(r, "r", (B, T, H), f32, dev)
    for t, n, shp in ((S0, "S0", (B, H, dk, dv)), (dS_T, "dS_T", (B, H, dk, dv)),
                      (var0, "var0", var_shape), (dvar_T, "dvar_T", var_shape),
                      (mu_h, "mu_h", (H,)), (c0_h, "c0_h", (H,))):
        if t is not None:
            _need(t, n, shp, f32, dev)
    mu = float(dk if mu is None else mu)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dalpha": torch.empty_like(alpha), "domega": torch.empty_like(omega),
         "dr": torch.empty_like(r)}
    if want_state_grads:
        g["dS0"] = torch.empty((B, H, dk, dv), dtype=f32, device=dev)
        g["dvar0"] = torch.empty(var_shape, dtype=f32, device=dev)
        g["dmu"] = torch.empty((B, H), dtype=f32, device=dev)
    if workspace is None:
        need = int(L.kdn_bwd_workspace_size(var, B, T, H, dk, dv))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = L.kdn_bwd(var, B, T, H, dk, dv, io, mu, _ptr(mu_h), _ptr(q), _ptr(k), _ptr(v),
                       _ptr(alpha), _ptr(omega), _ptr(r), _ptr(S0), _ptr(var0), _ptr(c0_h),
                       _ptr(d_o), _ptr(dS_T), _ptr(dvar_T), _ptr(g["dq"]), _ptr(g["dk"]),
                       _ptr(g["dv"]), _ptr(g["dalpha"]), _ptr(g["domega"]), _ptr(g["dr"]),
                       _ptr(g.get("dS0")), _ptr(g.get("dvar0")), _ptr(g.get("dmu")),
                       _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(st)
    return g


def kdn_bwd_preact(variant: str, q, k, v, a_pre, w_pre, r_pre, d_o, r_min: float = 0.01,
                   S0=None, var0=None, mu=None, mu_h=None, c0_h=None, dS_T=None, dvar_T=None,
                   workspace=None) -> dict:
    """Backward of kdn_fwd_preact: dq, dk, dv (io dtype), da_pre, dw_pre,
    dr_pre (fp32), dS0, dvar0, dmu."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    io = _io_code(q)
    iso = var == KDN_ISO
    f32 = torch.float32
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(d_o, "d_o", (B, T, H, dv), q.dtype, dev)
    _need(a_pre, "a_pre", (B, T, H, dk), q.dtype, dev)
    _need(w_pre, "w_pre", (B, T, H) if iso else (B, T, H, dk), q.dtype, dev)
    _need(r_pre, "r_pre", (B, T, H), q.dtype, dev)
    var_shape = (B, H) if iso else (B, H, dk)
    for t, n, shp in ((S0, "S0", (B, H, dk, dv)), (dS_T, "dS_T", (B, H, dk, dv)),
                      (var0, "var0", var_shape), (dvar_T, "dvar_T", var_shape),
                      (mu_h, "mu_h", (H,)), (c0_h, "c0_h", (H,))):
        if t is not None:
            _need(t, n, shp, f32, dev)
    mu = float(dk if mu is None else mu)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "da_pre": torch.empty(a_pre.shape, dtype=f32, device=dev),
         "dw_pre": torch.empty(w_pre.shape, dtype=f32, device=dev),
         "dr_pre": torch.empty(r_pre.shape, dtype=f32, device=dev),
         "dS0": torch.empty((B, H, dk, dv), dtype=f32, device=dev),
         "dvar0": torch.empty(var_shape, dtype=f32, device=dev),
         "dmu": torch.empty((B, H), dtype=f32, device=dev)}
    need = int(L.kdn_bwd_preact_workspace_size(var, B, T, H, dk, dv))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = L.kdn_bwd_preact(var, B, T, H, dk, dv, io, mu, _ptr(mu_h), _ptr(q), _ptr(k), _ptr(v),
                              _ptr(a_pre), _ptr(w_pre), _ptr(r_pre), float(r_min), _ptr(S0),
                              _ptr(var0), _ptr(c0_h), _ptr(d_o), _ptr(dS_T), _ptr(dvar_T),
                              *[_ptr(g[n]) for n in ("dq", "dk", "dv", "da_pre", "dw_pre",
                                                     "dr_pre", "dS0", "dvar0", "dmu")],
                              _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check(st)
    return g


def kdn_step(variant: str, q, k, v, alpha, omega, r, S, var_state, mu=None,
             o=None, mu_h=None, beta_eff=None) -> torch.Tensor:
    """One decode step; S [B,H,dk,dv] and var_state are updated in place.
    ``variant`` is "diag" or "iso".  Returns o [B,H,dv]."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    io = _io_code(q)
    _need(q, "q", (B, H, dk), q.dtype, dev)
    _need(k, "k", (B, H, dk), q.dtype, dev)
    _need(v, "v", (B, H, dv), q.dtype, dev)
    _need(alpha, "alpha", (B, H, dk), torch.float32, dev)
    _need(omega, "omega", (B, H, dk) if var == KDN_DIAG else (B, H), torch.float32, dev)
    _need(r, "r", (B, H), torch.float32, dev)
    _need(S, "S", (B, H, dk, dv), torch.float32, dev)
    _need(var_state, "var_state", (B, H, dk) if var == KDN_DIAG else (B, H), torch.float32, dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    _need(o, "o", (B, H, dv), q.dtype, dev)
    mu = float(dk if mu is None else mu)
    if mu_h is not None or beta_eff is not None:
        # extended step: per-head information scale and / or the effective
        # write strength [B,H]
        _head_vec(mu_h, "mu_h", H, dev)
        if beta_eff is not None:
            _need(beta_eff, "beta_eff", (B, H), torch.float32, dev)
        with torch.cuda.device(dev):
            st = L.kdn_step_ex(var, B, H, dk, dv, io, mu, _ptr(mu_h), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(alpha), _ptr(omega), _ptr(r), _ptr(S), _ptr(var_state),
                               _ptr(o), _ptr(beta_eff), _stream(dev))
        _lib.check(st)
        return o
    with torch.cuda.device(dev):
        st = L.kdn_step(var, B, H, dk, dv, io, mu, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                        _ptr(omega), _ptr(r), _ptr(S), _ptr(var_state), _ptr(o), _stream(dev))
    _lib.check(st)
    return o


def kdn_gain_scan(variant: str, k, alpha, omega, r, var0=None, mu=None,
                  want_kappa: bool = True):
    """Gain scan alone.  Returns (kappa [B,T,H,dk] fp32 or None, var_T)."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    B, T, H, dk = k.shape
    dev = k.device
    io = _io_code(k)
    _need(alpha, "alpha", (B, T, H, dk), torch.float32, dev)
    _need(omega, "omega", (B, T, H, dk) if var == KDN_DIAG else (B, T, H), torch.float32, dev)
    _need(r, "r", (B, T, H), torch.float32, dev)
    vshape = (B, H, dk) if var == KDN_DIAG else (B, H)
    if var0 is not None:
        _need(var0, "var0", vshape, torch.float32, dev)
    if not k.is_contiguous():
        raise ValueError("k must be contiguous")
    kappa = torch.empty((B, T, H, dk), dtype=torch.float32, device=dev) if want_kappa else None
    var_T = torch.empty(vshape, dtype=torch.float32, device=dev)
    mu = float(dk if mu is None else mu)
    ws_bytes = L.kdn_gain_workspace_size(var, B, T, H, dk)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = L.kdn_gain_scan(var, B, T, H, dk, io, mu, _ptr(k), _ptr(alpha), _ptr(omega),
                             _ptr(r), _ptr(var0), _ptr(kappa), _ptr(var_T), _ptr(ws),
                             ws.numel(), _stream(dev))
    _lib.check(st)
    return kappa, var_T


def kdn_gain_scan_static(variant: str, k, alpha, omega, r, var0=None, mu=None, kappa=None,
                         var_T=None):
    """Gain scan through the allocation-free entry point: its scratch is the
    library's static device array, so the call itself allocates nothing (give
    kappa and var_T to allocate nothing here either; kappa may be None to skip
    the gain).  Returns (kappa, var_T)."""
    L = _lib.lib()
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    B, T, H, dk = k.shape
    dev = k.device
    io = _io_code(k)
    _need(k, "k", (B, T, H, dk), k.dtype, dev)
    _need(alpha, "alpha", (B, T, H, dk), torch.float32, dev)
    _need(omega, "omega", (B, T, H, dk) if var == KDN_DIAG else (B, T, H), torch.float32, dev)
    _need(r, "r", (B, T, H), torch.float32, dev)
    vshape = (B, H, dk) if var == KDN_DIAG else (B, H)
    if var0 is not None:
        _need(var0, "var0", vshape, torch.float32, dev)
    if kappa is not None:
        _need(kappa, "kappa", (B, T, H, dk), torch.float32, dev)
    if var_T is None:
        var_T = torch.empty(vshape, dtype=torch.float32, device=dev)
    _need(var_T, "var_T", vshape, torch.float32, dev)
    mu = float(dk if mu is None else mu)
    with torch.cuda.device(dev):
        st = L.kdn_gain_scan_static(var, B, T, H, dk, io, mu, _ptr(k), _ptr(alpha), _ptr(omega),
                                    _ptr(r), _ptr(var0), _ptr(kappa), _ptr(var_T), _stream(dev))
    _lib.check(st)
    return kappa, var_T


def kdn_fwd_workspace_size(variant: str, B, T, H, dk, dv, io_dtype: torch.dtype) -> int:
    var = {"diag": KDN_DIAG, "iso": KDN_ISO}[variant]
    io = KDN_BF16 if io_dtype == torch.bfloat16 else KDN_F32
    return int(_lib.lib().kdn_fwd_workspace_size(var, B, T, H, dk, dv, io))


def kdn_version() -> str:
    return _lib.lib().kdn_version().decode()


# ---- the operators around the mixer ---------------------------------------

_ACT = {None: 0, "silu": 1}
_GATE = {"alpha": 0, "preact": 1}


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of t's last axis: t may be a slice of wider
    rows, but its channels lie side by side and its rows an equal way apart."""
    D = t.shape[-1]
    if t.is_contiguous():
        return D
    if D > 1 and t.stride(-1) != 1:
        raise ValueError("%s must have its channels side by side (stride 1)" % name)
    step = D
    rows = 0  # rows collapsed so far, from the innermost axis outwards
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if rows == 0:
            step, rows = stride, size
        elif stride == step * rows:
            rows *= size
        else:
            raise ValueError("%s must have its rows evenly spaced" % name)
    if step < D:
        raise ValueError("%s has rows that overlap" % name)
    return step


def _need_rows(t, name, shape, dtype, device) -> int:
    """_need for a tensor that may be a slice of wider rows; the row stride."""
    if (type(t) is torch.Tensor and t.dtype == dtype and t.shape == shape
            and t.is_contiguous() and t.device == device):
        return shape[-1]
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return _row_stride(t, name)


def _first(t, name, dims):
    """Device and io code of a call's first tensor, [.., D] with ``dims`` axes
    (None: any number)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != dims if dims is not None else t.dim() < 1:
        raise ValueError("%s must have %s, got shape %s" % (
            name, "at least one axis" if dims is None else "%d axes" % dims, tuple(t.shape)))
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    if t.dtype == torch.bfloat16:
        return t.device, KDN_BF16
    if t.dtype == torch.float32:
        return t.device, KDN_F32
    raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def _optional(dev, *tensors):
    for t, name, shape, dtype in tensors:
        if t is not None:
            _need(t, name, shape, dtype, dev)


def _given(t, name, like):
    """The caller's output tensor, or a new one, as ``like`` but dense."""
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _need(t, name, like.shape, like.dtype, like.device)
    return t


def _sequences(cu_seqlens, B, dev) -> int:
    """Number of sequences: the rows, or the packed ones of a single row."""
    if cu_seqlens is None:
        return B
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a tensor [N+1] of offsets, N >= 1")
    _need(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, dev)
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) need one row, got %d" % B)
    return cu_seqlens.numel() - 1


def _tail(cu_seqlens, *given) -> int:
    """KDN_CLEAR_TAIL where rows of packed sequences get no output of the
    caller's: nothing that this layer allocates is left unwritten.  A caller's
    output keeps what it holds behind the last sequence."""
    return KDN_CLEAR_TAIL if cu_seqlens is not None and all(t is None for t in given) else 0


def _beside(shape, dtype, dev, cu_seqlens, tail):
    """A new output of a call whose tail is cleared, or (beside one of the
    caller's) cleared here."""
    new = torch.zeros if cu_seqlens is not None and not tail else torch.empty
    return new(shape, dtype=dtype, device=dev)


def _workspace(workspace, need: int, dev):
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be contiguous uint8")
        if workspace.device != dev:
            raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
        return workspace, workspace.numel()
    return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need else (None, 0)


def kdn_layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, y=None,
                       want_stats: bool = False):
    """Layer norm over the last axis of x [..., D] (a slice of wider rows is
    fine).  Returns (y, mean, rstd): y in x's dtype, and with ``want_stats``
    the fp32 statistics [...] that kdn_layer_norm_bwd reads (None, None
    otherwise).  weight, bias: [D] fp32, each optional."""
    L = _lib.lib()
    dev, io = _first(x, "x", None)
    D = x.shape[-1]
    stride = _row_stride(x, "x")
    f32 = torch.float32
    _optional(dev, (weight, "weight", (D,), f32), (bias, "bias", (D,), f32))
    y = _given(y, "y", x)
    mean = rstd = None
    if want_stats:
        mean = torch.empty(x.shape[:-1], dtype=f32, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=f32, device=dev)
    _launch(dev, L.kdn_layer_norm_fwd, x.numel() // D if D else 0, D, io, float(eps),
            x.data_ptr(), stride, _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def kdn_layer_norm_bwd(dy, x, mean, rstd, weight=None, want_param_grads: bool = True, dx=None,
                       workspace=None) -> dict:
    """Backward of kdn_layer_norm_fwd with its mean and rstd.  Returns a dict
    with dx (x's dtype) and, with ``want_param_grads``, dweight and dbias [D]
    (fp32, summed over every row)."""
    L = _lib.lib()
    dev, io = _first(x, "x", None)
    D = x.shape[-1]
    stride = _row_stride(x, "x")
    f32 = torch.float32
    _need(dy, "dy", x.shape, x.dtype, dev)
    _need(mean, "mean", x.shape[:-1], f32, dev)
    _need(rstd, "rstd", x.shape[:-1], f32, dev)
    _optional(dev, (weight, "weight", (D,), f32))
    rows = x.numel() // D if D else 0
    g = {"dx": _given(dx, "dx", x)}
    ws, ws_bytes = None, 0
    if want_param_grads:
        g["dweight"] = torch.empty(D, dtype=f32, device=dev)
        g["dbias"] = torch.empty(D, dtype=f32, device=dev)
        ws, ws_bytes = _workspace(workspace, L.kdn_layer_norm_bwd_workspace_size(rows, D), dev)
    _launch(dev, L.kdn_layer_norm_bwd, rows, D, io, dy.data_ptr(), x.data_ptr(), stride,
            mean.data_ptr(), rstd.data_ptr(), _ptr(weight), g["dx"].data_ptr(),
            _ptr(g.get("dweight")), _ptr(g.get("dbias")), _ptr(ws), ws_bytes)
    return g


def _activation(activation) -> int:
    if activation not in _ACT:
        raise ValueError("activation must be None or 'silu', got %r" % (activation,))
    return _ACT[activation]


def _taps(weight, D) -> int:
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [W, D]")
    return weight.shape[0]


def kdn_conv_fwd(x, weight, bias=None, state0=None, cu_seqlens=None, activation=None,
                 want_state: bool = False, y=None, state_T=None):
    """Short causal convolution per channel over x [B,T,D] (a slice of wider
    rows is fine) with weight [W,D] (its last row multiplies the current
    token; W from 2 to 4) and bias [D], fp32; ``activation`` None or "silu".
    state0 [N,W-1,D] (x's dtype) holds the inputs before each sequence, zeros
    without; cu_seqlens (int32 [N+1]) packs N sequences into one row.  Returns
    (y, state_T): state_T [N,W-1,D], the last inputs of each sequence, if
    given or with ``want_state`` (None otherwise).  Behind the last sequence a
    new y holds zeros, and a caller's keeps what it held."""
    L = _lib.lib()
    dev, io = _first(x, "x", 3)
    B, T, D = x.shape
    stride = _row_stride(x, "x")
    W = _taps(weight, D)
    N = _sequences(cu_seqlens, B, dev)
    f32 = torch.float32
    _need(weight, "weight", (W, D), f32, dev)
    _optional(dev, (bias, "bias", (D,), f32), (state0, "state0", (N, W - 1, D), x.dtype))
    act = _activation(activation)
    tail = _tail(cu_seqlens, y)
    y = _given(y, "y", x)
    if state_T is not None:
        _need(state_T, "state_T", (N, W - 1, D), x.dtype, dev)
    elif want_state:
        state_T = torch.empty((N, max(W - 1, 0), D), dtype=x.dtype, device=dev)
    _launch(dev, L.kdn_conv_fwd, B, T, D, W, io | tail, act, x.data_ptr(), stride, weight.data_ptr(),
            _ptr(bias), _ptr(state0), _ptr(cu_seqlens), N, y.data_ptr(), _ptr(state_T))
    return y, state_T


def kdn_conv_bwd(dy, x, weight, bias=None, state0=None, cu_seqlens=None, activation=None,
                 dstate_T=None, dx=None, workspace=None) -> dict:
    """Backward of kdn_conv_fwd given by the same arguments, for dL/dy = dy and
    dL/dstate_T = dstate_T (optional).  Returns a dict with dx (x's dtype),
    dweight [W,D] (fp32), dbias [D] (fp32) where bias is given and dstate0
    (x's dtype) where state0 is given.  Behind the last sequence a new dx holds
    zeros, and a caller's keeps what it held."""
    L = _lib.lib()
    dev, io = _first(x, "x", 3)
    B, T, D = x.shape
    stride = _row_stride(x, "x")
    W = _taps(weight, D)
    N = _sequences(cu_seqlens, B, dev)
    f32 = torch.float32
    _need(dy, "dy", x.shape, x.dtype, dev)
    _need(weight, "weight", (W, D), f32, dev)
    _optional(dev, (bias, "bias", (D,), f32), (state0, "state0", (N, W - 1, D), x.dtype),
              (dstate_T, "dstate_T", (N, W - 1, D), x.dtype))
    act = _activation(activation)
    tail = _tail(cu_seqlens, dx)
    g = {"dx": _given(dx, "dx", x), "dweight": torch.empty((W, D), dtype=f32, device=dev)}
    if bias is not None:
        g["dbias"] = torch.empty(D, dtype=f32, device=dev)
    if state0 is not None:
        g["dstate0"] = torch.empty_like(state0)
    ws, ws_bytes = _workspace(workspace, L.kdn_conv_bwd_workspace_size(B, T, D, W), dev)
    _launch(dev, L.kdn_conv_bwd, B, T, D, W, io | tail, act, dy.data_ptr(), x.data_ptr(), stride,
            weight.data_ptr(), _ptr(bias), _ptr(state0), _ptr(cu_seqlens), N, _ptr(dstate_T),
            g["dx"].data_ptr(), g["dweight"].data_ptr(), _ptr(g.get("dbias")),
            _ptr(g.get("dstate0")), _ptr(ws), ws_bytes)
    return g


def kdn_conv_step(x, weight, state, bias=None, activation=None, y=None) -> torch.Tensor:
    """One token of kdn_conv_fwd: x [B,D]; state [B,W-1,D] (x's dtype) is moved
    on in place.  Returns y [B,D]."""
    L = _lib.lib()
    dev, io = _first(x, "x", 2)
    B, D = x.shape
    stride = _row_stride(x, "x")
    W = _taps(weight, D)
    _need(weight, "weight", (W, D), torch.float32, dev)
    _need(state, "state", (B, W - 1, D), x.dtype, dev)
    if bias is not None:
        _need(bias, "bias", (D,), torch.float32, dev)
    y = _given(y, "y", x)
    _launch(dev, L.kdn_conv_step, B, D, W, io, _activation(activation), x.data_ptr(), stride,
            weight.data_ptr(), _ptr(bias), state.data_ptr(), y.data_ptr())
    return y


def _gate(gate, io_dtype):
    """The gate's code and the dtype of its tensor."""
    if gate not in _GATE:
        raise ValueError("gate must be 'alpha' or 'preact', got %r" % (gate,))
    return _GATE[gate], io_dtype if gate == "preact" else torch.float32


def kdn_rec_fwd(x, a, h0=None, cu_seqlens=None, gate: str = "preact", blend: bool = False,
                want_checkpoints: bool = False, h=None, h_T=None, workspace=None):
    """Gated recurrence per channel, h_t = alpha_t h_{t-1} + x_t (with
    ``blend``: (1 - alpha_t) x_t), over x [B,T,D].  ``a`` [B,T,D] holds
    pre-activations in x's dtype, alpha = sigmoid(a) (gate="preact"), or alpha
    itself in fp32 (gate="alpha"); x and a may be slices of wider rows.  h0
    [N,D] fp32 is the state before each sequence (zeros without); cu_seqlens
    (int32 [N+1]) packs N sequences into one row.  Returns (h, h_T,
    checkpoints): h in x's dtype, h_T [N,D] fp32 and, with
    ``want_checkpoints``, the states that kdn_rec_bwd starts from (None
    otherwise).  Behind the last sequence a new h holds zeros, and a caller's
    keeps what it held."""
    L = _lib.lib()
    dev, io = _first(x, "x", 3)
    B, T, D = x.shape
    stride = _row_stride(x, "x")
    code, adt = _gate(gate, x.dtype)
    a_stride = _need_rows(a, "a", x.shape, adt, dev)
    N = _sequences(cu_seqlens, B, dev)
    f32 = torch.float32
    _optional(dev, (h0, "h0", (N, D), f32))
    tail = _tail(cu_seqlens, h)
    h = _given(h, "h", x)
    if h_T is not None:
        _need(h_T, "h_T", (N, D), f32, dev)
    else:
        h_T = torch.empty((N, D), dtype=f32, device=dev)
    chk = None
    if want_checkpoints:
        chk = _beside((B, -(-T // _lib.KDN_REC_CHECKPOINT), D), f32, dev, cu_seqlens, tail)
    ws, ws_bytes = _workspace(workspace, L.kdn_rec_fwd_workspace_size(B, T, D), dev)
    _launch(dev, L.kdn_rec_fwd, B, T, D, io | tail, code, int(bool(blend)), x.data_ptr(), stride,
            a.data_ptr(), a_stride, _ptr(h0), _ptr(cu_seqlens), N, h.data_ptr(), h_T.data_ptr(),
            _ptr(chk), _ptr(ws), ws_bytes)
    return h, h_T, chk


def kdn_rec_bwd(dh, x, a, checkpoints, h0=None, dh_T=None, cu_seqlens=None, gate: str = "preact",
                blend: bool = False, dx=None, workspace=None, da=None) -> dict:
    """Backward of kdn_rec_fwd given by the same arguments and its checkpoints,
    for dL/dh = dh and dL/dh_T = dh_T (optional).  Returns a dict with dx (x's
    dtype), da (a's dtype: the gradient by alpha or by its pre-activation)
    and dh0 [N,D] fp32.  Behind the last sequence new dx and da hold zeros, and
    the caller's keep what they held."""
    L = _lib.lib()
    dev, io = _first(x, "x", 3)
    B, T, D = x.shape
    stride = _row_stride(x, "x")
    code, adt = _gate(gate, x.dtype)
    a_stride = _need_rows(a, "a", x.shape, adt, dev)
    N = _sequences(cu_seqlens, B, dev)
    f32 = torch.float32
    _need(dh, "dh", x.shape, x.dtype, dev)
    _need(checkpoints, "checkpoints", (B, -(-T // _lib.KDN_REC_CHECKPOINT), D), f32, dev)
    _optional(dev, (h0, "h0", (N, D), f32), (dh_T, "dh_T", (N, D), f32),
              (dx, "dx", x.shape, x.dtype), (da, "da", x.shape, adt))
    tail = _tail(cu_seqlens, dx, da)
    new = lambda t, dtype: _beside(x.shape, dtype, dev, cu_seqlens, tail) if t is None else t
    g = {"dx": new(dx, x.dtype), "da": new(da, adt),
         "dh0": torch.empty((N, D), dtype=f32, device=dev)}
    ws, ws_bytes = _workspace(workspace, L.kdn_rec_bwd_workspace_size(B, T, D), dev)
    _launch(dev, L.kdn_rec_bwd, B, T, D, io | tail, code, int(bool(blend)), dh.data_ptr(), x.data_ptr(),
            stride, a.data_ptr(), a_stride, checkpoints.data_ptr(), _ptr(h0), _ptr(cu_seqlens), N,
            _ptr(dh_T), g["dx"].data_ptr(), g["da"].data_ptr(), g["dh0"].data_ptr(), _ptr(ws),
            ws_bytes)
    return g


def kdn_rec_step(x, a, state, gate: str = "preact", blend: bool = False, h=None) -> torch.Tensor:
    """One token of kdn_rec_fwd: x, a [B,D]; state [B,D] fp32 is updated in
    place.  Returns h [B,D]."""
    L = _lib.lib()
    dev, io = _first(x, "x", 2)
    B, D = x.shape
    stride = _row_stride(x, "x")
    code, adt = _gate(gate, x.dtype)
    a_stride = _need_rows(a, "a", x.shape, adt, dev)
    _need(state, "state", (B, D), torch.float32, dev)
    h = _given(h, "h", x)
    _launch(dev, L.kdn_rec_step, B, D, io, code, int(bool(blend)), x.data_ptr(), stride,
            a.data_ptr(), a_stride, state.data_ptr(), h.data_ptr())
    return h
