"""Layers beside the convolution: layer norm, gated recurrence and causal attention.

Tensor front ends of ``sc_layernorm``, ``sc_recur``, ``sc_causal_attn`` and their ``_bwd``
calls (``include/specconv.h`` states formulas, limits and errors): float32 or bfloat16 device
tensors on torch's current stream, token-major, every sum and state in float32.  Scratch comes
from torch's allocator unless the caller gives ``workspace`` (a contiguous device tensor of at
least the ``*_workspace_bytes``).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (KIND_BF16, KIND_F32, SC_ERR_UNSUPPORTED, SC_OK, SpecConvError, _lib, _ws_args)

__all__ = [
    "layer_norm", "layer_norm_bwd", "gated_recurrence", "gated_recurrence_bwd",
    "causal_attention", "causal_attention_bwd", "sc_attn", "sc_layernorm", "sc_layernorm_bwd",
    "sc_layernorm_bwd_workspace_bytes", "sc_recur", "sc_recur_bwd", "sc_recur_workspace_bytes",
    "sc_causal_attn", "sc_causal_attn_bwd", "sc_attn_workspace_bytes",
]


class sc_attn(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "Lq", "Lk", "H", "Hkv", "D")]
                + [(n, ctypes.c_int64 * 3) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")]
                + [("scale", ctypes.c_float), ("cap", ctypes.c_float), ("window", ctypes.c_int64),
                   ("slopes", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                   ("doc_start", ctypes.c_void_p)])


def _declare():
    vp, i64, sz, st, f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int,
                            ctypes.c_float)
    pa = ctypes.POINTER(sc_attn)
    for name, args, res in (
            ("sc_layernorm", [st] + [vp] * 6 + [i64] * 4 + [f32, vp], st),
            ("sc_layernorm_bwd_workspace_bytes", [st, i64, i64], sz),
            ("sc_layernorm_bwd", [st] + [vp] * 8 + [i64] * 5 + [vp, sz, vp], st),
            ("sc_recur_workspace_bytes", [st, i64, i64, i64], sz),
            ("sc_recur", [st] + [vp] * 5 + [i64] * 6 + [vp, sz, vp], st),
            ("sc_recur_bwd", [st] + [vp] * 9 + [i64] * 9 + [vp, sz, vp], st),
            ("sc_attn_workspace_bytes", [st, pa, ctypes.c_int], sz),
            ("sc_causal_attn", [st, pa] + [vp] * 6 + [sz, vp], st),
            ("sc_causal_attn_bwd", [st, pa] + [vp] * 10 + [sz, vp], st)):
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, res


_declare()


# ---------------------------------------------------------------- raw C-ABI mirrors

def sc_layernorm(kind, x, w, b, y, mean, rstd, rows, C, x_stride, y_stride, eps, stream):
    return _lib.sc_layernorm(kind, x, w, b, y, mean, rstd, rows, C, x_stride, y_stride, eps, stream)


def sc_layernorm_bwd_workspace_bytes(kind, rows, C) -> int:
    return int(_lib.sc_layernorm_bwd_workspace_bytes(kind, rows, C))


def sc_layernorm_bwd(kind, dy, x, w, mean, rstd, dx, dw, db, rows, C, dy_stride, x_stride,
                     dx_stride, ws, ws_bytes, stream):
    return _lib.sc_layernorm_bwd(kind, dy, x, w, mean, rstd, dx, dw, db, rows, C, dy_stride,
                                 x_stride, dx_stride, ws, ws_bytes, stream)


def sc_recur_workspace_bytes(kind, B, L, C) -> int:
    return int(_lib.sc_recur_workspace_bytes(kind, B, L, C))


def sc_recur(kind, z, u, h0, h, hT, B, L, C, z_stride, u_stride, h_stride, ws, ws_bytes, stream):
    return _lib.sc_recur(kind, z, u, h0, h, hT, B, L, C, z_stride, u_stride, h_stride, ws, ws_bytes,
                         stream)


def sc_recur_bwd(kind, dh, z, u, h, h0, dhT, dz, du, dh0, B, L, C, dh_stride, z_stride, u_stride,
                 h_stride, dz_stride, du_stride, ws, ws_bytes, stream):
    return _lib.sc_recur_bwd(kind, dh, z, u, h, h0, dhT, dz, du, dh0, B, L, C, dh_stride, z_stride,
                             u_stride, h_stride, dz_stride, du_stride, ws, ws_bytes, stream)


def sc_attn_workspace_bytes(kind, a, backward) -> int:
    return int(_lib.sc_attn_workspace_bytes(kind, ctypes.byref(a), int(backward)))


def sc_causal_attn(kind, a, q, k, v, o, lse, ws, ws_bytes, stream):
    return _lib.sc_causal_attn(kind, ctypes.byref(a), q, k, v, o, lse, ws, ws_bytes, stream)


def sc_causal_attn_bwd(kind, a, dout, q, k, v, o, lse, dq, dk, dv, ws, ws_bytes, stream):
    return _lib.sc_causal_attn_bwd(kind, ctypes.byref(a), dout, q, k, v, o, lse, dq, dk, dv, ws,
                                   ws_bytes, stream)


# ---------------------------------------------------------------- tensor front end

_KIND = {torch.float32: KIND_F32, torch.bfloat16: KIND_BF16}
# The current stream's handle without building a Stream object: a decoding step is a handful of
# microseconds, most of them spent here.  A torch without these entry points (one built without GPU
# support has none) takes the public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _check(x, *others):
    """One storage type and one GPU; others may hold None."""
    dt, dev = x.dtype, x.device
    if dt not in _KIND:
        raise TypeError("unsupported dtype %s" % dt)
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    for t in others:
        if t is None:
            continue
        if t.dtype != dt:
            raise ValueError("tensors must share a dtype")
        if t.device != dev:
            raise ValueError("tensors must be on the same GPU")
    return _KIND[dt]


def _typed(x, dt, *ts):
    """Contiguous tensors of type dt (or None) on x's GPU."""
    for t in ts:
        if t is not None:
            if t.dtype != dt or not t.is_contiguous():
                raise ValueError("expected a contiguous %s tensor" % dt)
            if t.device != x.device:
                raise ValueError("tensors must be on the same GPU")


def _row_stride(t):
    """Elements between the rows of (..., C), whose rows have to lie evenly spaced."""
    C = t.shape[-1]
    if t.is_contiguous():
        return max(C, 1)
    if C > 1 and t.stride(-1) != 1:
        raise ValueError("rows must be contiguous")
    step, span = None, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = span = s
        elif s != span:
            raise ValueError("rows must be evenly spaced")
        span *= n
    return max(C, 1) if step is None else step


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scratch(need, workspace, dev):
    if workspace is not None:
        ptr, n = _ws_args(workspace, dev)
        return workspace, ptr, n
    if not need:
        return None, None, 0
    t = torch.empty(need, dtype=torch.uint8, device=dev)
    return t, t.data_ptr(), need


def _out(out, like, name):
    if out is None:
        if like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
        raise ValueError("%s must match the inputs in shape, dtype and device" % name)
    return out


def _run(what, fn, dev, *args):
    """fn(*args, stream) on dev's current stream."""
    if dev.index == _get_device():
        st = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev.index))
    if st != SC_OK:
        raise SpecConvError(st, what)


def _params(x, *ps):
    for p in ps:
        if p is not None and (p.dim() != 1 or p.shape[0] != x.shape[-1] or not p.is_contiguous()):
            raise ValueError("weight and bias must be contiguous (C,) tensors")


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5,
               out: torch.Tensor | None = None, *, stats: bool = False):
    """y = (x - mean) rstd weight + bias over the last axis (sc_layernorm); x (..., C) with evenly
    spaced contiguous rows.  ``stats``: returns (y, mean, rstd), the statistics float32 of x's
    leading shape, as :func:`layer_norm_bwd` takes them (NaN for rows of no values)."""
    kind = _check(x, weight, bias)
    if x.dim() < 1:
        raise ValueError("x must be (..., C)")
    _params(x, weight, bias)
    y = _out(out, x, "out")
    C = x.shape[-1]
    rows = x.numel() // C if C else 0
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        if C == 0:   # the mean of no values, 0 / 0; the call itself has nothing to do then
            mean.fill_(math.nan)
            rstd.fill_(math.nan)
    _run("layer_norm", _lib.sc_layernorm, x.device, kind, x.data_ptr(), _ptr(weight), _ptr(bias),
         y.data_ptr(), _ptr(mean), _ptr(rstd), rows, C, _row_stride(x), _row_stride(y), eps)
    return (y, mean, rstd) if stats else y


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, dx: torch.Tensor | None = None, *,
                   params: bool = True, workspace: torch.Tensor | None = None):
    """(dx, dweight, dbias) of :func:`layer_norm` for the output gradient dy (sc_layernorm_bwd);
    ``params`` false: (dx, None, None)."""
    kind = _check(x, dy, weight, dx)
    _typed(x, torch.float32, mean, rstd)
    if dy.shape != x.shape or x.dim() < 1:
        raise ValueError("dy must have x's shape (..., C)")
    if mean.shape != x.shape[:-1] or rstd.shape != x.shape[:-1]:
        raise ValueError("mean and rstd must have x's leading shape")
    _params(x, weight)
    dx = _out(dx, x, "dx")
    C = x.shape[-1]
    rows = x.numel() // C if C else 0
    dw = db = None
    if params:
        dw = torch.empty(C, dtype=x.dtype, device=x.device)
        db = torch.empty_like(dw)
    keep, ws, n = _scratch(_lib.sc_layernorm_bwd_workspace_bytes(kind, rows, C) if params else 0,
                           workspace, x.device)
    _run("layer_norm_bwd", _lib.sc_layernorm_bwd, x.device, kind, dy.data_ptr(), x.data_ptr(),
         _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), rows, C,
         _row_stride(dy), _row_stride(x), _row_stride(dx), ws, n)
    return dx, dw, db


def _blc(z):
    if z.dim() < 2:
        raise ValueError("tensors must be (..., L, C)")
    B = 1
    for s in z.shape[:-2]:
        B *= s
    return B, z.shape[-2], z.shape[-1]


def _state(s, z, name):
    if s is not None and s.shape != z.shape[:-2] + z.shape[-1:]:
        raise ValueError("%s must be float32 (..., C)" % name)


def gated_recurrence(z: torch.Tensor, u: torch.Tensor, h0: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, hT: torch.Tensor | None = None, *,
                     workspace: torch.Tensor | None = None):
    """(h, hT) of h_t = f_t h_{t-1} + (1 - f_t) u_t, f = sigmoid(z), along the tokens of (..., L, C)
    tensors (sc_recur).  h0, hT: float32 (..., C) states before the first and after the last
    token; hT may be h0 (a decoding loop's state, L = 1)."""
    kind = _check(z, u, out)
    _typed(z, torch.float32, h0, hT)
    B, L, C = _blc(z)
    if u.shape != z.shape:
        raise ValueError("z and u must have one shape")
    _state(h0, z, "h0")
    _state(hT, z, "hT")
    h = _out(out, z, "out")
    if hT is None and h0 is not None:
        hT = torch.empty_like(h0)
    elif hT is None:
        hT = torch.empty(z.shape[:-2] + z.shape[-1:], dtype=torch.float32, device=z.device)
    keep, ws, n = _scratch(_lib.sc_recur_workspace_bytes(kind, B, L, C), workspace, z.device)
    _run("gated_recurrence", _lib.sc_recur, z.device, kind, z.data_ptr(), u.data_ptr(), _ptr(h0),
         h.data_ptr(), hT.data_ptr(), B, L, C, _row_stride(z), _row_stride(u), _row_stride(h), ws, n)
    return h, hT


def gated_recurrence_bwd(dh: torch.Tensor, z: torch.Tensor, u: torch.Tensor, h: torch.Tensor,
                         h0: torch.Tensor | None = None, dhT: torch.Tensor | None = None,
                         dz: torch.Tensor | None = None, du: torch.Tensor | None = None, *,
                         workspace: torch.Tensor | None = None):
    """(dz, du, dh0) of :func:`gated_recurrence` for the gradients dh of h and dhT of hT (None:
    zero), with h and h0 of the forward call (sc_recur_bwd)."""
    kind = _check(z, dh, u, h, dz, du)
    _typed(z, torch.float32, h0, dhT)
    B, L, C = _blc(z)
    if not dh.shape == u.shape == h.shape == z.shape:
        raise ValueError("dh, z, u and h must have one shape")
    _state(h0, z, "h0")
    _state(dhT, z, "dhT")
    dz = _out(dz, z, "dz")
    du = _out(du, z, "du")
    dh0 = torch.empty(z.shape[:-2] + z.shape[-1:], dtype=torch.float32, device=z.device)
    keep, ws, n = _scratch(_lib.sc_recur_workspace_bytes(kind, B, L, C), workspace, z.device)
    _run("gated_recurrence_bwd", _lib.sc_recur_bwd, z.device, kind, dh.data_ptr(), z.data_ptr(),
         u.data_ptr(), h.data_ptr(), _ptr(h0), _ptr(dhT), dz.data_ptr(), du.data_ptr(),
         dh0.data_ptr(), B, L, C, *(_row_stride(t) for t in (dh, z, u, h, dz, du)), ws, n)
    return dz, du, dh0


_int3 = ctypes.c_int64 * 3


def _strides(t):
    if t.dim() != 4:
        raise ValueError("attention tensors must be (B, L, H, D)")
    B, L, H, D = t.shape
    b, l, h, d = t.stride()
    if D > 1 and d != 1:
        raise ValueError("the D values of a head must be contiguous")
    return _int3(b if B > 1 else 0, l if L > 1 else 0, h if H > 1 else 0)


def _attn(q, k, v, window, scale, cap, slopes, doc_start, kv_len):
    sq, sk, sv = _strides(q), _strides(k), _strides(v)
    B, Lq, H, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if k.shape != (B, Lk, Hkv, D) or v.shape != k.shape:
        raise ValueError("k and v must be (B, Lk, Hkv, D) for q (B, Lq, H, D)")
    for t, shape, name in ((slopes, (H,), "slopes"), (kv_len, (B,), "kv_len"),
                           (doc_start, (B, Lk), "doc_start")):
        if t is not None and tuple(t.shape) != shape:
            raise ValueError("%s must be %s" % (name, shape))
    a = sc_attn(B, Lq, Lk, H, Hkv, D)
    a.q, a.k, a.v = sq, sk, sv
    a.scale = (1.0 / math.sqrt(D) if D else 1.0) if scale is None else float(scale)
    a.cap, a.window = float(cap), int(window)
    a.slopes, a.kv_len, a.doc_start = _ptr(slopes), _ptr(kv_len), _ptr(doc_start)
    return a


def causal_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, window: int = 0,
                     scale: float | None = None, cap: float = 0.0,
                     slopes: torch.Tensor | None = None, doc_start: torch.Tensor | None = None,
                     kv_len: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: bool = False, workspace: torch.Tensor | None = None):
    """Causal attention of q (B, Lq, H, D) over k, v (B, Lk, Hkv, D) (sc_causal_attn): the last Lq
    positions of each sequence of kv_len[b] (default Lk) keys attend to the ``window`` (0: all)
    keys up to their own, within their document (doc_start (B, Lk) int32).  ``scale`` defaults to
    D^-1/2; ``cap`` > 0 caps scores by a tanh; ``slopes`` (H) float32 subtract slope * distance.
    ``lse``: returns (o, lse), lse (B, H, Lq) float32; heads of no values (D = 0) have none
    (SC_ERR_UNSUPPORTED)."""
    kind = _check(q, k, v, out)
    _typed(q, torch.float32, slopes)
    _typed(q, torch.int32, doc_start, kv_len)
    a = _attn(q, k, v, window, scale, cap, slopes, doc_start, kv_len)
    o = _out(out, q, "out")
    a.o = _strides(o)
    if lse and a.D == 0 and a.B * a.H * a.Lq:   # the call has no result to write then, and no lse
        raise SpecConvError(SC_ERR_UNSUPPORTED, "causal_attention: lse of heads of no values")
    L = torch.empty((a.B, a.H, a.Lq), dtype=torch.float32, device=q.device) if lse else None
    pa = ctypes.byref(a)
    keep, ws, n = _scratch(_lib.sc_attn_workspace_bytes(kind, pa, 0), workspace, q.device)
    _run("causal_attention", _lib.sc_causal_attn, q.device, kind, pa, q.data_ptr(), k.data_ptr(),
         v.data_ptr(), o.data_ptr(), _ptr(L), ws, n)
    return (o, L) if lse else o


def causal_attention_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         o: torch.Tensor, lse: torch.Tensor, *, window: int = 0,
                         scale: float | None = None, cap: float = 0.0,
                         slopes: torch.Tensor | None = None,
                         doc_start: torch.Tensor | None = None,
                         kv_len: torch.Tensor | None = None, dq: torch.Tensor | None = None,
                         dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """(dq, dk, dv) of :func:`causal_attention` with the same options for the output gradient
    dout, from its o and lse (sc_causal_attn_bwd); dk, dv are summed over the heads that share a
    key head."""
    kind = _check(q, dout, k, v, o, dq, dk, dv)
    _typed(q, torch.float32, lse, slopes)
    _typed(q, torch.int32, doc_start, kv_len)
    a = _attn(q, k, v, window, scale, cap, slopes, doc_start, kv_len)
    if dout.shape != q.shape or o.shape != q.shape or tuple(lse.shape) != (a.B, a.H, a.Lq):
        raise ValueError("dout and o must have q's shape, lse be (B, H, Lq)")
    dq, dk, dv = _out(dq, q, "dq"), _out(dk, k, "dk"), _out(dv, v, "dv")
    a.o, a.dout, a.dq, a.dk, a.dv = (_strides(t) for t in (o, dout, dq, dk, dv))
    pa = ctypes.byref(a)
    keep, ws, n = _scratch(_lib.sc_attn_workspace_bytes(kind, pa, 1), workspace, q.device)
    _run("causal_attention_bwd", _lib.sc_causal_attn_bwd, q.device, kind, pa, dout.data_ptr(),
         q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(),
         dk.data_ptr(), dv.data_ptr(), ws, n)
    return dq, dk, dv
