"""Layers on heads beside attention: norm and rotation of q and k, and caches held in 8 bits.

Tensor front ends of ``sc_qk_norm_rotary``, ``sc_cache_write``, ``sc_cache_read`` and
``sc_cached_attn`` (``include/specconv.h`` states formulas, limits and errors), in the manner of
:mod:`fft_causal_long_amd.layers`.  A serving step is :func:`qk_norm_rotary` on the new tokens'
projections, :func:`cache_write` of their k and v, :func:`cached_attention` of their q.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import SC_ERR_UNSUPPORTED, SpecConvError, _lib
from .layers import _check, _int3, _out, _ptr, _run, _scratch, _typed

__all__ = [
    "qk_norm_rotary", "qk_norm_rotary_bwd", "KVCache", "cache_write", "cache_read",
    "cached_attention", "sc_qk", "sc_cache", "sc_cached", "sc_qk_norm_rotary",
    "sc_qk_norm_rotary_bwd", "sc_qk_norm_rotary_workspace_bytes", "sc_cache_write",
    "sc_cache_read", "sc_cached_attn", "sc_cached_attn_workspace_bytes", "CODE_I8", "CODE_E4M3",
    "CACHE_BLOCK",
]

CODE_I8, CODE_E4M3 = 0, 1
CACHE_BLOCK = 64


class sc_qk(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "L", "H", "Hkv", "D", "R")]
                + [(n, _int3) for n in ("q", "k", "q_out", "k_out", "dq", "dk")]
                + [("eps", ctypes.c_float), ("interleaved", ctypes.c_int32)]
                + [(n, ctypes.c_void_p) for n in ("inv_freq", "positions", "kv_len")])


class sc_cache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "N", "P", "Hkv", "D")] + [("code", ctypes.c_int32)]
                + [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "table")])


class sc_cached(ctypes.Structure):
    _fields_ = [("Lq", ctypes.c_int64), ("H", ctypes.c_int64), ("q", _int3), ("o", _int3),
                ("scale", ctypes.c_float), ("cap", ctypes.c_float), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64), ("slopes", ctypes.c_void_p), ("kv_len", ctypes.c_void_p)]


def _declare():
    vp, i64, sz, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    pq, pc, pa = (ctypes.POINTER(s) for s in (sc_qk, sc_cache, sc_cached))
    for name, args, res in (
            ("sc_qk_norm_rotary", [st, pq] + [vp] * 7, st),
            ("sc_qk_norm_rotary_workspace_bytes", [st, pq], sz),
            ("sc_qk_norm_rotary_bwd", [st, pq] + [vp] * 11 + [sz, vp], st),
            ("sc_cache_write", [st, pc, vp, _int3, vp, _int3, i64, vp, vp], st),
            ("sc_cache_read", [st, pc, vp, _int3, vp, _int3, i64, vp, vp], st),
            ("sc_cached_attn_workspace_bytes", [st, pc, pa], sz),
            ("sc_cached_attn", [st, pc, pa] + [vp] * 4 + [sz, vp], st)):
        f = getattr(_lib, name)
        f.argtypes, f.restype = args, res


_declare()


# ---------------------------------------------------------------- raw C-ABI mirrors

def sc_qk_norm_rotary(kind, a, q, k, wq, wk, q_out, k_out, stream):
    return _lib.sc_qk_norm_rotary(kind, ctypes.byref(a), q, k, wq, wk, q_out, k_out, stream)


def sc_qk_norm_rotary_workspace_bytes(kind, a) -> int:
    return int(_lib.sc_qk_norm_rotary_workspace_bytes(kind, ctypes.byref(a)))


def sc_qk_norm_rotary_bwd(kind, a, dq_out, dk_out, q, k, wq, wk, dq, dk, dwq, dwk, ws, ws_bytes, stream):
    return _lib.sc_qk_norm_rotary_bwd(kind, ctypes.byref(a), dq_out, dk_out, q, k, wq, wk, dq, dk, dwq,
                                      dwk, ws, ws_bytes, stream)


def sc_cache_write(kind, c, k, k_strides, v, v_strides, L, kv_len, stream):
    return _lib.sc_cache_write(kind, ctypes.byref(c), k, _int3(*k_strides), v, _int3(*v_strides), L, kv_len,
                               stream)


def sc_cache_read(kind, c, k, k_strides, v, v_strides, L, kv_len, stream):
    return _lib.sc_cache_read(kind, ctypes.byref(c), k, _int3(*k_strides), v, _int3(*v_strides), L, kv_len,
                              stream)


def sc_cached_attn_workspace_bytes(kind, c, a) -> int:
    return int(_lib.sc_cached_attn_workspace_bytes(kind, ctypes.byref(c), ctypes.byref(a)))


def sc_cached_attn(kind, c, a, q, o, lse, ws, ws_bytes, stream):
    return _lib.sc_cached_attn(kind, ctypes.byref(c), ctypes.byref(a), q, o, lse, ws, ws_bytes, stream)


# ---------------------------------------------------------------- norm and rotation

# A decoding step is a handful of microseconds, most of them spent in these functions: they look at each
# tensor once and fill a struct in one go.

_NONE = (0, 0, 0)


def _bld(t):
    """The {batch, token, head} strides of a (B, L, H, D) tensor (an axis of one place: whatever it says)."""
    s = t.stride()
    if len(s) != 4:
        raise ValueError("tensors must be (B, L, H, D)")
    if s[3] != 1 and t.shape[3] > 1:
        raise ValueError("the D values of a head must be contiguous")
    return s[:3]


def _lengths(kv_len, B, dev):
    if kv_len.dtype != torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
        raise ValueError("kv_len must be a contiguous int32 (B,) tensor")
    if kv_len.device != dev:
        raise ValueError("tensors must be on the same GPU")
    return kv_len.data_ptr()


def _qk_args(q, k, qo, ko, dq, dk, q_weight, k_weight, inv_freq, positions, kv_len, interleaved, eps):
    """The call's struct; qo, ko: the results, or their gradients."""
    sq = _bld(q)
    B, L, H, D = q.shape
    Hkv, sk, sko, sdk = 0, _NONE, _NONE, _NONE
    if k is not None:
        sk, sko = _bld(k), _bld(ko)
        Hkv = k.shape[2]
        if k.shape != (B, L, Hkv, D):
            raise ValueError("k must be (B, L, Hkv, D) for q (B, L, H, D)")
        if dk is not None:
            sdk = _bld(dk)
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (D,) or not w.is_contiguous()):
            raise ValueError("q_weight and k_weight must be contiguous (D,) tensors")
    R, f, pos, n = 0, None, None, None
    if inv_freq is not None:
        _typed(q, torch.float32, inv_freq)
        if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > D:
            raise ValueError("inv_freq must hold at most D / 2 values")
        R = 2 * inv_freq.shape[0]
        f = inv_freq.data_ptr() if R else None
    if positions is not None:
        _typed(q, torch.int32, positions)
        if kv_len is not None:
            raise ValueError("positions and kv_len exclude each other")
        if positions.shape != (B, L):
            raise ValueError("positions must be (B, L)")
        pos = positions.data_ptr()
    if kv_len is not None:
        n = _lengths(kv_len, B, q.device)
    return sc_qk(B, L, H, Hkv, D, R, sq, sk, _bld(qo), sko, _NONE if dq is None else _bld(dq), sdk, eps,
                 bool(interleaved), f, pos, n)


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                   k_weight: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, *,
                   positions: torch.Tensor | None = None, kv_len: torch.Tensor | None = None,
                   interleaved: bool = False, eps: float = 1e-6, q_out: torch.Tensor | None = None,
                   k_out: torch.Tensor | None = None):
    """(q_out, k_out): the rows of q (B, L, H, D) and k (B, L, Hkv, D, or None) normed by their root
    mean square, times the (D,) weights, their first 2 len(inv_freq) values turned by position times
    inv_freq (float32, radians a position; None: no rotation) as halves or ``interleaved`` pairs
    (sc_qk_norm_rotary).  Positions: ``positions`` (B, L) int32, or the last L of each sequence of
    ``kv_len`` (B,) int32, or 0 .. L - 1.  q_out may be q itself, k_out k."""
    kind = _check(q, k, q_weight, k_weight, q_out, k_out)
    q_out = _out(q_out, q, "q_out")
    if k is not None:
        k_out = _out(k_out, k, "k_out")
    a = _qk_args(q, k, q_out, k_out, None, None, q_weight, k_weight, inv_freq, positions, kv_len, interleaved, eps)
    _run("qk_norm_rotary", _lib.sc_qk_norm_rotary, q.device, kind, ctypes.byref(a), q.data_ptr(), _ptr(k),
         _ptr(q_weight), _ptr(k_weight), q_out.data_ptr(), _ptr(k_out))
    return q_out, k_out


def qk_norm_rotary_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor | None, q: torch.Tensor,
                       k: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, *,
                       positions: torch.Tensor | None = None, kv_len: torch.Tensor | None = None,
                       interleaved: bool = False, eps: float = 1e-6, dq: torch.Tensor | None = None,
                       dk: torch.Tensor | None = None, params: bool = True,
                       workspace: torch.Tensor | None = None):
    """(dq, dk, dq_weight, dk_weight) of :func:`qk_norm_rotary` with the same options for the gradients
    of its results, from its inputs (sc_qk_norm_rotary_bwd); ``params`` false: no weight gradients
    (None)."""
    kind = _check(q, dq_out, dk_out, k, q_weight, k_weight, dq, dk)
    if dq_out.shape != q.shape or (k is None) != (dk_out is None) or (k is not None and dk_out.shape != k.shape):
        raise ValueError("dq_out and dk_out must have the shapes of q and k")
    dq = _out(dq, q, "dq")
    if k is not None:
        dk = _out(dk, k, "dk")
    a = _qk_args(q, k, dq_out, dk_out, dq, dk, q_weight, k_weight, inv_freq, positions, kv_len, interleaved, eps)
    dwq = dwk = None
    if params:
        dwq = torch.empty(a.D, dtype=q.dtype, device=q.device)
        dwk = torch.empty_like(dwq) if k is not None else None
    pa = ctypes.byref(a)
    keep, ws, n = _scratch(_lib.sc_qk_norm_rotary_workspace_bytes(kind, pa) if params else 0, workspace, q.device)
    _run("qk_norm_rotary_bwd", _lib.sc_qk_norm_rotary_bwd, q.device, kind, pa, dq_out.data_ptr(), _ptr(dk_out),
         q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), dq.data_ptr(), _ptr(dk), _ptr(dwq), _ptr(dwk), ws, n)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- the cache

_CODES = {"int8": CODE_I8, "e4m3": CODE_E4M3}


def _fixed(name):
    return property(lambda self: getattr(self, name))


def _memory(name):
    """The cache's memory `name`, whose address the calls take from the struct."""
    held = "_" + name

    def put(self, t):
        now = getattr(self, held)
        if t.dtype != now.dtype or t.shape != now.shape or t.device != now.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s %s tensor on the cache's device" % (name, tuple(now.shape), now.dtype))
        setattr(self, held, t)
        setattr(self._struct, name, t.data_ptr())
    return property(lambda self: getattr(self, held), put)


class KVCache:
    """k and v of B sequences of up to ``length`` tokens in 8-bit codes, one scale for each 64 tokens
    of a head: ``code`` "int8" or "e4m3".  ``blocks``: blocks in the pool (default: enough for every
    sequence); ``table`` (B, N) int32, N = ceil(length / 64): each sequence's blocks in the pool
    (default: row b's are b N .. b N + N - 1).  The table's values may change between calls.  Other
    tensors may take the place of ``table``, ``k``, ``v``, ``k_scale`` and ``v_scale`` through these
    attributes (a block is a row of the last four); the sizes and the code stay.  ``copy.copy`` is a cache
    over the same memory with attributes of its own, ``copy.deepcopy`` has memory of its own."""

    B, N, blocks, Hkv, D, code, device = map(_fixed, ("_B", "_N", "_blocks", "_Hkv", "_D", "_code", "_device"))
    k, v, k_scale, v_scale = map(_memory, ("k", "v", "k_scale", "v_scale"))

    def __init__(self, B: int, length: int, Hkv: int, D: int, code: str = "int8", *, device="cuda",
                 blocks: int | None = None, table: torch.Tensor | None = None):
        if code not in _CODES:
            raise ValueError("code must be 'int8' or 'e4m3'")
        N = -(-length // CACHE_BLOCK)
        P = B * N if blocks is None else blocks
        if min(B, length, Hkv, D, P) < 0 or D % 16 or D > 128:
            raise ValueError("sizes must not be negative, D a multiple of 16 up to 128")
        if table is None and P < B * N:
            raise ValueError("a pool smaller than B N blocks needs a table")
        self._B, self._N, self._blocks, self._Hkv, self._D, self._code = B, N, P, Hkv, D, code
        dev = torch.device(device)
        self._k = torch.empty(P, Hkv, CACHE_BLOCK * D, dtype=torch.uint8, device=dev)
        self._v = torch.empty_like(self._k)
        self._k_scale = torch.zeros(P, Hkv, dtype=torch.float32, device=dev)
        self._v_scale = torch.zeros_like(self._k_scale)
        self._device = self._k.device
        self._table = None
        self._bind()
        self.table = table

    def _bind(self):
        """The struct that the calls take, of what the attributes hold."""
        self._struct = sc_cache(self._B, self._N, self._blocks, self._Hkv, self._D, _CODES[self._code],
                                *(t.data_ptr() for t in (self._k, self._v, self._k_scale, self._v_scale)), _ptr(self._table))
        self._ref = ctypes.byref(self._struct)

    # a copy, or what was pickled, has a struct of its own
    def __getstate__(self):
        return {n: x for n, x in self.__dict__.items() if n not in ("_struct", "_ref")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._device = self._k.device
        self._bind()

    @property
    def table(self):
        return self._table

    @table.setter
    def table(self, table):
        if table is None:
            if self._blocks < self._B * self._N:
                raise ValueError("a pool smaller than B N blocks needs a table")
        else:
            if table.dtype != torch.int32 or not table.is_contiguous() or table.device != self._device \
                    or tuple(table.shape) != (self._B, self._N):
                raise ValueError("table must be a contiguous int32 (B, N) tensor on the cache's device")
        self._table = table
        self._struct.table = _ptr(table)


def _cache_kv(cache, k, v, kv_len):
    """The checked call's strides of k and v and pointer of kv_len."""
    if k.device != cache._device:
        raise ValueError("tensors must be on the cache's GPU")
    sk, sv = _bld(k), _bld(v)
    if k.shape != v.shape or k.shape != (cache._B, k.shape[1], cache._Hkv, cache._D):
        raise ValueError("k and v must be (B, L, Hkv, D) of the cache's sizes")
    return _int3(*sk), _int3(*sv), _lengths(kv_len, cache._B, cache._device)


def cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, kv_len: torch.Tensor) -> None:
    """Stores k, v (B, L, Hkv, D) as the last L tokens of each sequence of kv_len (B,) int32
    (sc_cache_write); what a sequence held from there on is given up."""
    kind = _check(k, v)
    sk, sv, n = _cache_kv(cache, k, v, kv_len)
    _run("cache_write", _lib.sc_cache_write, k.device, kind, cache._ref, k.data_ptr(), sk, v.data_ptr(), sv,
         k.shape[1], n)


def cache_read(cache: KVCache, L: int, kv_len: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
               k: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """(k, v) (B, L, Hkv, D): the values of the last L tokens of each sequence of kv_len (B,) int32, 0
    before its first (sc_cache_read); ``k`` and ``v`` are written if given."""
    shape = (cache._B, L, cache._Hkv, cache._D)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache._device)
    if v is None:
        v = torch.empty_like(k) if k.is_contiguous() else torch.empty(shape, dtype=dtype, device=cache._device)
    kind = _check(k, v)
    sk, sv, n = _cache_kv(cache, k, v, kv_len)
    if k.shape[1] != L or k.dtype != dtype:
        raise ValueError("k and v must be (B, L, Hkv, D) of the asked dtype")
    _run("cache_read", _lib.sc_cache_read, k.device, kind, cache._ref, k.data_ptr(), sk, v.data_ptr(), sv, L, n)
    return k, v


def cached_attention(q: torch.Tensor, cache: KVCache, kv_len: torch.Tensor, *, window: int = 0,
                     sinks: int = 0, scale: float | None = None, cap: float = 0.0,
                     slopes: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: bool = False, workspace: torch.Tensor | None = None):
    """Causal attention of q (B, Lq, H, D), the last Lq positions of each sequence of kv_len (B,)
    int32, over ``cache`` (sc_cached_attn), options as :func:`causal_attention`; with a ``window`` the
    first ``sinks`` tokens stay visible.  ``lse``: returns (o, lse), lse (B, H, Lq) float32."""
    kind = _check(q, out)
    if q.device != cache._device:
        raise ValueError("tensors must be on the cache's GPU")
    sq = _bld(q)
    B, Lq, H, D = q.shape
    if B != cache._B or D != cache._D:
        raise ValueError("q must be (B, Lq, H, D) of the cache's B and D")
    if slopes is not None:
        _typed(q, torch.float32, slopes)
        if slopes.shape != (H,):
            raise ValueError("slopes must be (H,)")
    o = _out(out, q, "out")
    a = sc_cached(Lq, H, sq, _bld(o), (1.0 / math.sqrt(D) if D else 1.0) if scale is None else scale, cap, window, sinks,
                  _ptr(slopes), _lengths(kv_len, B, q.device))
    if lse and D == 0 and B * H * Lq:   # the call has no result to write then, and no lse
        raise SpecConvError(SC_ERR_UNSUPPORTED, "cached_attention: lse of heads of no values")
    L = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device) if lse else None
    pa = ctypes.byref(a)
    keep, ws, n = _scratch(_lib.sc_cached_attn_workspace_bytes(kind, cache._ref, pa), workspace, q.device)
    _run("cached_attention", _lib.sc_cached_attn, q.device, kind, cache._ref, pa, q.data_ptr(), o.data_ptr(), _ptr(L),
         ws, n)
    return (o, L) if lse else o
