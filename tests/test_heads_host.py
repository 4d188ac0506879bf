"""The calls on heads without a GPU: what they refuse on the host before any HIP call, and the float64
references the GPU tests compare with (gradients against differences, the cache model by hand)."""
import ctypes

import numpy as np
import pytest

from oracle import heads as ref
from oracle import layers as lref
from tests.test_layers_host import P, TOL, sc, slope  # noqa: F401  (sc: a fixture)

I3 = ctypes.c_int64 * 3


def qk(sc, **k):
    a = sc.sc_qk(2, 4, 2, 1, 64, 64)
    for n in ("q", "q_out", "dq"):
        getattr(a, n)[:] = [512, 128, 64]
    for n in ("k", "k_out", "dk"):
        getattr(a, n)[:] = [256, 64, 64]
    a.eps, a.inv_freq = 1e-6, P[10]
    for n, x in k.items():
        if n.startswith("s_"):
            getattr(a, n[2:])[:] = x
        else:
            setattr(a, n, x)
    return a


def test_qk_refusals(sc):
    h = sc.lib()
    OK, INV, UNS, WS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED, sc.SC_ERR_WORKSPACE

    def f(kind=0, q=P[0], k=P[1], wq=P[2], wk=P[3], qo=P[4], ko=P[5], **opt):
        return h.sc_qk_norm_rotary(kind, ctypes.byref(qk(sc, **opt)), q, k, wq, wk, qo, ko, None)

    assert f(B=0) == OK and f(L=0) == OK and f(D=0, R=0) == OK and f(H=0, Hkv=0) == OK
    assert h.sc_qk_norm_rotary(0, None, P[0], P[1], None, None, P[4], P[5], None) == INV
    assert f(kind=2) == INV and f(interleaved=2) == INV
    for n in ("B", "L", "H", "Hkv", "D", "R"):
        assert f(**{n: -1}) == INV, n
    assert f(R=63) == INV and f(R=66) == INV and f(inv_freq=None) == INV
    for e in (-1.0, float("nan"), float("inf")):
        assert f(eps=e) == INV
    assert f(positions=P[9], kv_len=P[8]) == INV
    assert f(positions=P[9] + 2) == INV and f(inv_freq=P[10] + 1) == INV
    assert f(D=513, R=0) == UNS and f(B=2**30, L=2**10) == UNS and f(H=2**23) == UNS
    assert f(q=None) == INV and f(ko=None) == INV and f(q=P[0] + 2) == INV and f(wq=P[2] + 2) == INV
    assert f(s_q=[512, -128, 64]) == INV and f(s_q_out=[512, 64, 64]) == INV
    assert f(qo=P[0] + 256) == INV                       # over q, but not its very place
    assert f(qo=P[0], s_q_out=[1024, 128, 64]) == INV     # its place, other strides
    assert f(qo=P[1]) == INV and f(ko=P[0]) == INV and f(qo=P[5]) == INV and f(ko=P[2]) == INV
    assert f(qo=P[10]) == INV and f(positions=P[4]) == INV and f(kv_len=P[5]) == INV
    assert f(s_q=[2**62, 2**62, 64]) == INV

    def g(dqo=P[0], dko=P[1], q=P[2], k=P[3], dq=P[4], dk=P[5], dwq=P[6], dwk=P[7], ws=None, n=0, **opt):
        return h.sc_qk_norm_rotary_bwd(1, ctypes.byref(qk(sc, **opt)), dqo, dko, q, k, None, None, dq, dk, dwq, dwk,
                                       ws, n, None)

    assert g(D=0, R=0) == OK and g(B=0, dwq=None, dwk=None) == OK
    assert g(dqo=None) == INV and g(dk=None) == INV and g(dq=P[0]) == INV and g(dq=P[2]) == INV
    assert g(dwq=P[7]) == INV and g(dwk=P[7] + 1) == INV and g(n=64) == INV and g(dk=P[4] + 64) == INV
    need = sc.sc_qk_norm_rotary_workspace_bytes(1, qk(sc))
    assert need > 0 and sc.sc_qk_norm_rotary_workspace_bytes(1, qk(sc, R=1)) == 0
    assert g(ws=P[9], n=need - 1) == WS and g(ws=P[9] + 8, n=need) == INV and g(ws=P[2], n=need) == INV


def cache(sc, **k):
    c = sc.sc_cache(2, 4, 8, 2, 64, 0, P[0], P[1], P[2], P[3], None)
    for n, x in k.items():
        setattr(c, n, x)
    return c


def test_cache_refusals(sc):
    h = sc.lib()
    OK, INV, UNS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED

    def run(fn, kind=0, k=P[4], v=P[5], L=3, n=P[6], s=(384, 128, 64), sv=None, **opt):
        return fn(kind, ctypes.byref(cache(sc, **opt)), k, I3(*s), v, I3(*(sv or s)), L, n, None)

    for fn in (h.sc_cache_write, h.sc_cache_read):
        assert run(fn, L=0) == OK and run(fn, B=0) == OK and run(fn, Hkv=0) == OK and run(fn, D=0) == OK
        assert fn(0, None, P[4], I3(), P[5], I3(), 1, P[6], None) == INV
        assert run(fn, kind=2) == INV and run(fn, code=2) == INV and run(fn, L=-1) == INV
        for n in ("B", "N", "P", "Hkv", "D"):
            assert run(fn, **{n: -1}) == INV, n
        assert run(fn, D=72) == UNS and run(fn, D=144) == UNS and run(fn, L=2**30 + 1) == UNS
        assert run(fn, N=2**24 + 1, table=P[7]) == UNS and run(fn, P=2**31, table=P[7]) == UNS
        assert run(fn, P=7) == INV                                         # fewer blocks than rows need
        assert run(fn, k=None) == INV and run(fn, n=None) == INV and run(fn, n=P[6] + 2) == INV
        assert run(fn, k=P[4] + 8) == INV and run(fn, s=(384, 130, 64)) == INV and run(fn, s=(384, -128, 64)) == INV
        assert run(fn, table=P[7] + 2) == INV
        assert fn(0, ctypes.byref(cache(sc, k=None)), P[4], I3(384, 128, 64), P[5], I3(384, 128, 64), 3, P[6], None) == INV
    w, r = h.sc_cache_write, h.sc_cache_read
    assert run(w, N=0) == OK and run(w, P=0, table=P[7]) == OK              # no blocks: nothing is kept
    assert run(w, k=P[0] + 4096) == INV and run(w, v=P[3]) == INV and run(w, n=P[2]) == INV and run(w, table=P[1]) == INV
    assert run(r, k=P[1]) == INV and run(r, v=P[4] + 128) == INV and run(r, n=P[4]) == INV
    assert run(r, s=(384, 64, 64)) == INV                                  # results over each other
    assert run(w, k=P[0]) == INV and run(w, k_scale=P[0], k=P[4]) == INV


def cached(sc, **k):
    a = sc.sc_cached(3, 4, I3(768, 256, 64), I3(768, 256, 64), 0.125, 0.0, 0, 0, None, P[6])
    for n, x in k.items():
        setattr(a, n, x)
    return a


def test_cached_attention_refusals(sc):
    h = sc.lib()
    OK, INV, UNS, WS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED, sc.SC_ERR_WORKSPACE

    def f(kind=0, q=P[4], o=P[5], lse=P[7], ws=None, n=0, c=None, **opt):
        return h.sc_cached_attn(kind, ctypes.byref(c or cache(sc)), ctypes.byref(cached(sc, **opt)), q, o, lse, ws, n,
                                None)

    assert f(Lq=0) == OK and f(H=0) == OK and f(c=cache(sc, B=0)) == OK and f(c=cache(sc, D=0)) == OK
    assert h.sc_cached_attn(0, ctypes.byref(cache(sc)), None, P[4], P[5], None, None, 0, None) == INV
    assert f(kind=2) == INV and f(c=cache(sc, code=5)) == INV
    for n in ("Lq", "H", "window", "sinks"):
        assert f(**{n: -1}) == INV, n
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=s) == INV
    assert f(cap=-1.0) == INV and f(cap=float("nan")) == INV
    assert f(H=3) == UNS and f(c=cache(sc, Hkv=0)) == UNS and f(Lq=2**30) == UNS and f(c=cache(sc, D=40)) == UNS
    assert f(q=None) == INV and f(o=None) == INV and f(kv_len=None) == INV and f(q=P[4] + 8) == INV
    assert f(o=P[4]) == INV and f(o=P[1]) == INV and f(lse=P[5]) == INV and f(lse=P[7] + 2) == INV
    assert f(slopes=P[5]) == INV and f(slopes=P[8] + 2) == INV and f(kv_len=P[7]) == INV
    bad = cached(sc)
    bad.o[:] = [768, 64, 64]                                               # results over each other
    assert h.sc_cached_attn(0, ctypes.byref(cache(sc)), ctypes.byref(bad), P[4], P[5], None, None, 0, None) == INV
    big, one = cache(sc, N=1024, P=2048), cached(sc, Lq=1)
    need = sc.sc_cached_attn_workspace_bytes(0, big, one)
    assert need > 0 and sc.sc_cached_attn_workspace_bytes(0, big, cached(sc, H=3)) == 0
    assert f(c=big, Lq=1, ws=P[9], n=need - 4) == WS and f(c=big, Lq=1, ws=P[9] + 16, n=need) == INV
    assert f(c=big, Lq=1, ws=P[5], n=need) == INV


def test_tensor_front_end_refuses(sc):
    import torch
    x = torch.zeros(1, 4, 2, 64)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sc.qk_norm_rotary(x, x)
    with pytest.raises(TypeError):
        sc.qk_norm_rotary(x.double(), x)
    with pytest.raises(ValueError):
        sc.qk_norm_rotary_bwd(x, x, x, x)
    with pytest.raises(ValueError):
        sc.KVCache(1, 64, 2, 64, "int4", device="cpu")
    with pytest.raises(ValueError):
        sc.KVCache(1, 64, 2, 60, device="cpu")
    with pytest.raises(ValueError):
        sc.KVCache(2, 64, 2, 64, device="cpu", blocks=1)
    c = sc.KVCache(1, 100, 2, 64, device="cpu")
    assert (c.N, c.blocks) == (2, 2) and c.k.numel() == 2 * 2 * 64 * 64
    with pytest.raises(ValueError):
        c.table = torch.zeros(1, 2)
    with pytest.raises(ValueError):
        sc.cache_write(c, x, x, n)
    with pytest.raises(ValueError):
        sc.cache_read(c, 4, n)
    with pytest.raises(ValueError):
        sc.cached_attention(x, c, n)


# ------------------------------------------------------------------ the references

@pytest.mark.parametrize("pairs", [False, True])
def test_qk_gradient_against_differences(pairs):
    r = np.random.default_rng(3)
    x, dy, w = r.standard_normal((2, 3, 2, 7)), r.standard_normal((2, 3, 2, 7)), r.standard_normal(7)
    pos, f = np.array([[0, 5, 9], [100, 101, 7]]), np.array([1.0, 0.3])
    (dx, dw), _ = ref.qk_norm_bwd(dy, x, w, pos, f, pairs, 1e-3)
    assert np.allclose(dx, slope(lambda t: ref.qk_norm(t, w, pos, f, pairs, 1e-3)[0], x, dy), **TOL)
    assert np.allclose(dw, slope(lambda t: ref.qk_norm(x, t, pos, f, pairs, 1e-3)[0], w, dy), **TOL)


def test_rotation_by_hand():
    x = np.array([3.0, 4.0, 1.0, 2.0, 5.0]).reshape(1, 1, 1, 5)
    w = np.ones(5)
    quarter = np.array([[1]]), np.array([np.pi / 2, np.pi])   # a quarter and a half turn
    n = x / np.sqrt((x * x).mean())
    y = ref.qk_norm(x, w, *quarter, False, 0.0)[0] / n[..., 0] * 3      # pairs (0, 2) and (1, 3)
    assert np.allclose(y, [-1, -4, 3, -2, 5])
    y = ref.qk_norm(x, w, *quarter, True, 0.0)[0] / n[..., 0] * 3       # pairs (0, 1) and (2, 3)
    assert np.allclose(y, [-4, 3, -1, -2, 5])


def test_e4m3_and_exponents_by_hand():
    import torch
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = every[np.isfinite(every)]
    assert np.array_equal(ref.e4m3(every), every)
    x = np.concatenate([np.linspace(-470, 470, 4001), np.linspace(-0.05, 0.05, 4001)])
    near = np.sort(every)[np.abs(np.sort(every)[None] - x[:, None]).argmin(1)]
    assert np.all(np.abs(ref.e4m3(x) - x) <= np.abs(near - x))
    assert ref.e4m3(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16.0, 20.0, 0.0, 2.0 ** -8]   # ties
    assert ref.exponent(np.array([0.0, 127.0, 127.1, 63.5, 1e-30, 1e30]), "int8").tolist() == [-60, 0, 1, -1, -60, 60]
    assert ref.exponent(np.array([448.0, 449.0, 224.0]), "e4m3").tolist() == [0, 1, -1]


def test_cache_model_grows_a_scale():
    c = ref.Cache(1, 1, 1, 1, 16, "int8")
    one = np.full((1, 1, 1, 16), 100.0)
    c.write(one, one, [1])
    c.write(one * 3, one, [2])                       # 300 needs a step of 4
    k, v, live = c.read(3, [2])
    assert live.tolist() == [[False, True, True]] and k[0, :, 0, 0].tolist() == [0.0, 100.0, 300.0]
    c.write(one * 30, one, [3])                      # a step of 32: 100 is 3 of them, 300 is 9
    assert c.read(3, [3])[0][0, :, 0, 0].tolist() == [96.0, 288.0, 3008.0] and c.exps[0, 0, 0] == 5


def test_attention_reference_against_the_float_one():
    # without sinks and with every key, it is the reference of causal_attention
    r = np.random.default_rng(5)
    q, k, v = r.standard_normal((2, 3, 4, 8)), r.standard_normal((2, 9, 2, 8)), r.standard_normal((2, 9, 2, 8))
    for window in (0, 4):
        (o, l), _ = ref.cached_attention(q, k, v, [9, 6], 0.3, window=window, cap=2.0, slopes=[0.5, 0.1, 0.2, 0.0])
        (o2, l2), _ = lref.attention(q, k, v, 0.3, window=window, cap=2.0, slopes=[0.5, 0.1, 0.2, 0.0], kv_len=[9, 6])
        assert np.allclose(o, o2) and np.allclose(l, l2)
    # sinks by hand: window 2, two sinks, position 5 sees 0, 1, 4, 5
    (_, l), _ = ref.cached_attention(q[:1, :1], k[:1], v[:1], [6], 0.3, window=2, sinks=2)
    s = 0.3 * k[0, [0, 1, 4, 5], 0] @ q[0, 0, 0]
    assert np.isclose(l[0, 0, 0], np.log(np.exp(s).sum()))
