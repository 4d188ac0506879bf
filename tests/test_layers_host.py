"""The layer calls without a GPU: what they refuse on the host before any HIP call, and the
float64 references the GPU tests compare with (gradients against central differences)."""
import ctypes

import numpy as np
import pytest

from oracle import layers as ref

# fake, never dereferenced, far enough apart not to overlap
P = [0x10000000000 * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def sc():
    from tests.test_abi import LIB
    import os
    assert os.path.exists(LIB), "libspecconv.so is not built"
    import fft_causal_long_amd as m
    return m


def test_layernorm_refusals(sc):
    h = sc.lib()
    OK, INV, UNS, WS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED, sc.SC_ERR_WORKSPACE

    def f(kind=0, x=P[0], w=P[1], b=P[2], y=P[3], mean=P[4], rstd=P[5], rows=0, C=8, xs=8, ys=8, eps=1e-5):
        return h.sc_layernorm(kind, x, w, b, y, mean, rstd, rows, C, xs, ys, eps, None)

    assert f() == OK and f(rows=4, C=0, xs=0, ys=0, x=None, y=None) == OK      # nothing to do
    assert f(kind=2) == INV and f(kind=9) == INV                              # float kinds only
    assert f(rows=-1) == INV and f(C=-1) == INV and f(xs=-1) == INV
    assert f(rows=4, ys=7) == INV                                             # output rows overlap
    for eps in (-1e-5, float("nan"), float("inf")):
        assert f(rows=4, eps=eps) == INV
    assert f(rows=4, x=None) == INV and f(rows=4, y=None) == INV
    assert f(rows=4, x=P[0] + 2) == INV and f(rows=4, mean=P[4] + 2) == INV    # element alignment
    assert f(rows=4, y=P[0]) == INV and f(rows=4, y=P[0] + 64) == INV          # y over x
    assert f(rows=4, y=P[1]) == INV and f(rows=4, rstd=P[4]) == INV
    assert f(rows=4, y=P[0] + 32, xs=12, ys=12) == INV                         # columns 8.. reach the next row's x
    assert f(rows=2**61, xs=8, ys=8) == INV                                    # extents past 63 bits
    assert f(C=2**30 + 1, xs=2**31, ys=2**31) == UNS

    def g(rows=4, C=8, dys=8, xs=8, dxs=8, dw=P[6], db=P[7], ws=None, n=0, dx=P[5], dy=P[0], kind=0):
        return h.sc_layernorm_bwd(kind, dy, P[1], P[2], P[3], P[4], dx, dw, db, rows, C, dys, xs, dxs, ws, n, None)

    assert g(rows=0, dw=None, db=None) == OK and g(C=0, dys=0, xs=0, dxs=0) == OK
    assert g(kind=3) == INV and g(dxs=7) == INV and g(dx=P[0]) == INV and g(dw=P[7]) == INV
    assert g(dy=None) == INV and g(n=512) == INV                               # bytes without a workspace
    need = sc.sc_layernorm_bwd_workspace_bytes(0, 4, 8)
    assert need > 0
    assert g(ws=P[9] + 16, n=need) == INV and g(ws=P[9], n=need - 4) == WS
    assert g(ws=P[1], n=need) == INV                                           # over an input
    assert sc.sc_layernorm_bwd_workspace_bytes(2, 4, 8) == 0


def test_recur_refusals(sc):
    h = sc.lib()
    OK, INV, UNS, WS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED, sc.SC_ERR_WORKSPACE

    def f(kind=0, z=P[0], u=P[1], h0=P[2], o=P[3], hT=P[4], B=1, L=8, C=8, zs=8, us=8, hs=8, ws=None, n=0):
        return h.sc_recur(kind, z, u, h0, o, hT, B, L, C, zs, us, hs, ws, n, None)

    assert f(B=0) == OK and f(C=0, zs=0, us=0, hs=0) == OK
    assert f(L=0, hT=None) == OK and f(L=0, h0=P[4]) == OK                     # states in place: nothing to copy
    assert f(kind=2) == INV and f(B=-1) == INV and f(L=-1) == INV and f(C=-1) == INV
    assert f(zs=-1) == INV and f(hs=7) == INV
    assert f(z=None) == INV and f(u=None) == INV and f(o=None) == INV
    assert f(z=P[0] + 2) == INV and f(hT=P[4] + 2) == INV
    assert f(o=P[0]) == INV and f(o=P[1]) == INV and f(o=P[2]) == INV and f(hT=P[0]) == INV
    assert f(hT=P[2] + 16) == INV                                              # the state half over itself
    assert f(B=2**31, C=1) == UNS and f(C=2**30 + 1, zs=2**31, us=2**31, hs=2**31, L=1) == UNS
    assert f(B=2**20, L=2**20, C=2**25) == INV                                 # sizes past 63 bits
    need = sc.sc_recur_workspace_bytes(0, 1, 65536, 8)
    assert need > 0 and sc.sc_recur_workspace_bytes(0, 1, 8, 8) == 0
    assert f(L=65536, ws=P[9], n=need - 1) == WS and f(L=65536, ws=P[9] + 4, n=need) == INV
    assert f(L=65536, ws=P[3], n=need) == INV

    def g(strides=(8,) * 6, dz=P[4], du=P[5], dh0=P[6], dhT=P[7], h0=P[8], L=8, dh=P[0]):
        return h.sc_recur_bwd(0, dh, P[1], P[2], P[3], h0, dhT, dz, du, dh0, 1, L, 8, *strides, None, 0, None)

    assert g(L=0, dhT=P[6]) == OK and g(dh=None) == INV and g(dz=P[5]) == INV and g(dz=P[3]) == INV
    assert g(strides=(8, 8, 8, 8, 7, 8)) == INV and g(strides=(8, -8, 8, 8, 8, 8)) == INV
    assert g(dh0=P[8]) == INV and g(dh0=P[7] + 4) == INV


def attn(sc, **k):
    a = sc.sc_attn(1, 8, 8, 2, 2, 64)
    for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
        getattr(a, n)[:] = [1024, 128, 64]
    a.scale = 0.125
    for n, x in k.items():
        if n.startswith("s_"):     # strides of a tensor
            getattr(a, n[2:])[:] = x
        else:
            setattr(a, n, x)
    return a


def test_attention_refusals(sc):
    h = sc.lib()
    OK, INV, UNS, WS = sc.SC_OK, sc.SC_ERR_INVALID_ARGUMENT, sc.SC_ERR_UNSUPPORTED, sc.SC_ERR_WORKSPACE

    def f(kind=0, q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], ws=None, n=0, **opt):
        return h.sc_causal_attn(kind, ctypes.byref(attn(sc, **opt)), q, k, v, o, lse, ws, n, None)

    assert f(B=0) == OK and f(Lq=0) == OK and f(D=0) == OK and f(H=0, Hkv=0) == OK
    assert h.sc_causal_attn(0, None, P[0], P[1], P[2], P[3], None, None, 0, None) == INV
    assert f(kind=2) == INV
    for n in ("B", "Lq", "Lk", "H", "Hkv", "D", "window"):
        assert f(**{n: -1}) == INV, n
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=s) == INV
    assert f(cap=-1.0) == INV and f(cap=float("nan")) == INV
    assert f(D=60) == UNS and f(D=136) == UNS and f(H=3) == UNS and f(Hkv=0) == UNS
    assert f(Lk=2**30 + 1) == UNS and f(Lq=2**30, H=4) == UNS
    assert f(q=None) == INV and f(k=None) == INV and f(o=None) == INV
    assert f(q=P[0] + 8) == INV and f(s_k=[1024, 130, 64]) == INV               # 16-byte rows
    assert f(s_o=[1024, 64, 64]) == INV and f(s_o=[1024, 128, 32]) == INV          # an output over itself
    assert f(s_o=[0, 128, 64], B=2) == INV and f(s_k=[1024, -128, 64]) == INV
    assert f(o=P[0]) == INV and f(o=P[2] + 256) == INV and f(lse=P[1]) == INV
    assert f(lse=P[4] + 2) == INV and f(slopes=P[5] + 2) == INV and f(kv_len=P[3]) == INV
    big = dict(Lq=1, Lk=65536)
    need = sc.sc_attn_workspace_bytes(0, attn(sc, **big), 0)
    assert need > 0 and sc.sc_attn_workspace_bytes(0, attn(sc, D=60), 0) == 0
    assert f(ws=P[9], n=need - 4, **big) == WS and f(ws=P[9] + 16, n=need, **big) == INV
    assert f(ws=P[3], n=need, **big) == INV

    def g(kind=1, dout=P[0], q=P[1], k=P[2], v=P[3], o=P[4], lse=P[5], dq=P[6], dk=P[7], dv=P[8], ws=None, n=0,
          **opt):
        return h.sc_causal_attn_bwd(kind, ctypes.byref(attn(sc, **opt)), dout, q, k, v, o, lse, dq, dk, dv, ws, n,
                                    None)

    assert g(B=0) == OK and g(Lq=0, Lk=0) == OK
    assert g(lse=None) == INV and g(dout=None) == INV and g(dq=P[7]) == INV and g(dk=P[2]) == INV
    assert g(s_dv=[1024, 64, 64]) == INV and g(D=4) == UNS
    need = sc.sc_attn_workspace_bytes(1, attn(sc), 1)
    assert need > 0 and g(ws=P[9], n=need - 1) == WS
    # columns of one array: dk and dv side by side are apart, dk over dv is not
    side = dict(s_dk=[2048, 256, 64], s_dv=[2048, 256, 64])
    assert g(dk=P[7], dv=P[7] + 128, ws=P[9], n=need - 1, **side) == INV
    assert g(dk=P[7], dv=P[7] + 256, ws=P[9], n=need - 1, **side) == WS


def test_tensor_front_end_refuses_host_tensors(sc):
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        sc.layer_norm(x)
    with pytest.raises(TypeError):
        sc.layer_norm(x.double())
    with pytest.raises(ValueError):
        sc.gated_recurrence(x, x)
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        sc.causal_attention(q, q, q)


# ------------------------------------------------------------------ the references

def slope(f, x, g, eps=1e-5):
    """Central difference of sum(f(x) * g) along each element of x."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        d[i] = ((f(a) - f(b)) * g).sum() / (2 * eps)
    return d


# differences of step 1e-5 in 64 bits: 1e-11 relative rounding over the step, 1e-10 curvature
TOL = dict(rtol=1e-6, atol=1e-7)


def test_layernorm_gradient_against_differences():
    r = np.random.default_rng(0)
    x, w, b, dy = r.standard_normal((3, 7)), r.standard_normal(7), r.standard_normal(7), r.standard_normal((3, 7))
    (_, mean, rstd), _ = ref.layernorm(x, w, b, 1e-3)
    (dx, dw, db), _ = ref.layernorm_bwd(dy, x, w, mean, rstd)
    assert np.allclose(dx, slope(lambda t: ref.layernorm(t, w, b, 1e-3)[0][0], x, dy), **TOL)
    assert np.allclose(dw, slope(lambda t: ref.layernorm(x, t, b, 1e-3)[0][0], w, dy), **TOL)
    assert np.allclose(db, slope(lambda t: ref.layernorm(x, w, t, 1e-3)[0][0], b, dy), **TOL)


def test_recurrence_gradient_against_differences():
    r = np.random.default_rng(1)
    z, u, dh = (r.standard_normal((2, 6, 3)) for _ in range(3))
    h0, dhT = r.standard_normal((2, 3)), r.standard_normal((2, 3))

    def f(z, u, h0):
        (h, hT), _ = ref.recurrence(z, u, h0)
        return np.concatenate([h.ravel(), hT.ravel()])

    g = np.concatenate([dh.ravel(), dhT.ravel()])
    (h, _), _ = ref.recurrence(z, u, h0)
    (dz, du, dh0), _ = ref.recurrence_bwd(dh, z, u, h, h0, dhT)
    assert np.allclose(dz, slope(lambda t: f(t, u, h0), z, g), **TOL)
    assert np.allclose(du, slope(lambda t: f(z, t, h0), u, g), **TOL)
    assert np.allclose(dh0, slope(lambda t: f(z, u, t), h0, g), **TOL)


@pytest.mark.parametrize("cap", [0.0, 1.5])
def test_attention_gradient_against_differences(cap):
    r = np.random.default_rng(2)
    B, L, H, Hkv, D = 2, 7, 4, 2, 8
    q, do = r.standard_normal((B, L, H, D)), r.standard_normal((B, L, H, D))
    k, v = r.standard_normal((B, L, Hkv, D)), r.standard_normal((B, L, Hkv, D))
    doc = np.array([[0, 0, 0, 3, 3, 9, 3], [0, 1, 1, 1, 1, 1, 1]])
    opt = dict(window=3, cap=cap, slopes=[0.5, 0.25, 0.1, 0.0], kv_len=[7, 5], doc=doc)

    def f(q, k, v):
        return ref.attention(q, k, v, 0.3, **opt)[0][0]

    (o, lse), _ = ref.attention(q, k, v, 0.3, **opt)
    (dq, dk, dv), _ = ref.attention_bwd(do, q, k, v, o, lse, 0.3, **opt)
    assert np.allclose(dq, slope(lambda t: f(t, k, v), q, do), **TOL)
    assert np.allclose(dk, slope(lambda t: f(q, t, v), k, do), **TOL)
    assert np.allclose(dv, slope(lambda t: f(q, k, t), v, do), **TOL)


def test_attention_masks_by_hand():
    see, far = ref.visible(3, 5, 2, 5, np.array([0, 0, 2, 9, 2]))
    # positions 2, 3, 4; window 2; token 3 is padding
    assert see.tolist() == [[False, False, True, False, False], [False] * 5, [False, False, False, False, True]]
    assert far[0].tolist() == [2, 1, 0, -1, -2]
    see, _ = ref.visible(2, 3, 0, 1, None)     # one key: the first row lies before the sequence
    assert see.tolist() == [[False] * 3, [True, False, False]]
