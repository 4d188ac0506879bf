"""The pointer-level Python mirrors of the layer calls against the tensor front end."""
import pytest
import torch

from tests.layer_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def rand(*shape):
    return torch.randn(*shape, device=DEV)


def stream():
    return torch.cuda.current_stream().cuda_stream


def same(got, want):
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_layernorm(sc):
    R, C = 37, 200
    x, w, b, dy = rand(R, C), rand(C), rand(C), rand(R, C)
    want = sc.layer_norm(x, w, b, 1e-4, stats=True)
    got = [torch.full_like(t, 7.0) for t in want]
    p = [t.data_ptr() for t in got]
    st = sc.sc_layernorm(sc.KIND_F32, x.data_ptr(), w.data_ptr(), b.data_ptr(), *p, R, C, C, C, 1e-4, stream())
    assert st == sc.SC_OK
    same(got, want)
    want = sc.layer_norm_bwd(dy, x, got[1], got[2], w)
    back = [torch.full_like(t, 7.0) for t in want]
    n = sc.sc_layernorm_bwd_workspace_bytes(sc.KIND_F32, R, C)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    st = sc.sc_layernorm_bwd(sc.KIND_F32, dy.data_ptr(), x.data_ptr(), w.data_ptr(), p[1], p[2],
                             *(t.data_ptr() for t in back), R, C, C, C, C, ws.data_ptr(), n, stream())
    assert st == sc.SC_OK
    same(back, want)


def test_recur(sc):
    B, L, C = 1, 3000, 48
    z, u, dh, h0, dhT = rand(B, L, C) + 1, rand(B, L, C), rand(B, L, C), rand(B, C), rand(B, C)
    n = sc.sc_recur_workspace_bytes(sc.KIND_F32, B, L, C)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    want = sc.gated_recurrence(z, u, h0)
    got = [torch.full_like(t, 7.0) for t in want]
    st = sc.sc_recur(sc.KIND_F32, z.data_ptr(), u.data_ptr(), h0.data_ptr(), *(t.data_ptr() for t in got), B, L, C,
                     C, C, C, ws.data_ptr(), n, stream())
    assert st == sc.SC_OK
    same(got, want)
    want = sc.gated_recurrence_bwd(dh, z, u, got[0], h0, dhT)
    back = [torch.full_like(t, 7.0) for t in want]
    st = sc.sc_recur_bwd(sc.KIND_F32, dh.data_ptr(), z.data_ptr(), u.data_ptr(), got[0].data_ptr(), h0.data_ptr(),
                         dhT.data_ptr(), *(t.data_ptr() for t in back), B, L, C, C, C, C, C, C, C, ws.data_ptr(), n,
                         stream())
    assert st == sc.SC_OK
    same(back, want)


def test_causal_attn(sc):
    B, Lq, Lk, H, Hkv, D = 2, 50, 130, 4, 2, 64
    q, k, v, do = rand(B, Lq, H, D), rand(B, Lk, Hkv, D), rand(B, Lk, Hkv, D), rand(B, Lq, H, D)
    opt = dict(window=60, cap=9.0)
    o, lse = sc.causal_attention(q, k, v, lse=True, **opt)
    a = sc.sc_attn(B, Lq, Lk, H, Hkv, D)
    for n in ("q", "o", "dout", "dq"):
        getattr(a, n)[:] = [Lq * H * D, H * D, D]
    for n in ("k", "v", "dk", "dv"):
        getattr(a, n)[:] = [Lk * Hkv * D, Hkv * D, D]
    a.scale, a.cap, a.window = D ** -0.5, 9.0, 60

    def scratch(backward):
        n = sc.sc_attn_workspace_bytes(sc.KIND_F32, a, backward)
        t = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        return t, None if t is None else t.data_ptr(), n

    got = [torch.full_like(t, 7.0) for t in (o, lse)]
    keep, ws, n = scratch(0)
    st = sc.sc_causal_attn(sc.KIND_F32, a, q.data_ptr(), k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in got), ws,
                           n, stream())
    assert st == sc.SC_OK
    same(got, (o, lse))
    want = sc.causal_attention_bwd(do, q, k, v, o, lse, **opt)
    back = [torch.full_like(t, 7.0) for t in want]
    keep, ws, n = scratch(1)
    st = sc.sc_causal_attn_bwd(sc.KIND_F32, a, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               lse.data_ptr(), *(t.data_ptr() for t in back), ws, n, stream())
    assert st == sc.SC_OK
    same(back, want)
