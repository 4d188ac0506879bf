"""Norm and rotation of q and k against the float64 reference: sizes, layouts, positions, gradients."""
import numpy as np
import pytest
import torch

from oracle import heads as ref
from tests.layer_util import DEV, DTYPES, check, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def place(rng, B, L, H, D, dtype, how):
    """A (B, L, H, D) tensor and its values: dense, columns of a wider array, or rows that start
    anywhere."""
    if how == "dense":
        return draw(rng, (B, L, H, D), dtype, 1.5, 0.2)
    if how == "columns":
        t, x = draw(rng, (B, L, H + 3, D), dtype, 1.5, 0.2)
        return t[:, :, 1:H + 1], x[:, :, 1:H + 1]
    if how == "heads":   # (B, H, L, D) seen as (B, L, H, D)
        t, x = draw(rng, (B, H, L, D), dtype, 1.5, 0.2)
        return t.transpose(1, 2), x.swapaxes(1, 2)
    t, x = draw(rng, (B, L, H, D + 3), dtype, 1.5, 0.2)   # odd
    return t[..., 1:D + 1], x[..., 1:D + 1]


CASES = [
    # dtype, B, L, H, Hkv, D, R, pairs, positions, layout
    ("f32", 2, 5, 3, 1, 64, 64, False, "row", "dense"),
    ("bf16", 2, 5, 3, 1, 64, 64, False, "row", "columns"),
    ("bf16", 1, 1, 16, 4, 128, 128, False, "len", "dense"),
    ("f32", 1, 3, 4, 2, 128, 64, True, "list", "heads"),
    ("bf16", 2, 7, 2, 2, 64, 32, True, "list", "heads"),
    ("f32", 3, 4, 2, 3, 40, 24, False, "len", "columns"),     # R not of whole vectors
    ("bf16", 3, 4, 2, 3, 80, 48, False, "len", "columns"),
    ("bf16", 3, 4, 2, 3, 80, 80, True, "len", "columns"),
    ("bf16", 2, 3, 5, 1, 96, 96, False, "list", "odd"),
    ("f32", 2, 3, 5, 1, 7, 4, False, "list", "odd"),
    ("f32", 2, 3, 5, 1, 7, 6, True, "list", "dense"),
    ("bf16", 1, 6, 1, 1, 1, 0, False, "row", "dense"),
    ("f32", 1, 6, 1, 1, 2, 2, False, "list", "dense"),
    ("bf16", 1, 2, 2, 1, 512, 512, False, "len", "dense"),
    ("f32", 1, 2, 2, 1, 512, 256, True, "len", "dense"),
    ("f32", 1, 2, 2, 1, 511, 510, False, "len", "dense"),
    ("bf16", 1, 2, 2, 1, 256, 254, False, "list", "dense"),
    ("bf16", 2, 9, 2, 0, 64, 64, False, "row", "dense"),       # no k
    ("bf16", 2, 9000, 1, 1, 64, 64, False, "row", "dense"),    # more tokens than workgroups hold at once
    ("f32", 1, 2100, 3, 2, 40, 20, True, "list", "odd"),
    ("f32", 2, 5, 3, 2, 20, 12, False, "list", "dense"),       # vectors of every length
    ("bf16", 2, 5, 3, 2, 40, 20, False, "list", "dense"),
    ("bf16", 2, 5, 3, 2, 40, 24, False, "len", "columns"),
    ("bf16", 2, 5, 3, 2, 40, 30, True, "len", "heads"),
    ("bf16", 2, 5, 3, 2, 64, 26, False, "list", "dense"),
    ("f32", 2, 5, 3, 2, 120, 58, False, "list", "columns"),
    ("bf16", 2, 5, 3, 2, 127, 126, False, "list", "odd"),
    ("f32", 2, 5, 3, 2, 129, 128, True, "len", "odd"),
    ("f32", 2, 700, 3, 2, 256, 132, False, "len", "dense"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(sc, case):
    print("case qk", case, flush=True)
    dtype, B, L, H, Hkv, D, R, pairs, how, layout = case
    rng = np.random.default_rng(B * 7919 + L * 131 + D * 17 + R)
    q, qx = place(rng, B, L, H, D, dtype, layout)
    wq, wqx = draw(rng, (D,), dtype, 0.2, 1.0)
    gq, gqx = place(rng, B, L, H, D, dtype, layout)
    k = gk = wk = None
    if Hkv:
        k, kx = place(rng, B, L, Hkv, D, dtype, layout)
        wk, wkx = draw(rng, (D,), dtype, 0.2, 1.0)
        gk, gkx = place(rng, B, L, Hkv, D, dtype, layout)
    f = torch.from_numpy((10000.0 ** (-2.0 * np.arange(R // 2) / max(R, 1))).astype(np.float32)).to(DEV)
    fx = f64(f)
    pos = np.arange(L)[None].repeat(B, 0)
    opt = {"interleaved": pairs, "eps": 1e-5}
    if how == "len":
        n = np.array([60000 + 37 * b for b in range(B)], np.int32)
        pos = n[:, None] - L + pos
        opt["kv_len"] = torch.from_numpy(n).to(DEV)
    elif how == "list":
        pos = rng.integers(-5, 1 << 20, (B, L)).astype(np.int32)
        opt["positions"] = torch.from_numpy(pos).to(DEV)
    eps = float(np.float32(1e-5))
    y, z = sc.qk_norm_rotary(q, k, wq, wk, f, **opt)
    check(y, *ref.qk_norm(qx, wqx, pos, fx, pairs, eps), dtype, "q_out")
    out = sc.qk_norm_rotary_bwd(gq, gk, q, k, wq, wk, f, **opt)
    again = sc.qk_norm_rotary_bwd(gq, gk, q, k, wq, wk, f, **opt)
    for a, b in zip(out, again):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    (dx, dw), (bx, bw) = ref.qk_norm_bwd(gqx, qx, wqx, pos, fx, pairs, eps)
    check(out[0], dx, bx, dtype, "dq")
    check(out[2], dw, bw, dtype, "dq_weight")
    if Hkv:
        check(z, *ref.qk_norm(kx, wkx, pos, fx, pairs, eps), dtype, "k_out")
        (dx, dw), (bx, bw) = ref.qk_norm_bwd(gkx, kx, wkx, pos, fx, pairs, eps)
        check(out[1], dx, bx, dtype, "dk")
        check(out[3], dw, bw, dtype, "dk_weight")
    else:
        assert z is None and out[1] is None and out[3] is None


def test_far_positions(sc):
    # the angle of the last positions int32 holds, and frequencies down to 1e-6 of a radian
    print("case qk far", flush=True)
    rng = np.random.default_rng(1)
    pos = np.array([[2**29 - 1, -(2**29) + 1, 2**24 + 1, 1000003, 12345678, 0]], np.int32)
    x, xx = draw(rng, (1, 6, 1, 64), "f32")
    f = torch.from_numpy((500000.0 ** (-np.arange(32) / 32.0)).astype(np.float32)).to(DEV)
    y, _ = sc.qk_norm_rotary(x, None, None, None, f, positions=torch.from_numpy(pos).to(DEV))
    check(y, *ref.qk_norm(xx, np.ones(64), pos, f64(f), False, float(np.float32(1e-6))), "f32", "far")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 23])
def test_in_place_of_a_projections_columns(sc, dtype, D):
    print("case qk in place", dtype, D, flush=True)
    rng = np.random.default_rng(2)
    p, px = draw(rng, (2, 5, 8, D), dtype)
    before = p.clone()
    f = torch.rand(D // 2, device=DEV)
    want = sc.qk_norm_rotary(p[:, :, :4], p[:, :, 4:6], None, None, f)
    q, k = p[:, :, :4], p[:, :, 4:6]
    got = sc.qk_norm_rotary(q, k, None, None, f, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == p.data_ptr()
    assert torch.equal(p[:, :, 6:], before[:, :, 6:])      # the columns beside them are as they were
    with pytest.raises(sc.SpecConvError):
        sc.qk_norm_rotary(q, k, None, None, f, q_out=p[:, :, 2:6])
    with pytest.raises(sc.SpecConvError):
        sc.qk_norm_rotary(q, k, None, None, f, q_out=q, k_out=p[:, :, 3:5])


def test_rows_of_nan_and_infinity_stay_alone(sc):
    print("case qk nan", flush=True)
    for dtype in ("f32", "bf16"):
        for D in (64, 20):
            x, _ = draw(np.random.default_rng(3), (1, 6, 3, D), dtype)
            g = torch.ones_like(x)
            bad = x.clone()
            bad[0, 2, 1, 5] = float("nan")
            bad[0, 4, 0, 7] = float("inf")
            f = torch.rand(D // 2, device=DEV)
            good, worse = (sc.qk_norm_rotary(t, None, None, None, f)[0] for t in (x, bad))
            dg, dw = (sc.qk_norm_rotary_bwd(g, None, t, None, None, None, f, params=False)[0] for t in (x, bad))
            hit = torch.zeros(1, 6, 3, dtype=torch.bool, device=DEV)
            hit[0, 2, 1] = hit[0, 4, 0] = True
            for a, b in ((good, worse), (dg, dw)):
                assert torch.equal(a[~hit], b[~hit])
                assert not torch.isfinite(b[0, 2, 1]).any()


def test_zero_rows_and_empty_calls(sc):
    print("case qk empty", flush=True)
    z = torch.zeros(1, 3, 2, 64, device=DEV)
    y, _ = sc.qk_norm_rotary(z, None, None, None, None)
    assert torch.equal(y, z)
    dx, _, dw, _ = sc.qk_norm_rotary_bwd(z + 1, None, z, None)
    assert torch.isfinite(dx).all() and torch.equal(dw, torch.zeros(64, device=DEV))
    for shape in ((0, 3, 2, 64), (1, 0, 2, 64), (1, 3, 0, 64)):
        e = torch.zeros(shape, device=DEV)
        assert sc.qk_norm_rotary(e, e)[0].shape == e.shape
        dx, dk, dw, dv = sc.qk_norm_rotary_bwd(e, e, e, e)
        assert dw.eq(0).all() and dv.eq(0).all() and dw.shape == (64,)


def test_workspace_and_refusals(sc):
    print("case qk workspace", flush=True)
    x = torch.randn(1, 50, 2, 64, device=DEV)
    f = torch.rand(32, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    a, b = sc.qk_norm_rotary_bwd(x, x, x, x, None, None, f), sc.qk_norm_rotary_bwd(x, x, x, x, None, None, f, workspace=ws)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    with pytest.raises(sc.SpecConvError):
        sc.qk_norm_rotary_bwd(x, x, x, x, None, None, f, workspace=ws[:256])
    for bad in (dict(positions=torch.zeros(1, 49, dtype=torch.int32, device=DEV)),
                dict(kv_len=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(positions=torch.zeros(1, 50, dtype=torch.int64, device=DEV)),
                dict(q_out=torch.empty(1, 50, 2, 32, device=DEV))):
        with pytest.raises(ValueError):
            sc.qk_norm_rotary(x, x, None, None, f, **bad)
    for bad in ((x[:, :3], x, None, None, f), (x, x, torch.ones(32, device=DEV), None, f),
                (x, x, None, None, torch.rand(33, device=DEV)), (x, x.bfloat16(), None, None, f)):
        with pytest.raises(ValueError):
            sc.qk_norm_rotary(*bad)
