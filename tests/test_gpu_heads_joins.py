"""Attention over the 8-bit cache where the keys are split over workgroups."""
import numpy as np
import pytest
import torch

from oracle import heads as ref
from tests.layer_util import DEV, check, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


def parts(sc, c, Lq, H, kind, window=0):
    """Parts that the keys are split into, from the workspace they ask for."""
    a = sc.sc_cached(Lq, H)
    a.scale, a.window = 1.0, window
    need = sc.sc_cached_attn_workspace_bytes(kind, c._struct, a)
    return max(1, need // (c.B * Lq * H * (c.D + 1) * 4))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq", [1, 40])
def test_a_row_of_nan_is_nan_and_alone(sc, dtype, code, Lq):
    # split or not: lse is -infinity only where a row sees nothing
    print("case attn8 nan over parts", dtype, code, Lq, flush=True)
    rng = np.random.default_rng(4)
    for T in (130, 6000):
        c = sc.KVCache(1, T, 1, 64, code, device=DEV)
        k, _ = draw(rng, (1, T, 1, 64), "f32")
        sc.cache_write(c, k, k, lengths(T))
        q, _ = draw(rng, (1, Lq, 2, 64), dtype)
        kind = sc.KIND_F32 if dtype == "f32" else sc.KIND_BF16
        assert (parts(sc, c, Lq, 2, kind) > 1) == (T == 6000)
        want, wl = sc.cached_attention(q, c, lengths(T), lse=True)
        q[0, Lq - 1, 1, 9] = float("nan")
        o, lse = sc.cached_attention(q, c, lengths(T), lse=True)
        assert torch.isnan(lse[0, 1, Lq - 1]) and torch.isnan(o[0, Lq - 1, 1]).all(), T
        o[0, Lq - 1, 1], lse[0, 1, Lq - 1] = want[0, Lq - 1, 1], wl[0, 1, Lq - 1]
        assert torch.equal(o, want) and torch.equal(lse, wl)
        o, lse = sc.cached_attention(q, c, lengths(0), lse=True)
        assert torch.isneginf(lse).all() and o.eq(0).all()


@pytest.mark.parametrize("Hkv,want", [(192, 4), (256, 3), (384, 2)])
def test_parts_that_the_grid_limits(sc, Hkv, want):
    # many key heads over a long cache: few parts each
    print("case attn8 grid parts", Hkv, flush=True)
    T, D = 16400, 16
    gen = torch.Generator(device=DEV).manual_seed(Hkv)
    c = sc.KVCache(1, T, Hkv, D, "int8", device=DEV)
    k, v, q = (torch.randn(1, n, Hkv, D, generator=gen, device=DEV) for n in (T, T, 1))
    sc.cache_write(c, k, v, lengths(T))
    assert parts(sc, c, 1, Hkv, sc.KIND_F32) == want
    for n in (T, 100, 9000):
        o, lse = sc.cached_attention(q, c, lengths(n), lse=True)
        heads = [0, 1, Hkv // 2, Hkv - 1]
        kx, vx = (f64(t[:, :, heads]) for t in sc.cache_read(c, n, lengths(n), torch.float32))
        (ro, rl), (bo, bl) = ref.cached_attention(f64(q[:, :, heads]), kx, vx, [n], 0.25)
        check(o[:, :, heads], ro, bo, "f32", "o")
        check(lse[:, heads], rl, bl, "f32", "lse")


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 64), ("bf16", 128), ("f32", 48)])
@pytest.mark.parametrize("Lq,H", [(17, 1), (5, 4), (16, 2), (64, 1), (13, 5)])
def test_more_rows_over_split_keys(sc, Lq, H, dtype, D, code):
    # 17, 20, 32, 64 and 65 packed rows: workgroups of 64 rows with and without rows for each wave
    print("case attn8 rows over parts", Lq, H, dtype, D, code, flush=True)
    rng = np.random.default_rng(Lq * H)
    T = 5000
    c = sc.KVCache(2, T, 1, D, code, device=DEV)
    c.k.fill_(0xff)
    c.v.fill_(0xff)
    k, _ = draw(rng, (2, T, 1, D), "f32")
    v, _ = draw(rng, (2, T, 1, D), "f32")
    lens = [T, 1300]
    sc.cache_write(c, k, v, lengths(*lens))
    kx, vx = (f64(t) for t in sc.cache_read(c, c.N * 64, lengths(c.N * 64, c.N * 64), torch.float32))
    q, qx = draw(rng, (2, Lq, H, D), dtype, 1.5)
    kind = sc.KIND_F32 if dtype == "f32" else sc.KIND_BF16
    scale = float(np.float32(D ** -0.5))
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=DEV)
    for opt in ({}, dict(window=2100, sinks=70), dict(cap=20.0, slopes=slopes)):
        assert parts(sc, c, Lq, H, kind, opt.get("window", 0)) > 1
        o, lse = sc.cached_attention(q, c, lengths(*lens), lse=True, **opt)
        (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, lens, scale, opt.get("window", 0), opt.get("sinks", 0),
                                                  opt.get("cap", 0.0), f64(slopes) if "slopes" in opt else None,
                                                  bf16=dtype == "bf16")
        check(o, ro, bo, dtype, "o")
        check(lse, rl, bl, "f32", "lse")


@pytest.mark.parametrize("T,D,want", [(34000, 64, 66), (41000, 128, 80), (66000, 64, 129), (100000, 64, 195), (140000, 128, 256)])
def test_more_parts_than_a_wave_joins(sc, T, D, want):
    # The largest score stands in one key, taken through the parts that each wave of the join weighs: a
    # part that were lost or weighed wrongly would change everything.
    print("case attn8 many parts", T, D, flush=True)
    gen = torch.Generator(device=DEV).manual_seed(T)
    c = sc.KVCache(1, T, 1, D, "int8", device=DEV)
    k = torch.randn(1, T, 1, D, generator=gen, device=DEV)
    v = torch.randn(1, T, 1, D, generator=gen, device=DEV)
    q = torch.randn(1, 1, 3, D, generator=gen, device=DEV)
    assert parts(sc, c, 1, 3, sc.KIND_F32) == want
    scale = float(np.float32(D ** -0.5))
    for part in sorted({0, 1, 63, 64, 65, want // 2, want - 2, want - 1}):
        at = T - 1 - min(T - 1, part * T // want + 77)      # (parts go from the newest key to the oldest)
        kk = k.clone()
        kk[0, at, 0] = 14 * q[0, 0, 1] / q[0, 0, 1].norm() ** 2 / scale
        sc.cache_write(c, kk, v, lengths(T))
        o, lse = sc.cached_attention(q, c, lengths(T), lse=True)
        kx, vx = (f64(t) for t in sc.cache_read(c, T, lengths(T), torch.float32))
        s = scale * f64(q)[0, 0] @ kx[0, :, 0].T
        assert s[1].argmax() == at and s[1].max() > 12
        (ro, rl), (bo, bl) = ref.cached_attention(f64(q), kx, vx, [T], scale)
        # the sums are no chain of T additions: a part's of four waves, then the parts', 600 together
        n = (T - 600) * 2.0 ** -24
        w = np.exp(s - s.max(1, keepdims=True))
        bo = bo - n * ((w / w.sum(1, keepdims=True)) @ np.abs(vx[0, :, 0]))[None, None]
        check(o, ro, bo, "f32", "o")
        check(lse, rl, bl - n, "f32", "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq,H", [(1, 4), (20, 4)])
@pytest.mark.parametrize("T", [200, 6000])
def test_an_outlier_in_one_channel(sc, T, Lq, H, dtype):
    # A block whose v has one value 2^k times the others has a scale as much larger.  Weights are held
    # relative to the row's largest weight times scale, so the other channels of the row lose: up to 2^-32
    # of that for each key, times its code (where one half is kept, as bfloat16 does for many rows, 2^-12 of
    # the weight besides).
    print("case attn8 outlier", T, Lq, H, dtype, flush=True)
    rng = np.random.default_rng(T + Lq)
    D = 64
    k, _ = draw(rng, (1, T, 1, D), "f32", 0.5)
    v0, _ = draw(rng, (1, T, 1, D), "f32")
    q, qx = draw(rng, (1, Lq, H, D), dtype)
    half = 2.0 ** -12 if dtype == "bf16" and Lq * H > 16 else 2.0 ** -23
    for up in (10, 21, 30, 40):
        v = v0.clone()
        v[0, 70, 0, 5] = 2.0 ** up
        c = sc.KVCache(1, T, 1, D, "int8", device=DEV)
        sc.cache_write(c, k, v, lengths(T))
        kx, vx = (f64(t) for t in sc.cache_read(c, T, lengths(T), torch.float32))
        o = f64(sc.cached_attention(q, c, lengths(T)))
        vs = f64(c.v_scale)[np.arange(T) // 64, 0]
        codes = np.abs(vx[0, :, 0]) / vs[:, None]
        assert codes.max() <= 127
        for i in range(Lq):
            m = T - Lq + i + 1
            for h in range(H):
                s = 0.125 * kx[0, :m, 0] @ qx[0, i, h]
                w = np.exp(s - s.max())
                w /= w.sum()
                want = w @ vx[0, :m, 0]
                mag = w @ np.abs(vx[0, :m, 0])
                lost = 2.0 ** -32 * (w * vs[:m]).max() * codes[:m].sum(0)
                # the rest as in the reference: scores (2 D + 8 additions of |q| |k|, a query value's two
                # halves), exponents with the scales' and the base's roundings, sums
                sc_err = ((2 * D + 8) * 2.0 ** -24 + 2.0 ** -22) * (0.125 * np.abs(kx[0, :m, 0]) @ np.abs(qx[0, i, h])).max()
                rel = 2 * (sc_err + 8 * 2.0 ** -24 * (2 * np.abs(s).max() + 2 * up + 70)) + (m / 4 + 300) * 2.0 ** -24 + half
                bound = rel * mag + lost
                bound = bound + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(want) + bound)
                err = np.abs(o[0, i, h] - want)
                assert np.all(err <= bound), (up, i, h, (err / bound).max())
