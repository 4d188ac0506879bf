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
