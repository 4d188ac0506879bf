"""How many bits the weights of attention over the 8-bit cache keep."""
import numpy as np
import pytest
import torch

from tests.layer_util import DEV, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


def softmax(s):
    e = np.exp(s - s.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


# 16 packed rows at most: one block, two, and keys over workgroups
FEW = [(40, 1, 4, 1), (64, 1, 16, 1), (100, 3, 4, 2), (200, 16, 1, 1), (6000, 1, 16, 2), (4000, 2, 8, 1)]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(map(str, c)))
def test_few_rows_keep_the_weights_bits(sc, case, dtype, code):
    # Neighbouring keys have nearly one score and opposite values, so that o is small beside the sum of
    # w |v| and shows what the weights lost.  Scores are exact products of one value of q and one code.
    print("case attn8 weights", case, dtype, code, flush=True)
    T, Lq, H, Hkv = case
    D, scale = 16, 2.0 ** -7
    rng = np.random.default_rng(T + Lq)
    n = np.arange(T)
    k = np.zeros((1, T, Hkv, D))
    # codes whose neighbours differ by one step (e4m3: integers up to 16)
    k[0, :, :, 0] = ((n // 2 * 7) % 100 + n % 2)[:, None] if code == "int8" else ((n // 2 * 3) % 15 + n % 2)[:, None]
    k[0, :, :, 1] = 127 if code == "int8" else 448         # the block's largest: scale 1 (q's value there is 0)
    v = np.zeros((1, T, Hkv, D))
    pairs = (1, (T + 1) // 2, Hkv, D)
    size = rng.integers(60, 128, pairs) if code == "int8" else 32.0 * rng.integers(8, 15, pairs)
    size = size * (1 - 2 * (np.arange(pairs[1]) % 2))[None, :, None, None]
    v[0] = size[0][n // 2] * (1 - 2 * (n % 2))[:, None, None]
    v[0, ::64], v[0, 1::64] = (127, -127) if code == "int8" else (448, -448)
    q = np.zeros((1, Lq, H, D))
    q[..., 0] = rng.choice([-1.0, -0.75, 0.5, 0.875, 1.0], (1, Lq, H))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    kt, vt, qt = (torch.from_numpy(x).to(DEV, torch.float32) for x in (k, v, q))
    c = sc.KVCache(1, T, Hkv, D, code, device=DEV)
    sc.cache_write(c, kt, vt, lengths(T))
    got = sc.cache_read(c, T, lengths(T), torch.float32)
    assert np.array_equal(f64(got[0]), k) and np.array_equal(f64(got[1]), v)      # every value is a code
    o, lse = sc.cached_attention(qt.to(dt), c, lengths(T), scale=scale, lse=True)
    ro, bo = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(Lq):
        m = T - Lq + i + 1
        for h in range(H):
            g = h // (H // Hkv)
            s = scale * q[0, i, h, 0] * k[0, :m, g, 0]
            w = softmax(s)
            ro[0, i, h] = w @ v[0, :m, g]
            # Exponents in base 2, at most 16: |s| + 7 and the base, three roundings of 2^-21 each with
            # the factor's, ln 2 times that in a weight; the exponential's 2^-23; a weight's two halves
            # 2^-22; additions in float32, of a wave's keys (a quarter, or one block) and what joins them:
            # once of the products, once of the sum that divides them.
            a = 2.2 * 2.0 ** -21 + 2.0 ** -22 + (m / 4 + 80) * 2.0 ** -24
            bo[0, i, h] = a * (w @ np.abs(v[0, :m, g]) + np.abs(ro[0, i, h]))
    check(o, ro, bo, dtype, "o")
    assert np.abs(ro).max() < 0.1 * np.abs(v).max()
