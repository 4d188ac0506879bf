"""Attention over the 8-bit cache where the factors of a score pass float32's range on their way."""
import numpy as np
import pytest
import torch

from tests.layer_util import DEV, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


CASES = [
    # q's value, scale, cap, k's scale
    (1.5 * 2.0 ** 127, 1.0, 0.0, 2.0 ** 20),       # the row's power of two times the block's scale
    (1.5 * 2.0 ** 127, 2.0 ** 20, 0.0, 1.0),       # the row's power of two times the call's
    (2.0 ** 30, 1.0, 1e-37, 2.0 ** 20),            # over the cap
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq", [1, 20])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join("%.3g" % x for x in c))
def test_products_of_zero_stay_zero(sc, case, Lq, dtype):
    # q and every key have their values in different places: scores of 0, whatever the factors
    print("case attn8 factors", case, Lq, dtype, flush=True)
    big, scale, cap, ks = case
    rng = np.random.default_rng(2)
    T = 70
    k = np.zeros((1, T, 1, 64), np.float32)
    k[..., 1::2] = rng.integers(-127, 128, (1, T, 1, 32)) * ks
    k[0, ::64, 0, 1] = 127 * ks
    v = rng.integers(-127, 128, (1, T, 1, 64)).astype(np.float32)
    v[0, ::64] = 127
    q = np.zeros((1, Lq, 2, 64), np.float32)
    q[..., ::2] = big
    c = sc.KVCache(1, T, 1, 64, "int8", device=DEV)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    sc.cache_write(c, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), n)
    qt = torch.from_numpy(q).to(DEV, torch.float32 if dtype == "f32" else torch.bfloat16)
    o, lse = sc.cached_attention(qt, c, n, scale=scale, cap=cap, lse=True)
    m = T - Lq + 1 + np.arange(Lq)
    want = np.cumsum(v[0, :, 0].astype(np.float64), 0)[m - 1] / m[:, None]
    # weights of 1: an exponential (2^-23), additions of up to 70 values, a quotient; two more of log2 and ln 2
    assert np.abs(f64(o)[0] - want[:, None]).max() <= 127 * (90 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0))
    assert np.abs(f64(lse)[0] - np.log(m)).max() <= 90 * 2.0 ** -24 * 5


def test_a_score_inside_the_range(sc):
    # 2^20 q alone passes float32; times k it is 2^87 for one key and less for the others
    print("case attn8 factors inside", flush=True)
    T = 65
    k = np.full((1, T, 1, 64), 2.0 ** -60, np.float32)
    k[0, 40] *= 3
    k[0, :, 0, 1] = 127 * 2.0 ** -60
    v = np.arange(T, dtype=np.float32).reshape(1, T, 1, 1).repeat(64, 3)
    c = sc.KVCache(1, T, 1, 64, "int8", device=DEV)
    n = torch.tensor([T], dtype=torch.int32, device=DEV)
    sc.cache_write(c, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), n)
    q = torch.zeros(1, 1, 1, 64, device=DEV)
    q[..., 0] = 2.0 ** 127
    o, lse = sc.cached_attention(q, c, n, scale=2.0 ** 20, lse=True)
    assert o.eq(40).all() and abs(float(lse[0, 0, 0]) / (3 * 2.0 ** 87) - 1) < 2.0 ** -20
