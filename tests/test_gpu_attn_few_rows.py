"""Attention of few rows (decoding) in bfloat16: the result is that of float32 weights, rounded once."""
import numpy as np
import pytest
import torch

from oracle import layers as ref
from tests.layer_util import DEV, check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("Lq,Lk,H,Hkv,D", [(1, 700, 8, 8, 64), (1, 3000, 8, 1, 128), (2, 129, 16, 2, 40),
                                           (16, 333, 3, 3, 96), (1, 31, 16, 1, 64)])
@pytest.mark.parametrize("cap,bias,window", [(0.0, False, 0), (20.0, True, 0), (0.0, True, 100)])
def test_weights_keep_their_bits(sc, Lq, Lk, H, Hkv, D, cap, bias, window):
    print("case attn few rows Lq=%d Lk=%d H=%d D=%d cap=%g W=%d" % (Lq, Lk, H, D, cap, window), flush=True)
    rng = np.random.default_rng([Lq, Lk, H, D])
    B = 3
    q, qr = draw(rng, (B, Lq, H, D), "bf16")
    k, kr = draw(rng, (B, Lk, Hkv, D), "bf16")
    v, vr = draw(rng, (B, Lk, Hkv, D), "bf16")
    slopes = np.asarray([2.0 ** (-8 * (h + 1) / H) for h in range(H)], np.float32) if bias else None
    kv_len = [Lk, max(Lk // 2, Lq), Lk - 1]
    o = sc.causal_attention(q, k, v, window=window, cap=cap, slopes=None if slopes is None else torch.from_numpy(slopes).to(DEV),
                            kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV))
    opt = dict(window=window, cap=cap, slopes=slopes, kv_len=kv_len)
    scale = float(np.float32(D ** -0.5))
    (want, _), (bound, _) = ref.attention(qr, kr, vr, scale, **opt)
    rounded = ref.attention(qr, kr, vr, scale, bf16=True, **opt)[1][0]
    # a weight as the sum of two bfloat16 values is off by up to (2^-8)^2 of itself
    check(o, want, bound + ref.UB * (rounded - bound), "bf16", "o")
