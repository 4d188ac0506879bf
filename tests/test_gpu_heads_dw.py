"""The sums of the weights' gradients of qk_norm_rotary over many workgroups."""
import numpy as np
import pytest
import torch

from oracle import heads as ref
from tests.layer_util import DEV, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("D", [64, 20, 130])
def test_parts_that_cancel(sc, D):
    # Rows of +-1 without eps: the norm is 1 and a row's share of dw is +-dy, exact.  The first and the last
    # token carry 2^20 and -2^20, tokens near them nothing, the others 2^-6: together a number of 14
    # bits, of which a float32 sum that holds 2^20 meanwhile would lose all below 2^-4.  (8192 tokens are
    # dealt to 2048 workgroups once, so no register holds a large and a small share.)
    print("case qk dw cancels", D, flush=True)
    L = 8192
    rng = np.random.default_rng(D)
    x = np.where(rng.random((1, L, 1, D)) < 0.5, -1.0, 1.0)
    share = np.full((1, L, 1, D), 2.0 ** -6)
    share[:, :64] = share[:, -64:] = 0
    share[:, 0], share[:, -1] = 2.0 ** 20, -(2.0 ** 20)
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    g = torch.from_numpy((share * x).astype(np.float32)).to(DEV)
    _, _, dw, _ = sc.qk_norm_rotary_bwd(g, None, t, None, eps=0.0)
    assert np.array_equal(f64(dw), np.full(D, (L - 128) * 2.0 ** -6))


@pytest.mark.parametrize("B,L,H,Hkv,D,R", [(2, 9000, 1, 1, 64, 64), (1, 20000, 3, 1, 40, 20), (5, 2500, 2, 2, 130, 0)])
def test_no_token_is_lost_or_counted_twice(sc, B, L, H, Hkv, D, R):
    # more tokens than the workgroups hold at once, the first and last tokens' gradients far larger than
    # the others', and a bound by the depth of the sums
    print("case qk dw tokens", B, L, H, Hkv, D, R, flush=True)
    rng = np.random.default_rng(L)
    q, qx = draw(rng, (B, L, H, D), "f32", 1.5, 0.2)
    k, kx = draw(rng, (B, L, Hkv, D), "f32", 1.5, 0.2)
    w, wx = draw(rng, (D,), "f32", 0.2, 1.0)
    f = torch.from_numpy((10000.0 ** (-2.0 * np.arange(R // 2) / max(R, 1))).astype(np.float32)).to(DEV)
    pos = np.arange(L)[None].repeat(B, 0)
    size = np.ones((B, L, 1, 1), np.float32)
    for at in (0, 1, L // 2, L - 2, L - 1):
        size[:, at] = 1000.0
    gq, gk = (torch.from_numpy((rng.standard_normal((B, L, n, D)) * size).astype(np.float32)).to(DEV) for n in (H, Hkv))
    _, _, dq, dk = sc.qk_norm_rotary_bwd(gq, gk, q, k, w, w, f, eps=1e-5)
    for got, x, g in ((dq, qx, gq), (dk, kx, gk)):
        (_, want), _ = ref.qk_norm_bwd(f64(g), x, wx, pos, f64(f), False, float(np.float32(1e-5)))
        # a row's share is right to the roundings of its norm, turn and product (D / 2 + 40 at most); a
        # workgroup (of 2048 at least, for q and k together) adds its rows by lanes of at most 64 a
        # row, then 6 times among them and over its waves; the workgroups' sums are added in 64 bits
        rows = B * L * (x.shape[2])
        deep = -(-rows // (2048 // 4)) + 10
        mag = np.abs(f64(g) * x / np.sqrt((x * x).mean(-1, keepdims=True)))
        other = np.abs(f64(g)).max(-1, keepdims=True) * np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True)) if R else mag
        bound = (0.5 * min(D, 64) + 40 + deep) * 2.0 ** -24 * (mag + other).sum((0, 1, 2))
        err = np.abs(f64(got) - want)
        assert np.all(err <= bound), (err / bound).max()
        # what one large token adds is far past the bound
        one = (ref.qk_norm_bwd(f64(g)[:, -1:], x[:, -1:], wx, pos[:, -1:], f64(f), False, 1e-5)[0][1])
        assert np.median(np.abs(one) / bound) > 20
