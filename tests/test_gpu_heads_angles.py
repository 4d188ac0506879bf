"""The rotation's angles at positions up to the ends of int32 and frequencies above one."""
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


@pytest.mark.parametrize("top", [1.0, 1000.0, 1e5])
def test_the_last_positions(sc, top):
    # p inv_freq has up to 55 bits, more than a double; the angles stay under 2^48
    print("case qk last positions", top, flush=True)
    rng = np.random.default_rng(1)
    pos = np.array([[2**31 - 1, -(2**31), 2**30 + 1, -(2**30) - 3, 2**29 + 1, 2**31 - 12345, 7]], np.int32)
    x, xx = draw(rng, (1, 7, 1, 64), "f32")
    g, gx = draw(rng, (1, 7, 1, 64), "f32")
    f = torch.from_numpy((top * 500000.0 ** (-np.arange(32) / 32.0)).astype(np.float32)).to(DEV)
    p = torch.from_numpy(pos).to(DEV)
    eps = float(np.float32(1e-6))
    y, _ = sc.qk_norm_rotary(x, None, None, None, f, positions=p)
    check(y, *ref.qk_norm(xx, np.ones(64), pos, f64(f), False, eps), "f32", "y")
    dx = sc.qk_norm_rotary_bwd(g, None, x, None, None, None, f, positions=p)[0]
    (rx, _), (bx, _) = ref.qk_norm_bwd(gx, xx, np.ones(64), pos, f64(f), False, eps)
    check(dx, rx, bx, "f32", "dx")
