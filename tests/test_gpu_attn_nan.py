"""causal_attention on rows of NaN, with the keys in one part and split over workgroups."""
import numpy as np
import pytest
import torch

from tests.layer_util import DEV, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq", [1, 40])
@pytest.mark.parametrize("Lk", [100, 4000])
def test_a_row_of_nan_is_nan_and_alone(sc, dtype, Lq, Lk):
    # lse is -infinity only where a row sees nothing
    print("case attn nan", dtype, Lq, Lk, flush=True)
    rng = np.random.default_rng(7)
    k, _ = draw(rng, (1, Lk, 1, 64), dtype)
    v, _ = draw(rng, (1, Lk, 1, 64), dtype)
    q, _ = draw(rng, (1, Lq, 2, 64), dtype)
    want, wl = sc.causal_attention(q, k, v, lse=True)
    q[0, Lq - 1, 1, 9] = float("nan")
    o, lse = sc.causal_attention(q, k, v, lse=True)
    assert torch.isnan(lse[0, 1, Lq - 1]) and torch.isnan(o[0, Lq - 1, 1]).all()
    o[0, Lq - 1, 1], lse[0, 1, Lq - 1] = want[0, Lq - 1, 1], wl[0, 1, Lq - 1]
    assert torch.equal(o, want) and torch.equal(lse, wl)
    # a key of NaN: every row that sees it
    k[0, 70, 0, 3] = float("nan")
    o, lse = sc.causal_attention(q, k, v, lse=True)
    sees = torch.arange(Lk - Lq, Lk, device=DEV) >= 70
    assert torch.isnan(lse[0, :, sees]).all() and torch.isnan(o[0, sees]).all()
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = sc.causal_attention(q, k, v, kv_len=n, lse=True)
    assert torch.isneginf(lse).all() and o.eq(0).all()
