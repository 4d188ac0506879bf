"""Attention gradients written into the parts of one array, heads outside tokens and inside."""
import pytest
import torch

from tests.layer_util import DEV, DTYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["bxhld", "bhxld", "bhlxd", "xbhld", "blxhd", "lbxhd"])
def test_thirds_of_one_array(sc, dtype, order):
    print("case attn gradients in thirds %s %s" % (dtype, order), flush=True)
    B, L, H, D = 3, 70, 2, 64
    size = dict(b=B, l=L, h=H, x=3, d=D)
    q, k, v, do = (torch.randn(B, L, H, D, device=DEV).to(DTYPES[dtype]) for _ in range(4))
    o, lse = sc.causal_attention(q, k, v, window=40, lse=True)
    plain = sc.causal_attention_bwd(do, q, k, v, o, lse, window=40)
    g = torch.full([size[a] for a in order], 7.0, dtype=q.dtype, device=DEV)
    parts = g.permute([order.index(a) for a in "xblhd"])
    got = sc.causal_attention_bwd(do, q, k, v, o, lse, window=40, dq=parts[0], dk=parts[1], dv=parts[2])
    for a, b in zip(plain, got):
        assert torch.equal(a, b)
    with pytest.raises(sc.SpecConvError):   # dv over dk
        sc.causal_attention_bwd(do, q, k, v, o, lse, window=40, dq=parts[0], dk=parts[1], dv=parts[1])
