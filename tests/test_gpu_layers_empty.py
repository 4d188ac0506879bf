"""Layer calls whose inputs are empty along an axis that some output does not have: every output
is written, or the call is refused."""
import pytest
import torch

from tests.layer_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Lq,Lk,D", [(5, 7, 64), (5, 300, 128), (0, 33, 40)])
def test_no_query_heads(sc, dtype, Lq, Lk, D):
    # no head reads the key heads: their gradients are 0, whatever the memory and the keys held
    print("case attn backward without query heads %s Lq=%d Lk=%d D=%d" % (dtype, Lq, Lk, D), flush=True)
    q = torch.empty(2, Lq, 0, D, dtype=dtype, device=DEV)
    lse = torch.empty(2, 0, Lq, device=DEV)
    k, v = (torch.full((2, Lk, 3, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    doc = torch.zeros(2, Lk, dtype=torch.int32, device=DEV)
    for opt in ({}, dict(window=3, cap=5.0, doc_start=doc, slopes=torch.empty(0, device=DEV))):
        dk, dv = (torch.full_like(k, 7.0) for _ in range(2))
        dq, a, b = sc.causal_attention_bwd(q, q, k, v, q, lse, dk=dk, dv=dv, **opt)
        assert dq.shape == q.shape and a is dk and b is dv
        assert not dk.any() and not dv.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_statistics_of_rows_without_values(sc, dtype):
    # a mean over no values is 0 / 0
    print("case layernorm C=0 %s" % dtype, flush=True)
    x = torch.empty(3, 5, 0, dtype=dtype, device=DEV)
    y, mean, rstd = sc.layer_norm(x, stats=True)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 5)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_heads_without_values(sc, dtype):
    # heads of no values: an empty result, but no log-sum is made up for them
    print("case attn D=0 %s" % dtype, flush=True)
    q = torch.empty(2, 5, 3, 0, dtype=dtype, device=DEV)
    assert sc.causal_attention(q, q, q).shape == q.shape
    with pytest.raises(sc.SpecConvError) as e:
        sc.causal_attention(q, q, q, lse=True)
    assert e.value.status == sc.SC_ERR_UNSUPPORTED
    o, lse = sc.causal_attention(q[:0], q[:0], q[:0], lse=True)     # nothing to make up
    assert o.shape == (0, 5, 3, 0) and lse.shape == (0, 3, 5)
    g = sc.causal_attention_bwd(q, q, q, q, q, torch.empty(2, 3, 5, device=DEV))
    assert all(t.shape == q.shape for t in g)
