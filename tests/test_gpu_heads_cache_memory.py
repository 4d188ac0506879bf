"""Caches whose sequences are put in another order, and caches copied."""
import copy

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


def test_sequences_in_another_order_and_copies(sc):
    print("case cache memory", flush=True)
    rng = np.random.default_rng(3)
    n = torch.tensor([100, 128, 77], dtype=torch.int32, device=DEV)
    c = sc.KVCache(3, 128, 2, 64, device=DEV)
    k, _ = draw(rng, (3, 128, 2, 64), "bf16")
    v, _ = draw(rng, (3, 128, 2, 64), "bf16")
    q, _ = draw(rng, (3, 1, 4, 64), "bf16")
    sc.cache_write(c, k, v, n)
    o = sc.cached_attention(q, c, n)
    held = sc.cache_read(c, 128, n)
    kept = copy.deepcopy(c)
    order = torch.tensor([2, 0, 1], device=DEV)
    blocks = (2 * order[:, None] + torch.arange(2, device=DEV)).flatten()
    for name in ("k", "v", "k_scale", "v_scale"):
        setattr(c, name, getattr(c, name)[blocks])
    torch.empty(1 << 20, device=DEV).fill_(float("nan"))      # (over what the first memory may have been)
    assert torch.equal(sc.cached_attention(q[order].contiguous(), c, n[order]), o[order])
    assert all(torch.equal(a, b[order]) for a, b in zip(sc.cache_read(c, 128, n[order]), held))
    # a copy's table is its own, over the same memory
    b = copy.copy(c)
    b.table = torch.tensor([[2, 3], [4, 5], [0, 1]], dtype=torch.int32, device=DEV)
    assert torch.equal(sc.cached_attention(q, b, n), o)
    assert torch.equal(sc.cached_attention(q[order].contiguous(), c, n[order]), o[order])
    # the deep copy holds what it held, whatever is written to the first
    c.k.zero_()
    c.v.zero_()
    assert torch.equal(sc.cached_attention(q, kept, n), o)
