"""Causal attention under caps from far below the scores to far above them: a cap that no score
comes near leaves the scores as they are, to a relative error."""
import numpy as np
import pytest
import torch

from tests.layer_util import DEV, DTYPES, check, f64
from tests.test_gpu_attn import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [0.25, 2.0, 20.0, 64.0, 66.0, 1e4, 1e6])
def test_caps(sc, dtype, cap):
    print("case attn cap %s cap=%g" % (dtype, cap), flush=True)
    run(sc, 2, 90, 90, 4, 2, 64, dtype, cap=cap, window=60, qmul=3.0)
    run(sc, 1, 45, 45, 2, 1, 128, dtype, cap=cap, bias=True, qmul=10.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [2.0, 1e4, 1e6])
def test_caps_over_a_cache(sc, dtype, cap):
    print("case attn cap cache %s cap=%g" % (dtype, cap), flush=True)
    run(sc, 2, 1, 1500, 4, 2, 64, dtype, cap=cap, kv_len=[1500, 3], qmul=3.0, bwd=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_smallest_caps(sc, dtype):
    # scale / cap past the largest float32: every score is the cap, with its sign
    print("case attn smallest cap %s" % dtype, flush=True)
    run(sc, 2, 70, 70, 2, 1, 64, dtype, cap=1e-42)
    run(sc, 1, 1, 600, 2, 1, 128, dtype, cap=1e-42, bias=True, bwd=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cap", [1.0, 30.0, 64.0, 1000.0])
def test_lse_of_rows_of_one_key(sc, dtype, cap):
    # lse is float32 whatever the storage: the capped score itself where a row sees one key.  Products
    # of one nonzero value are exact, so its roundings are tanh's 9 units, 2 of its argument, and 5 of
    # the cap, its base and their products (20 allowed).
    print("case attn lse of one key %s cap=%g" % (dtype, cap), flush=True)
    n = 400
    x = torch.logspace(-2, 3.3, n, dtype=torch.float64) * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
    q = torch.zeros(1, n, 1, 64, dtype=DTYPES[dtype], device=DEV)
    q[0, :, 0, 5] = x.to(DTYPES[dtype]).to(DEV)
    k = torch.zeros_like(q)
    k[..., 5] = 1.0
    want = cap * np.tanh(f64(q)[0, :, 0, 5] / 8 / cap)
    for name, (a, b, w) in {"rows": (q, k, 1), "decode": (q.transpose(0, 1), k.transpose(0, 1), 0)}.items():
        _, lse = sc.causal_attention(a.contiguous(), b.contiguous(), b.contiguous(), window=w, cap=cap, lse=True)
        check(lse.reshape(n), want, 20 * 2.0 ** -24 * np.abs(want), "f32", name)
