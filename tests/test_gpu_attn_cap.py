"""Causal attention under caps from far below the scores to far above them: a cap that no score
comes near leaves the scores as they are, to a relative error."""
import pytest
import torch

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
