"""Layer norm backward with so many columns that a launch of one workgroup for each 32 sums of dw
and db would pass 2^32 threads."""
import numpy as np
import pytest
import torch

from oracle import layers as ref
from tests.layer_util import DEV, check, draw, f64

pytestmark = pytest.mark.gpu


def test_many_columns():
    import fft_causal_long_amd as sc
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    C = 2 ** 26
    print("case layernorm rows=1 C=2^26 bf16", flush=True)
    rng = np.random.default_rng(26)
    x, xr = draw(rng, (1, C), "bf16", 1.5, 0.4)
    dy, dyr = draw(rng, (1, C), "bf16")
    mean, rstd = torch.full((1,), 0.4, device=DEV), torch.full((1,), 0.7, device=DEV)
    dx, dw, db = sc.layer_norm_bwd(dy, x, mean, rstd)
    print("kernels done", flush=True)
    (dxr, dwr, dbr), (bx, bw, bb) = ref.layernorm_bwd(dyr, xr, np.ones(C), f64(mean), f64(rstd))
    # the reference allows sums of 100 additions in a row; a thread here adds C / 256 values of its row
    check(dx, dxr, bx * ((C // 256 + 120) / 120), "bf16", "dx")
    check(dw, dwr, bw, "bf16", "dw")
    check(db, dbr, bb, "bf16", "db")
