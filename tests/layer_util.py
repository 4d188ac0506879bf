"""Helpers of the layer tests: stored values, and the comparison with a bound."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda:0"


def draw(rng, shape, dtype, mul=1.0, add=0.0):
    """A device tensor of N(add, mul^2) values and what it stores, in float64."""
    x = torch.from_numpy(np.asarray(rng.standard_normal(shape) * mul + add, np.float32)).to(DTYPES[dtype])
    return x.to(DEV), x.double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, bound, dtype, what):
    """|got - ref| <= bound, widened by the one rounding to the storage type."""
    got = f64(got)
    assert got.shape == ref.shape, what
    b = bound + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + bound) + 1e-37
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what + ": infinities"
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, ref))
    worst = float(np.max(err / b)) if err.size else 0.0
    at = np.unravel_index(int(np.argmax(err / b)), err.shape) if err.size else ()
    print("%s: worst err/bound %.3g%s" % (what, worst, "" if not err.size else " at %s: got %.9g, want %.9g"
                                          % (tuple(map(int, at)), got[at], ref[at])), flush=True)
    assert not np.isnan(err).any(), what + ": NaN"
    assert np.all(err <= b), "%s: %d of %d outside, worst %.3g" % (what, int((err > b).sum()), err.size, worst)
