"""Layer norm on the GPU against the float64 reference (oracle/layers.py), both directions.

Rows that fit 16, 64 and 256 threads and rows that do not fit the registers, each with lengths
that end inside a vector; strided and unaligned rows; tolerances are the reference's roundings
term by term."""
import numpy as np
import pytest
import torch

from oracle import layers as ref
from tests.layer_util import DEV, check, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


SHAPES = [(1, 1), (3, 2), (5, 8), (70, 64), (33, 65), (9, 129), (40, 257), (17, 768), (6, 1000),
          (21, 1024), (4, 1025), (5, 2049), (3, 4104), (3, 8192), (2, 8193), (2, 16390), (3, 20001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_both_directions(sc, dtype, rows, C):
    print("case layernorm %s rows=%d C=%d" % (dtype, rows, C), flush=True)
    rng = np.random.default_rng([rows, C])
    x, xr = draw(rng, (rows, C), dtype, 1.5, 0.4)
    w, wr = draw(rng, (C,), dtype, 0.3, 1.0)
    b, br = draw(rng, (C,), dtype, 0.3)
    dy, dyr = draw(rng, (rows, C), dtype)
    y, mean, rstd = sc.layer_norm(x, w, b, 1e-5, stats=True)
    (yr, mr, rr), (by, bm, brs) = ref.layernorm(xr, wr, br, 1e-5)
    check(y, yr, by, dtype, "y")
    check(mean, mr, bm, "f32", "mean")
    check(rstd, rr, brs, "f32", "rstd")
    dx, dw, db = sc.layer_norm_bwd(dy, x, mean, rstd, w)
    (dxr, dwr, dbr), (bx, bw, bb) = ref.layernorm_bwd(dyr, xr, wr, f64(mean), f64(rstd))
    check(dx, dxr, bx, dtype, "dx")
    check(dw, dwr, bw, dtype, "dw")
    check(db, dbr, bb, dtype, "db")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset,C,wide", [(0, 96, 256), (8, 96, 256), (3, 96, 200), (1, 700, 1501)])
def test_columns_of_a_wider_array(sc, dtype, offset, C, wide):
    # aligned and unaligned column blocks, input and output interleaved in one array
    print("case layernorm columns %s" % ((dtype, offset, C, wide),), flush=True)
    rng = np.random.default_rng([offset, C, wide])
    full, fr = draw(rng, (2, 19, wide), dtype)
    x = full[..., offset:offset + C]
    out = full[..., wide - C:] if offset + C <= wide - C else None
    y, mean, rstd = sc.layer_norm(x, None, None, 1e-6, out=out, stats=True)
    xr = fr[..., offset:offset + C].reshape(-1, C)
    one, zero = np.ones(C), np.zeros(C)
    (yr, mr, _), (by, bm, _) = ref.layernorm(xr, one, zero, 1e-6)
    check(y.reshape(-1, C), yr, by, dtype, "y")
    assert np.array_equal(f64(full[..., :offset]), fr[..., :offset]), "columns beside x are untouched"
    dy, dyr = draw(rng, (2, 19, C), dtype)
    dx, dw, db = sc.layer_norm_bwd(dy, x.contiguous() if out is not None else x, mean, rstd)
    (dxr, dwr, dbr), (bx, bw, bb) = ref.layernorm_bwd(dyr.reshape(-1, C), f64(x).reshape(-1, C), one,
                                                      f64(mean).ravel(), f64(rstd).ravel())
    check(dx.reshape(-1, C), dxr, bx, dtype, "dx")
    check(dw, dwr, bw, dtype, "dw")
    check(db, dbr, bb, dtype, "db")


def test_many_rows_repeat_bit_for_bit(sc):
    rng = np.random.default_rng(5)
    x, xr = draw(rng, (5000, 200), "f32")
    dy, dyr = draw(rng, (5000, 200), "f32")
    w, wr = draw(rng, (200,), "f32")
    _, mean, rstd = sc.layer_norm(x, w, None, stats=True)
    first = sc.layer_norm_bwd(dy, x, mean, rstd, w)
    again = sc.layer_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    want, bound = ref.layernorm_bwd(dyr, xr, wr, f64(mean), f64(rstd))
    for g, r, b, n in zip(first, want, bound, ("dx", "dw", "db")):
        check(g, r, b, "f32", n)


def test_rows_apart(sc):
    # a row of NaN or infinity stays its own; a constant row has y = bias
    x = torch.randn(6, 300, device=DEV)
    one = torch.ones(300, device=DEV)
    ref_y = sc.layer_norm(x, None, one)
    x[1] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 2.5
    y = sc.layer_norm(x, None, one)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).any()
    assert torch.equal(y[4], one)
    for r in (0, 2, 5):
        assert torch.equal(y[r], ref_y[r])


def test_large_offset_keeps_the_variance(sc):
    # values far from 0: the sum about the mean keeps what a sum of squares would lose
    rng = np.random.default_rng(3)
    x, xr = draw(rng, (4, 777), "f32", 1.0, 3000.0)
    y, mean, rstd = sc.layer_norm(x, stats=True)
    want, bound = ref.layernorm(xr, np.ones(777), np.zeros(777), 1e-5)
    for g, r, b, n in zip((y, mean, rstd), want, bound, ("y", "mean", "rstd")):
        check(g, r, b, "f32", n)


def test_empty(sc):
    e = torch.empty(0, 40, device=DEV)
    s = torch.empty(0, device=DEV)
    assert sc.layer_norm(e).shape == (0, 40)
    dx, dw, db = sc.layer_norm_bwd(e, e, s, s)
    assert dx.shape == (0, 40) and not dw.any() and not db.any() and dw.shape == (40,)
    dx, dw, db = sc.layer_norm_bwd(e, e, s, s, params=False)
    assert dw is None and db is None


def test_workspace_and_stream(sc):
    rng = np.random.default_rng(9)
    x, xr = draw(rng, (300, 513), "bf16")
    dy, dyr = draw(rng, (300, 513), "bf16")
    n = sc.sc_layernorm_bwd_workspace_bytes(sc.KIND_BF16, 300, 513)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        _, mean, rstd = sc.layer_norm(x, stats=True)
        a = sc.layer_norm_bwd(dy, x, mean, rstd, workspace=ws)
    side.synchronize()
    b = sc.layer_norm_bwd(dy, x, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(sc.SpecConvError):
        sc.layer_norm_bwd(dy, x, mean, rstd, workspace=ws[:n - 256])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(9001, 64), (8300, 61), (2500, 768), (2051, 1001), (700, 5000), (530, 4099),
                                    (150, 16384)])
def test_more_rows_than_workgroups(sc, dtype, rows, C):
    # backward workgroups that take several rows, and their shares of dw and db
    test_both_directions(sc, dtype, rows, C)
