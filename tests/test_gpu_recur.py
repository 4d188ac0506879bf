"""The gated recurrence on the GPU against the float64 reference, both directions.

Lengths around the single-thread walk, the tile (256 or 128 tokens) and the cut into segments;
channel counts that end inside a vector and a channel group; strided and unaligned rows;
saturated gates; states in and out, the decoding loop's state in place."""
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


def both(sc, B, L, C, dtype, state, zadd=1.0, zmul=1.5, seed=0):
    rng = np.random.default_rng([B, L, C, seed])
    z, zr = draw(rng, (B, L, C), dtype, zmul, zadd)
    u, ur = draw(rng, (B, L, C), dtype)
    dh, dhr = draw(rng, (B, L, C), dtype)
    h0 = dhT = None
    h0r = dhTr = np.zeros((B, C))
    if state:
        h0, h0r = draw(rng, (B, C), "f32")
        dhT, dhTr = draw(rng, (B, C), "f32")
    h, hT = sc.gated_recurrence(z, u, h0)
    (hr, hTr), (bh, bT) = ref.recurrence(zr, ur, h0r)
    check(h, hr, bh, dtype, "h")
    check(hT, hTr, bT, "f32", "hT")
    got = sc.gated_recurrence_bwd(dh, z, u, h, h0, dhT)
    want, bound = ref.recurrence_bwd(dhr, zr, ur, f64(h), h0r, dhTr)
    for g, r, b, n, d in zip(got, want, bound, ("dz", "du", "dh0"), (dtype, dtype, "f32")):
        check(g, r, b, d, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,C", [(1, 1, 1), (3, 1, 40), (2, 2, 33), (2, 16, 64), (2, 17, 64),
                                   (1, 100, 7), (2, 255, 31), (1, 257, 96), (3, 700, 100),
                                   (1, 2048, 32), (1, 2049, 40), (2, 5000, 36)])
def test_both_directions(sc, dtype, B, L, C):
    print("case recur %s B=%d L=%d C=%d" % (dtype, B, L, C), flush=True)
    both(sc, B, L, C, dtype, state=(L % 2 == 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("zadd,zmul", [(9.0, 0.5), (-9.0, 0.5), (0.0, 60.0)])
def test_saturated_gates(sc, dtype, zadd, zmul):
    # memories of thousands of tokens, none at all, and gates that jump between the two
    print("case recur saturated %s %g %g" % (dtype, zadd, zmul), flush=True)
    both(sc, 1, 3000, 40, dtype, True, zadd, zmul)


@pytest.mark.parametrize("L", [12, 600])
def test_infinite_gates(sc, L):
    # z = +inf keeps the state, z = -inf replaces it
    z = torch.zeros(1, L, 8, device=DEV)
    z[:, :, 0], z[:, :, 1] = float("inf"), -float("inf")
    u, h0 = torch.randn(1, L, 8, device=DEV), torch.randn(1, 8, device=DEV)
    h, hT = sc.gated_recurrence(z, u, h0)
    assert torch.equal(h[0, :, 0], h0[0, 0].expand(L)) and torch.equal(h[0, :, 1], u[0, :, 1])
    assert torch.isfinite(h).all() and torch.equal(hT[0, :2], h[0, -1, :2])
    grads = sc.gated_recurrence_bwd(torch.ones_like(z), z, u, h, h0)
    assert all(torch.isfinite(g).all() for g in grads)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [5, 400, 4000])
@pytest.mark.parametrize("offset", [0, 3])
def test_columns_of_a_projection(sc, dtype, L, offset):
    # z and u the halves of one projection, gradients into the halves of another; offset 3 is
    # unaligned
    print("case recur columns %s L=%d offset=%d" % (dtype, L, offset), flush=True)
    C = 48
    rng = np.random.default_rng([L, offset])
    zu, zur = draw(rng, (2, L, 2 * C + offset), dtype)
    z, u = zu[..., offset:offset + C], zu[..., offset + C:]
    zr, ur = zur[..., offset:offset + C], zur[..., offset + C:]
    dh, dhr = draw(rng, (2, L, C), dtype)
    h, hT = sc.gated_recurrence(z, u)
    zero = np.zeros((2, C))
    (hr, hTr), (bh, bT) = ref.recurrence(zr, ur, zero)
    check(h, hr, bh, dtype, "h")
    check(hT, hTr, bT, "f32", "hT")
    g = torch.full_like(zu, 7.0)
    dz, du, _ = sc.gated_recurrence_bwd(dh, z, u, h, dz=g[..., offset:offset + C], du=g[..., offset + C:])
    want, bound = ref.recurrence_bwd(dhr, zr, ur, f64(h), zero, zero)
    check(dz, want[0], bound[0], dtype, "dz")
    check(du, want[1], bound[1], dtype, "du")
    assert (g[..., :offset] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_equal_the_sequence(sc, dtype):
    # a decoding loop with its state in place, in steps of 1 and of 20 tokens
    rng = np.random.default_rng(11)
    z, zr = draw(rng, (3, 60, 72), dtype, 1.0, 1.0)
    u, ur = draw(rng, (3, 60, 72), dtype)
    h0, h0r = draw(rng, (3, 72), "f32")
    (hr, hTr), (bh, bT) = ref.recurrence(zr, ur, h0r)
    for step in (1, 20):
        state = h0.clone()
        parts = []
        for t in range(0, 60, step):
            h, out = sc.gated_recurrence(z[:, t:t + step].contiguous(), u[:, t:t + step].contiguous(),
                                         state, hT=state)
            assert out is state
            parts.append(h)
        check(torch.cat(parts, 1), hr, bh, dtype, "steps of %d" % step)
        check(state, hTr, bT, "f32", "state after steps of %d" % step)


def test_segments_repeat_and_take_a_workspace(sc):
    B, L, C = 1, 9000, 64
    n = sc.sc_recur_workspace_bytes(sc.KIND_F32, B, L, C)
    assert n > 0, "a shape that is cut into segments"
    z, u = torch.randn(B, L, C, device=DEV) + 1, torch.randn(B, L, C, device=DEV)
    state = torch.randn(B, C, device=DEV)
    a = sc.gated_recurrence(z, u, state)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    b = sc.gated_recurrence(z, u, state, workspace=ws)
    keep = state.clone()
    c = sc.gated_recurrence(z, u, state, hT=state)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    with pytest.raises(sc.SpecConvError):
        sc.gated_recurrence(z, u, keep, workspace=ws[:n - 256])


def test_empty(sc):
    z = torch.empty(2, 0, 24, device=DEV)
    s = torch.randn(2, 24, device=DEV)
    h, hT = sc.gated_recurrence(z, z, s)
    assert h.shape == z.shape and torch.equal(hT, s)
    assert not sc.gated_recurrence(z, z)[1].any()
    assert torch.equal(sc.gated_recurrence_bwd(z, z, z, z, s, s)[2], s)
    e = torch.empty(0, 5, 24, device=DEV)
    assert sc.gated_recurrence(e, e)[0].shape == e.shape
