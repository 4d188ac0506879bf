"""Which layouts of dq, dk and dv the attention backward accepts, without a GPU: outputs that share
an element are refused, outputs cut from one array so that they share none are not.

A call whose workspace is a byte short is refused for that (SC_ERR_WORKSPACE) after every other
check and before anything is launched."""
import ctypes
import itertools

import numpy as np
import pytest

# fake, never dereferenced, far enough apart not to overlap
P = [0x10000000000 * (i + 1) for i in range(12)]
D = 8


@pytest.fixture(scope="module")
def sc():
    from tests.test_abi import LIB
    import os
    assert os.path.exists(LIB), "libspecconv.so is not built"
    import fft_causal_long_amd as m
    return m


def accepted(sc, B, L, H, Hkv, grads, kind=0):
    """grads: (first element, (batch, token, head) strides) of dq, dk, dv in one float32 array."""
    a = sc.sc_attn(B, L, L, H, Hkv, D)
    for n in ("q", "o", "dout"):
        getattr(a, n)[:] = [L * H * D, H * D, D]
    for n in ("k", "v"):
        getattr(a, n)[:] = [L * Hkv * D, Hkv * D, D]
    for n, (_, s) in zip(("dq", "dk", "dv"), grads):
        getattr(a, n)[:] = s
    a.scale = 0.125
    need = sc.sc_attn_workspace_bytes(kind, a, 1)
    assert need > 0
    st = sc.sc_causal_attn_bwd(kind, a, P[0], P[1], P[2], P[3], P[4], P[5], *(P[6] + 4 * g[0] for g in grads),
                               P[9], need - 1, None)
    assert st in (sc.SC_ERR_WORKSPACE, sc.SC_ERR_INVALID_ARGUMENT)
    return st == sc.SC_ERR_WORKSPACE


def elements(first, s, n):
    i = [np.arange(k) * t for k, t in zip(n, s)]
    return set((first + i[0][:, None, None, None] + i[1][:, None, None] + i[2][:, None] + np.arange(D)).ravel().tolist())


def disjoint(sets):
    return len(set.union(*sets)) == sum(len(x) for x in sets)


def packed(order, size):
    """Strides (b, l, h, x) of a contiguous array of axes in this order, D values innermost."""
    s, at = [0] * 4, D
    for ax in reversed(order):
        s[ax] = at
        at *= size[ax]
    return s


@pytest.mark.parametrize("order", list(itertools.permutations(range(4))))
def test_thirds_of_one_array(sc, order):
    # dq, dk, dv at x = 0, 1, 2 of an array of axes b, l, h, x in any order
    for B, L, H in ((2, 5, 3), (1, 4, 2), (3, 1, 2), (2, 6, 1), (1, 1, 4)):
        s = packed(order, (B, L, H, 3))
        assert accepted(sc, B, L, H, H, [(x * s[3], s[:3]) for x in range(3)]), (B, L, H)
        # one of them a row too far, over its neighbour
        for axis, n in ((0, B), (1, L), (2, H)):
            if n > 1 and s[axis] < s[3]:
                assert not accepted(sc, B, L, H, H, [(0, s[:3]), (s[3], s[:3]), (2 * s[3] - s[axis], s[:3])])


@pytest.mark.parametrize("order", list(itertools.permutations(range(4))))
def test_boxes_of_one_array(sc, order):
    # boxes of an array, wherever they lie: accepted exactly if they share no element
    r = np.random.default_rng(list(order))
    seen = set()
    for _ in range(300):
        size = r.integers(1, 6, 4)
        B, L, H = (int(r.integers(1, k + 1)) for k in size[:3])
        Hkv = int(r.choice([h for h in range(1, H + 1) if H % h == 0]))
        s = [int(t) for t in packed(order, size)]
        grads, sets = [], []
        for h in (H, Hkv, Hkv):
            n = (B, L, h)
            first = sum(int(r.integers(0, k - m + 1)) * t for k, m, t in zip(size, n + (1,), s))
            grads.append((first, s[:3]))
            sets.append(elements(first, s, n))
        apart = disjoint(sets)
        seen.add(apart)
        assert accepted(sc, B, L, H, Hkv, grads) == apart, (size, B, L, H, Hkv, grads)
    assert seen == {True, False}


def test_no_shared_element_is_accepted(sc):
    # strides of any kind: whatever is accepted shares nothing
    r = np.random.default_rng(3)
    count = 0
    for _ in range(4000):
        B, L, H = (int(r.integers(1, 4)) for _ in range(3))
        grads, sets = [], []
        for _ in range(3):
            s = [4 * int(r.integers(0, 40)) for _ in range(3)]
            first = 4 * int(r.integers(0, 120))
            grads.append((first, s))
            sets.append(elements(first, s, (B, L, H)))
        if accepted(sc, B, L, H, H, grads):
            count += 1
            assert disjoint(sets), (B, L, H, grads)
    assert count > 20
