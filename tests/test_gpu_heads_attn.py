"""Attention over the 8-bit cache against the float64 reference on the values the cache holds."""
import numpy as np
import pytest
import torch

from oracle import heads as ref
from tests.layer_util import DEV, DTYPES, check, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


def filled(sc, rng, B, T, Hkv, D, code, lens, table=None, blocks=None, mul=1.0, dtype="f32"):
    """A cache with lens[b] tokens a row, its stale bytes all ones (NaN in e4m3), and its values."""
    c = sc.KVCache(B, T, Hkv, D, code, device=DEV, blocks=blocks,
                   table=None if table is None else torch.from_numpy(table).to(DEV))
    c.k.fill_(0xff)
    c.v.fill_(0xff)
    k, _ = draw(rng, (B, T, Hkv, D), dtype, mul)
    v, _ = draw(rng, (B, T, Hkv, D), dtype, 1.0)
    # values of growing size along the sequence, so that the blocks' scales differ
    v *= torch.linspace(0.1, 8.0, T, device=DEV).to(v.dtype)[None, :, None, None]
    sc.cache_write(c, k, v, lengths(*lens))
    cap = c.N * 64
    kx, vx = (f64(t) for t in sc.cache_read(c, cap, lengths(*([cap] * B)), torch.float32))
    live = np.ones((B, cap), bool)
    if table is not None:
        live = ((table >= 0) & (table < c.blocks)).repeat(64, 1)
    return c, kx, vx, live


CASES = [
    # dtype, code, B, T, Lq, H, Hkv, D, window, sinks, cap, bias, lens, paged
    ("f32", "int8", 2, 70, 1, 2, 2, 64, 0, 0, 0.0, False, [70, 33], False),
    ("bf16", "e4m3", 2, 70, 1, 4, 1, 64, 0, 0, 0.0, True, [70, 1], True),
    ("f32", "e4m3", 3, 300, 5, 6, 2, 32, 64, 4, 0.0, True, [300, 0, 3], True),
    ("bf16", "int8", 2, 900, 3, 8, 2, 128, 100, 70, 30.0, False, [900, 555], False),
    ("bf16", "int8", 1, 40, 40, 2, 2, 16, 7, 1, 0.0, False, [40], False),        # several 16-row strips
    ("f32", "int8", 2, 200, 200, 3, 1, 48, 0, 0, 5.0, True, [200, 190], True),
    ("bf16", "e4m3", 1, 513, 513, 4, 2, 64, 128, 3, 0.0, True, [513], False),
    ("bf16", "int8", 2, 700, 130, 8, 1, 80, 65, 64, 0.0, False, [700, 131], True),
    ("f32", "e4m3", 1, 700, 130, 8, 2, 128, 0, 0, 0.0, False, [640], False),
    ("bf16", "e4m3", 1, 1500, 600, 16, 1, 96, 1, 0, 0.0, False, [1500], False),   # a window of the row's own key
    ("bf16", "int8", 8, 400, 300, 64, 64, 16, 0, 0, 0.0, False, [400, 300, 301, 320, 350, 399, 310, 400], False),  # 128-row workgroups
    ("f32", "int8", 8, 400, 300, 64, 64, 16, 50, 10, 0.0, True, [400, 300, 301, 320, 350, 399, 310, 400], True),
    ("bf16", "int8", 1, 20000, 1, 8, 1, 64, 0, 0, 0.0, False, [20000], True),     # keys over workgroups
    ("f32", "e4m3", 1, 20000, 4, 4, 1, 128, 9000, 500, 0.0, True, [19999], False),
    ("bf16", "e4m3", 2, 5000, 33, 4, 1, 64, 0, 0, 20.0, False, [5000, 77], False),   # and of more rows
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:12])))
def test_against_the_reference(sc, case):
    print("case attn8", case, flush=True)
    dtype, code, B, T, Lq, H, Hkv, D, window, sinks, cap, bias, lens, paged = case
    rng = np.random.default_rng(T + Lq + D)
    N = -(-T // 64)
    table = rng.permutation(B * N + 3)[:B * N].reshape(B, N).astype(np.int32) if paged else None
    c, kx, vx, live = filled(sc, rng, B, T, Hkv, D, code, lens, table, B * N + 3 if paged else None)
    q, qx = draw(rng, (B, Lq, H, D), dtype, 1.5)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=DEV) if bias else None
    o, lse = sc.cached_attention(q, c, lengths(*lens), window=window, sinks=sinks, cap=cap, slopes=slopes, lse=True)
    scale = float(np.float32(D ** -0.5))
    (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, lens, scale, window, sinks, float(np.float32(cap)),
                                              None if slopes is None else f64(slopes), live, dtype == "bf16")
    check(o, ro, bo, dtype, "o")
    check(lse, rl, bl, "f32", "lse")
    again = sc.cached_attention(q, c, lengths(*lens), window=window, sinks=sinks, cap=cap, slopes=slopes)
    assert torch.equal(o, again)


def test_rows_that_see_nothing(sc):
    # more queries than tokens, lengths of zero, below and past the cache, blocks that are none
    print("case attn8 empty rows", flush=True)
    rng = np.random.default_rng(2)
    big = 2**31 - 1
    for code in ("int8", "e4m3"):
        for Lq in (1, 3, 90):
            table = np.array([[0, 1], [-1, -5], [2, 99], [3, 4], [5, 6], [7, 8], [9, 10]], np.int32)
            c, kx, vx, live = filled(sc, rng, 7, 128, 2, 64, code, [100, 128, 128, 90, 128, 128, 128], table, 11)
            lens = [100, 128, 128, 2, 0, 128 + Lq // 2, big]
            if Lq == 90:
                lens[5], lens[6] = -3, -(2**31)
            q, qx = draw(rng, (7, Lq, 4, 64), "bf16")
            o, lse = sc.cached_attention(q, c, lengths(*lens), window=50, sinks=2, lse=True)
            (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, lens, 0.125, 50, 2, live=live, bf16=True)
            assert np.isinf(rl).any() and np.isfinite(rl).any()
            check(o, ro, bo, "bf16", "o")
            check(lse, rl, bl, "f32", "lse")


def test_scales_far_apart(sc):
    # a block of values 2^40 times another's with a weight as small: both count
    print("case attn8 scales", flush=True)
    rng = np.random.default_rng(3)
    for dtype in ("f32", "bf16"):
        c = sc.KVCache(1, 192, 1, 64, "int8", device=DEV)
        k, _ = draw(rng, (1, 192, 1, 64), "f32", 0.1)
        v, _ = draw(rng, (1, 192, 1, 64), "f32")
        q, qx = draw(rng, (1, 2, 3, 64), dtype)
        unit = q[0, 0, 0].float() / q[0, 0, 0].float().norm()
        k[0, 64:128, 0] -= unit * 27 * 8 / q[0, 0, 0].float().norm()     # scores about -27 for the first row
        v[0, 64:128] *= 2.0 ** 40
        v[0, 128:] *= 2.0 ** -55
        sc.cache_write(c, k, v, lengths(192))
        kx, vx = (f64(t) for t in sc.cache_read(c, 192, lengths(192), torch.float32))
        o, lse = sc.cached_attention(q, c, lengths(192), lse=True)
        (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, [192], 0.125, bf16=dtype == "bf16")
        check(o, ro, bo, dtype, "o")
        check(lse, rl, bl, "f32", "lse")


def test_query_rows_of_any_size(sc):
    # rows of zeros, rows 2^60 apart, a row of NaN: each is its own
    print("case attn8 query sizes", flush=True)
    rng = np.random.default_rng(4)
    for dtype in ("f32", "bf16"):
        c, kx, vx, live = filled(sc, rng, 1, 130, 1, 64, "e4m3", [130])
        q, qx = draw(rng, (1, 6, 2, 64), dtype)
        mul = torch.tensor([1.0, 0.0, 2.0 ** -60, 30.0, 2.0 ** -100, 1.0], device=DEV)[None, :, None, None].to(q.dtype)
        q = q * mul
        q[0, 5, 1, 9] = float("nan")
        o, lse = sc.cached_attention(q, c, lengths(130), lse=True)
        assert torch.isnan(lse[0, 1, 5]) and torch.isnan(o[0, 5, 1]).all()
        q[0, 5, 1, 9] = 0
        (ro, rl), (bo, bl) = ref.cached_attention(f64(q), kx, vx, [130], 0.125, bf16=dtype == "bf16")
        o[0, 5, 1] = torch.from_numpy(ro[0, 5, 1]).to(DEV, o.dtype)
        lse[0, 1, 5] = float(rl[0, 1, 5])
        check(o, ro, bo, dtype, "o")
        check(lse, rl, bl, "f32", "lse")


def test_strides_workspace_and_refusals(sc):
    print("case attn8 strides", flush=True)
    rng = np.random.default_rng(5)
    c, kx, vx, live = filled(sc, rng, 2, 3000, 1, 64, "int8", [3000, 2000])
    p, px = draw(rng, (2, 2, 6, 64), "bf16")
    n = lengths(3000, 2000)
    q, qx = p[:, :, 1:5], px[:, :, 1:5]
    out = torch.full((2, 2, 9, 64), 3.0, device=DEV, dtype=torch.bfloat16)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    o = sc.cached_attention(q, c, n, out=out[:, :, 2:6], workspace=ws)
    (ro, _), (bo, _) = ref.cached_attention(qx, kx, vx, [3000, 2000], 0.125, bf16=True)
    check(o, ro, bo, "bf16", "o")
    assert out[:, :, :2].eq(3).all() and out[:, :, 6:].eq(3).all()
    with pytest.raises(sc.SpecConvError):
        sc.cached_attention(q, c, n, workspace=ws[:512])
    with pytest.raises(sc.SpecConvError):
        sc.cached_attention(q, c, n, out=q)
    with pytest.raises(sc.SpecConvError):
        sc.cached_attention(q[:, :, :, :64], c, n, scale=0.0)
    for bad in (lambda: sc.cached_attention(q[..., :32], c, n), lambda: sc.cached_attention(q, c, n[:1]),
                lambda: sc.cached_attention(q, c, n.long()), lambda: sc.cached_attention(q[:1], c, n[:1]),
                lambda: sc.cached_attention(q, c, n, slopes=torch.ones(3, device=DEV))):
        with pytest.raises(ValueError):
            bad()


def test_offsets_past_32_bits(sc):
    # blocks at the end of a pool of 5 GB for each of k and v
    print("case attn8 long offsets", flush=True)
    rng = np.random.default_rng(6)
    P = 80000
    table = np.array([[P - 1, 3, P - 2], [P - 3, 70000, 0]], np.int32)
    c = sc.KVCache(2, 192, 8, 128, "int8", device=DEV, blocks=P, table=torch.from_numpy(table).to(DEV))
    assert c.k.numel() > 2**32
    k, _ = draw(rng, (2, 180, 8, 128), "bf16")
    v, _ = draw(rng, (2, 180, 8, 128), "bf16")
    m = ref.Cache(2, 3, 6, 8, 128, "int8")
    sc.cache_write(c, k, v, lengths(180, 170))
    m.write(f64(k), f64(v), [180, 170])
    kx, vx, _ = m.read(192, [192, 192])
    got = sc.cache_read(c, 192, lengths(192, 192), torch.float32)
    for b, n in ((0, 180), (1, 170)):
        assert np.array_equal(f64(got[0])[b, :n], kx[b, :n]) and np.array_equal(f64(got[1])[b, :n], vx[b, :n])
    for Lq in (1, 20):
        q, qx = draw(rng, (2, Lq, 16, 128), "bf16")
        o, lse = sc.cached_attention(q, c, lengths(180, 170), lse=True)
        (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, [180, 170], float(np.float32(128 ** -0.5)), bf16=True)
        check(o, ro, bo, "bf16", "o")
        check(lse, rl, bl, "f32", "lse")


EDGES = [
    # dtype, code, B, T, Lq, H, Hkv, D, window, sinks, lens
    ("bf16", "e4m3", 2, 64, 1, 1, 1, 112, 0, 0, [64, 63]),          # a block to its end
    ("f32", "int8", 2, 128, 64, 1, 1, 16, 64, 0, [128, 64]),        # a window of a block
    ("bf16", "int8", 1, 129, 1, 16, 1, 64, 0, 0, [129]),            # sixteen rows, one token in the last block
    ("bf16", "int8", 1, 129, 17, 1, 1, 64, 3, 200, [128]),          # seventeen; more sinks than tokens
    ("f32", "e4m3", 3, 320, 2, 24, 3, 128, 64, 64, [320, 129, 128]),   # a window that begins where sinks end
    ("bf16", "e4m3", 1, 256, 256, 5, 5, 48, 1, 1, [256]),
    ("bf16", "int8", 40, 100, 1, 4, 2, 32, 10, 2, [100 - 2 * i for i in range(40)]),
]


@pytest.mark.parametrize("case", EDGES, ids=lambda c: "-".join(map(str, c[:10])))
def test_edges_of_blocks_and_windows(sc, case):
    print("case attn8 edges", case, flush=True)
    dtype, code, B, T, Lq, H, Hkv, D, window, sinks, lens = case
    rng = np.random.default_rng(T + Lq)
    c, kx, vx, live = filled(sc, rng, B, T, Hkv, D, code, lens)
    q, qx = draw(rng, (B, Lq, H, D), dtype, 1.5)
    o, lse = sc.cached_attention(q, c, lengths(*lens), window=window, sinks=sinks, scale=0.2, lse=True)
    (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, lens, float(np.float32(0.2)), window, sinks, bf16=dtype == "bf16")
    check(o, ro, bo, dtype, "o")
    check(lse, rl, bl, "f32", "lse")


def test_blocks_of_zeros(sc):
    # a block whose values are all 0 has the smallest scale: its weights count all the same
    print("case attn8 zeros", flush=True)
    for code in ("int8", "e4m3"):
        for dtype in ("f32", "bf16"):
            rng = np.random.default_rng(7)
            c = sc.KVCache(1, 192, 1, 64, code, device=DEV)
            k, _ = draw(rng, (1, 192, 1, 64), "f32")
            v, _ = draw(rng, (1, 192, 1, 64), "f32")
            v[:, :64] = 0
            k[:, 64:128] = 0
            sc.cache_write(c, k, v, lengths(192))
            kx, vx = (f64(t) for t in sc.cache_read(c, 192, lengths(192), torch.float32))
            for Lq, n in ((1, 192), (1, 64), (3, 64), (70, 150)):
                q, qx = draw(rng, (1, Lq, 3, 64), dtype)
                o, lse = sc.cached_attention(q, c, lengths(n), lse=True)
                (ro, rl), (bo, bl) = ref.cached_attention(qx, kx, vx, [n], 0.125, bf16=dtype == "bf16")
                check(o, ro, bo, dtype, "o")
                check(lse, rl, bl, "f32", "lse")


def test_a_table_that_changes(sc):
    # sequences take another's blocks: by new values in the table, and by another tensor
    print("case attn8 tables", flush=True)
    rng = np.random.default_rng(9)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    c = sc.KVCache(2, 128, 2, 64, "int8", device=DEV, blocks=6, table=table)
    k, _ = draw(rng, (2, 100, 2, 64), "bf16")
    sc.cache_write(c, k, k, lengths(100, 90))
    q, _ = draw(rng, (1, 1, 2, 64), "bf16")
    q = q.expand(2, 1, 2, 64).contiguous()
    a = sc.cached_attention(q, c, lengths(100, 90))
    table.copy_(torch.tensor([[2, 3], [0, 1]]))
    b = sc.cached_attention(q, c, lengths(90, 100))
    assert torch.equal(a[0], b[1]) and torch.equal(a[1], b[0])
    c.table = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=DEV)
    d = sc.cached_attention(q, c, lengths(100, 100))
    assert torch.equal(d[0], a[0]) and torch.equal(d[1], a[0])
    c.table = None              # row b's blocks are 2 b, 2 b + 1 again
    assert torch.equal(sc.cached_attention(q, c, lengths(100, 90)), a)
    with pytest.raises(ValueError):
        c.table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
