"""The 8-bit cache: what is written and read back, bit for bit against the float64 model."""
import numpy as np
import pytest
import torch

from oracle import heads as ref
from tests.layer_util import DEV, DTYPES, draw, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


def same(sc, c, m, L, lens, dtype="f32"):
    k, v = sc.cache_read(c, L, lengths(*lens), DTYPES[dtype])
    kr, vr, _ = m.read(L, lens)
    for got, want, n in ((k, kr, "k"), (v, vr, "v")):
        got = f64(got)
        bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
        assert not bad.any(), (n, lens, int(bad.sum()), np.argwhere(bad)[0], got[bad][:3], want[bad][:3])


def scales(c, m):
    """Scales of blocks that hold something."""
    for s, t in ((c.k_scale, 0), (c.v_scale, 1)):
        got = f64(s)
        used = (m.codes[t] != 0).any((1, 3))
        assert np.array_equal(got[used], 2.0 ** m.exps[t][used])


def fill(c, byte):
    c.k.fill_(byte)
    c.v.fill_(byte)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128])
def test_appends_of_every_length(sc, code, dtype, D):
    print("case cache appends", code, dtype, D, flush=True)
    rng = np.random.default_rng(D)
    B, N, H = 3, 4, 2
    table = rng.permutation(B * N + 2)[:B * N].reshape(B, N).astype(np.int32)
    c = sc.KVCache(B, N * 64 - 5, H, D, code, device=DEV, blocks=B * N + 2, table=torch.from_numpy(table).to(DEV))
    assert c.N == N
    fill(c, 0xff)
    m = ref.Cache(B, N, B * N + 2, H, D, code, table)
    lens = np.array([0, 0, 0])
    # magnitudes that grow, so that the older tokens of a block are rounded again, and shrink
    for step, (L, mul) in enumerate([(1, 1.0), (1, 3.0), (17, 0.5), (2, 70.0), (64, 1.0), (3, 2.0), (65, 1000.0), (70, 1e-3)]):
        k, kx = draw(rng, (B, L, H, D), dtype, mul)
        v, vx = draw(rng, (B, L, H, D), dtype, mul * 0.1)
        lens = lens + L - np.array([0, min(L, step % 2), min(L, 2 * (step % 2))])   # rows that drop their first new tokens
        sc.cache_write(c, k, v, lengths(*lens))
        m.write(kx, vx, lens)
        same(sc, c, m, int(lens.max()) + 3, lens, dtype)
        same(sc, c, m, 7, lens, "f32")
        scales(c, m)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_every_value_a_code_stands_for(sc, code):
    # all codes come back as they are, and halfway values go to the even one
    print("case cache codes", code, flush=True)
    if code == "int8":
        top, x = 127.0, np.concatenate([np.arange(-127, 128), np.arange(-127, 127) + 0.5])
    else:
        v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        v = np.unique(v[np.isfinite(v)])
        top, x = 448.0, np.concatenate([v, (v[1:] + v[:-1]) / 2, v * 1.0001])
    x = np.concatenate([x, np.zeros(-len(x) % 64)]).reshape(1, -1, 1, 16)
    x[0, ::64, 0, 0] = top
    for e in (-60, -3, 0, 60):
        L = x.shape[1]
        c = sc.KVCache(1, L, 1, 16, code, device=DEV)
        t = torch.from_numpy((x * 2.0 ** e).astype(np.float32)).to(DEV)
        m = ref.Cache(1, c.N, c.N, 1, 16, code)
        sc.cache_write(c, t, -t, lengths(L))
        m.write(f64(t), -f64(t), [L])
        same(sc, c, m, L, [L])
        scales(c, m)   # (448.04 of e4m3 takes the next scale)


def test_grown_scales_of_every_code(sc):
    # older codes of every value rounded again at scales 2^1 .. 2^12 larger
    print("case cache growth", flush=True)
    for code, top in (("int8", 127.0), ("e4m3", 448.0)):
        v = np.arange(-127, 128.0) if code == "int8" else np.unique(
            ref.e4m3(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()[:127]))
        v = np.resize(v, (1, 20, 1, 16)).copy()
        v[0, 0, 0, 0] = top
        for up in range(1, 13):
            c = sc.KVCache(1, 64, 1, 16, code, device=DEV)
            m = ref.Cache(1, 1, 1, 1, 16, code)
            for x, n in ((v, 20), (np.full((1, 1, 1, 16), top * 2.0 ** up), 21), (np.ones((1, 9, 1, 16)), 30)):
                t = torch.from_numpy(x.astype(np.float32)).to(DEV)
                sc.cache_write(c, t, t, lengths(n))
                m.write(x, x, [n])
            same(sc, c, m, 30, [30])


def test_extreme_values(sc):
    print("case cache extremes", flush=True)
    nan, inf = float("nan"), float("inf")
    for code in ("int8", "e4m3"):
        for dtype in ("f32", "bf16"):
            x = np.zeros((1, 70, 2, 32))
            x[0, 0, 0, :4] = [nan, inf, -inf, 3.0]
            x[0, 1, 1] = inf                        # a head of a block without a finite value but zeros
            x[0, 65, 0] = nan
            x[0, 66, 0, 0] = 1e38                   # past the largest scale
            x[0, 66, 1, :2] = [1e-40, 1e-30]        # below the smallest
            t = torch.from_numpy(x.astype(np.float32)).to(DEV, DTYPES[dtype])
            c = sc.KVCache(1, 128, 2, 32, code, device=DEV)
            m = ref.Cache(1, 2, 2, 2, 32, code)
            sc.cache_write(c, t, t, lengths(70))
            m.write(f64(t), f64(t), [70])
            same(sc, c, m, 70, [70])


def test_positions_that_do_not_exist(sc):
    # before the first token, past the capacity, in blocks that are none: not written, read as 0
    print("case cache edges", flush=True)
    rng = np.random.default_rng(8)
    B, N, H, D = 6, 2, 1, 64
    big = 2**31 - 1
    table = np.array([[0, 1], [2, 99], [-1, 3], [4, 5], [6, 7], [8, 9]], np.int32)
    c = sc.KVCache(B, N * 64, H, D, "e4m3", device=DEV, blocks=12, table=torch.from_numpy(table).to(DEV))
    fill(c, 0x31)
    m = ref.Cache(B, N, 12, H, D, "e4m3", table)
    k, kx = draw(rng, (B, 100, H, D), "f32")
    v, vx = draw(rng, (B, 100, H, D), "f32")
    lens = [40, 100, 128, 150, -7, 0]
    sc.cache_write(c, k, v, lengths(*lens))
    m.write(kx, vx, lens)
    lens = [40, 100, 128, 128, 0, 0]
    same(sc, c, m, 130, lens)
    assert c.k[10:].eq(0x31).all() and c.k[8:10].eq(0x31).all() and c.k[6:8].eq(0x31).all()   # blocks of no token
    for lens in ([200, 150, 129, 228, -100, -(2**31)], [big, big - 50, big, 300, 229, 128]):
        got = sc.cache_read(c, 100, lengths(*lens), torch.float32)
        want = m.read(100, lens)
        # positions that were written, or do not exist (the others hold what the memory held)
        at = np.array(lens, np.int64)[:, None] - 100 + np.arange(100)
        held = np.array([[0, 40], [0, 100], [64, 128], [50, 128], [0, 0], [0, 0]])
        known = ((at >= held[:, :1]) & (at < held[:, 1:])) | (at < 0) | (at >= 128)
        assert known.any(1).sum() >= 4
        for g, w in zip(got, want):
            assert np.array_equal(f64(g)[known], w[known]), lens
    before = c.k.clone(), c.v.clone(), c.k_scale.clone()
    sc.cache_write(c, k, v, lengths(0, -3, big, 300, -(2**31), big - 7))     # nothing of it exists
    assert torch.equal(before[0], c.k) and torch.equal(before[1], c.v) and torch.equal(before[2], c.k_scale)


def test_strided_tokens_and_results(sc):
    print("case cache strides", flush=True)
    rng = np.random.default_rng(9)
    p, px = draw(rng, (2, 90, 7, 64), "bf16")
    c = sc.KVCache(2, 128, 2, 64, device=DEV)
    m = ref.Cache(2, 2, 4, 2, 64, "int8")
    sc.cache_write(c, p[:, :, 3:5], p[:, :, 5:], lengths(90, 77))
    m.write(px[:, :, 3:5], px[:, :, 5:], [90, 77])
    out = torch.full((2, 95, 6, 64), 7.0, device=DEV)
    k, v = sc.cache_read(c, 95, lengths(90, 77), torch.float32, k=out[:, :, 1:3], v=out[:, :, 3:5])
    kr, vr, _ = m.read(95, [90, 77])
    assert np.array_equal(f64(out[:, :, 1:3]), kr) and np.array_equal(f64(v), vr)
    assert out[:, :, 0].eq(7).all() and out[:, :, 5].eq(7).all()
    for bad in (dict(k=out[:, :, :2], v=out[:, :, 1:3]),):
        with pytest.raises(sc.SpecConvError):
            sc.cache_read(c, 95, lengths(90, 77), torch.float32, **bad)
    with pytest.raises(ValueError):
        sc.cache_read(c, 94, lengths(90, 77), torch.float32, k=out[:, :, :2], v=out[:, :, 2:4])
    with pytest.raises(ValueError):
        sc.cache_write(c, p[:, :, :3], p[:, :, 3:6], lengths(90, 77))
    with pytest.raises(ValueError):
        sc.cache_write(c, p[:, :, :2], p[:, :, 2:4], torch.tensor([90, 77], device=DEV))


def test_shared_blocks_are_read_by_all(sc):
    # two sequences with one prefix: its blocks written once, their own blocks after it
    print("case cache shared", flush=True)
    rng = np.random.default_rng(10)
    table = np.array([[0, 1], [0, 2]], np.int32)
    c = sc.KVCache(2, 128, 1, 32, device=DEV, blocks=3, table=torch.from_numpy(table).to(DEV))
    m = ref.Cache(2, 2, 3, 1, 32, "int8", table)
    k, kx = draw(rng, (2, 64, 1, 32), "f32")
    sc.cache_write(c, k, k, lengths(64, 0))
    m.write(kx, kx, [64, 0])
    k, kx = draw(rng, (2, 9, 1, 32), "f32")
    sc.cache_write(c, k, k, lengths(73, 73))
    m.write(kx, kx, [73, 73])
    same(sc, c, m, 73, [73, 73])
