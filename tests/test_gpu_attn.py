"""Causal attention on the GPU against the float64 reference: forward, backward, and the form
for new tokens over a cache.

Lengths around the 16, 32, 64 and 128 row and key blocks; windows, documents, padding, ragged
lengths, caps and distance biases; shared key heads; strided tensors; rows that see nothing and
garbage where nothing is seen."""
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


def documents(rng, B, L, mean, pad):
    d = np.zeros((B, L), np.int32)
    for b in range(B):
        at = 0
        while at < L:
            n = int(rng.integers(1, 2 * mean))
            d[b, at:at + n] = at
            at += n
        if pad:
            d[b, L - (b + 1) * pad:] = L + 3
            d[b, 1] = 40   # padding inside the row
    return d


def run(sc, B, Lq, Lk, H, Hkv, D, dtype, window=0, cap=0.0, bias=False, kv_len=None, docs=0, pad=0,
        bwd=True, qmul=1.0, seed=0):
    rng = np.random.default_rng([B, Lq, Lk, H, D, seed])
    q, qr = draw(rng, (B, Lq, H, D), dtype, qmul)
    k, kr = draw(rng, (B, Lk, Hkv, D), dtype)
    v, vr = draw(rng, (B, Lk, Hkv, D), dtype)
    slopes = np.asarray([2.0 ** (-8 * (h + 1) / H) for h in range(H)], np.float32) if bias else None
    doc = documents(rng, B, Lk, docs, pad) if docs else None
    opt = dict(window=window, cap=cap, slopes=slopes, kv_len=kv_len, doc=doc, bf16=dtype == "bf16")
    dev = dict(window=window, cap=cap,
               slopes=None if slopes is None else torch.from_numpy(slopes).to(DEV),
               kv_len=None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device=DEV),
               doc_start=None if doc is None else torch.from_numpy(doc).to(DEV))
    o, lse = sc.causal_attention(q, k, v, lse=True, **dev)
    scale = float(np.float32(D ** -0.5))
    (orf, lr), (bo, bl) = ref.attention(qr, kr, vr, scale, **opt)
    check(o, orf, bo, dtype, "o")
    check(lse, lr, bl, "f32", "lse")
    if not bwd:
        return
    do, dor = draw(rng, (B, Lq, H, D), dtype)
    got = sc.causal_attention_bwd(do, q, k, v, o, lse, **dev)
    want, bound = ref.attention_bwd(dor, qr, kr, vr, f64(o), f64(lse), scale, **opt)
    for g, r, b, n in zip(got, want, bound, ("dq", "dk", "dv")):
        check(g, r, b, dtype, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 130, 300])
def test_lengths(sc, dtype, L):
    print("case attn length %s L=%d" % (dtype, L), flush=True)
    run(sc, 2, L, L, 2, 2, 64, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 24, 40, 64, 72, 96, 128])
def test_head_sizes(sc, dtype, D):
    print("case attn head size %s D=%d" % (dtype, D), flush=True)
    run(sc, 1, 150, 150, 2, 1, D, dtype, window=90, bias=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 100000])
def test_windows(sc, dtype, window):
    print("case attn window %s W=%d" % (dtype, window), flush=True)
    run(sc, 1, 333, 333, 2, 2, 64, dtype, window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (8, 1), (6, 2), (5, 5)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True), (5.0, True)])
def test_shared_heads_caps_and_biases(sc, dtype, H, Hkv, cap, bias):
    print("case attn heads %s H=%d Hkv=%d cap=%g bias=%s" % (dtype, H, Hkv, cap, bias), flush=True)
    run(sc, 2, 90, 90, H, Hkv, 64, dtype, cap=cap, bias=bias, window=70, qmul=3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("docs,pad,window", [(1, 0, 0), (5, 3, 0), (40, 20, 0), (70, 9, 30), (300, 130, 0)])
def test_documents_and_padding(sc, dtype, docs, pad, window):
    print("case attn documents %s %d %d %d" % (dtype, docs, pad, window), flush=True)
    run(sc, 2, 400, 400, 2, 1, 64, dtype, docs=docs, pad=pad, window=window, bias=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 300), (1, 1000), (5, 700), (16, 2000), (40, 129), (7, 3)])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (12, 1)])
def test_new_tokens_over_a_cache(sc, dtype, Lq, Lk, H, Hkv):
    print("case attn cache %s Lq=%d Lk=%d H=%d Hkv=%d" % (dtype, Lq, Lk, H, Hkv), flush=True)
    for kv_len in (None, [Lk, Lk // 2, 0]):
        run(sc, 3, Lq, Lk, H, Hkv, 64, dtype, kv_len=kv_len, bias=True, bwd=Lq < 40)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,docs", [(0, 0), (100, 0), (0, 500)])
def test_decoding_options(sc, dtype, window, docs):
    print("case attn decode %s W=%d docs=%d" % (dtype, window, docs), flush=True)
    for D in (64, 128):
        run(sc, 2, 1, 5000, 4, 2, D, dtype, window=window, docs=docs, cap=8.0, kv_len=[5000, 3333], bwd=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_garbage_where_nothing_is_seen(sc, dtype):
    # keys at the sequence's end and beyond, and padding tokens, may hold NaN in q, k, v and dout
    print("case attn garbage %s" % dtype, flush=True)
    rng = np.random.default_rng(21)
    B, L, H, D = 2, 200, 2, 64
    doc = documents(rng, B, L, 60, 11)
    n = np.array([200, 150], np.int32)
    pad = (doc > np.arange(L)) | (np.arange(L) >= n[:, None])
    q, _ = draw(rng, (B, L, H, D), dtype)
    k, _ = draw(rng, (B, L, H, D), dtype)
    v, _ = draw(rng, (B, L, H, D), dtype)
    do, _ = draw(rng, (B, L, H, D), dtype)
    dev = dict(kv_len=torch.from_numpy(n).to(DEV), doc_start=torch.from_numpy(doc).to(DEV))
    # rows are positions n - L + i: row i of sequence 1 sits at position i - 50
    bad_k = torch.from_numpy(pad).to(DEV)
    bad_q = bad_k.clone()
    bad_q[1] = torch.cat([torch.ones(50, dtype=torch.bool, device=DEV), bad_k[1, :150]])
    o1, l1 = sc.causal_attention(q, k, v, lse=True, **dev)
    g1 = sc.causal_attention_bwd(do, q, k, v, o1, l1, **dev)
    for t, m in ((q, bad_q), (k, bad_k), (v, bad_k), (do, bad_q)):
        t[m] = float("nan")
    o2, l2 = sc.causal_attention(q, k, v, lse=True, **dev)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert not o2[bad_q].any() and torch.isinf(l2.transpose(1, 2)[bad_q]).all()
    g2 = sc.causal_attention_bwd(do, q, k, v, o2, l2, **dev)
    for a, b, m in zip(g1, g2, (bad_q, bad_k, bad_k)):
        assert torch.equal(a, b) and not b[m].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_tensors(sc, dtype):
    # q, k, v columns of one projection, gradients into columns of another, heads outside tokens
    print("case attn strides %s" % dtype, flush=True)
    rng = np.random.default_rng(8)
    B, L, H, Hkv, D = 2, 140, 4, 2, 64
    x, xr = draw(rng, (B, L, H + 2 * Hkv, D), dtype)
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    do, _ = draw(rng, (B, H, L, D), dtype)
    do = do.transpose(1, 2)
    o, lse = sc.causal_attention(q, k, v, window=50, lse=True)
    o2, lse2 = sc.causal_attention(q.contiguous(), k.contiguous(), v.transpose(1, 2).contiguous().transpose(1, 2),
                                   window=50, lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    plain = sc.causal_attention_bwd(do.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), o, lse, window=50)
    g = torch.full((B, L, H + 2 * Hkv + 1, D), 7.0, dtype=x.dtype, device=DEV)
    got = sc.causal_attention_bwd(do, q, k, v, o, lse, window=50, dq=g[:, :, :H], dk=g[:, :, H:H + Hkv],
                                  dv=g[:, :, H + Hkv:H + 2 * Hkv])
    for a, b in zip(plain, got):
        assert torch.equal(a, b)
    assert (g[:, :, -1] == 7.0).all()
    # a key cache broadcast over the batch (stride 0)
    one = sc.causal_attention(q.contiguous(), k[:1].contiguous().expand(B, -1, -1, -1), v, window=50)
    two = sc.causal_attention(q.contiguous(), k[:1].contiguous().repeat(B, 1, 1, 1), v, window=50)
    assert torch.equal(one, two)


def test_large_scores(sc):
    # scores far apart and far from 0: the running maximum keeps the exponentials in range
    rng = np.random.default_rng(2)
    q, qr = draw(rng, (1, 80, 1, 64), "f32", 30.0)
    k, kr = draw(rng, (1, 80, 1, 64), "f32", 10.0)
    v, vr = draw(rng, (1, 80, 1, 64), "f32")
    o, lse = sc.causal_attention(q, k, v, lse=True)
    want, bound = ref.attention(qr, kr, vr, 0.125)
    check(o, want[0], bound[0], "f32", "o")
    check(lse, want[1], bound[1], "f32", "lse")


def test_repeats_bit_for_bit_on_another_stream(sc):
    q, k, v, do = (torch.randn(2, 500, 4, 64, device=DEV).bfloat16() for _ in range(4))
    o, lse = sc.causal_attention(q, k, v, lse=True, window=128)
    g = sc.causal_attention_bwd(do, q, k, v, o, lse, window=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = sc.causal_attention(q, k, v, lse=True, window=128)
        g2 = sc.causal_attention_bwd(do, q, k, v, o2, lse2, window=128)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(g, g2))


def test_empty(sc):
    e = torch.empty(2, 0, 4, 64, device=DEV)
    q = torch.randn(2, 3, 4, 64, device=DEV)
    o, lse = sc.causal_attention(q, e, e, lse=True)       # no keys: nothing is seen
    assert not o.any() and torch.isinf(lse).all()
    assert not sc.causal_attention_bwd(q, q, e, e, o, lse)[0].any()
    o, lse = sc.causal_attention(e, q, q, lse=True)       # no rows
    assert o.shape == e.shape
    _, dk, dv = sc.causal_attention_bwd(e, e, q, q, o, lse)
    assert not dk.any() and not dv.any()


# enough heads for the workgroups of 128 rows and keys, which fewer never reach
MANY = [dict(L=200, H=16, Hkv=16, D=64, window=70, bias=True),
        dict(L=200, H=16, Hkv=16, D=40, docs=50, pad=3, bias=True),
        dict(L=129, H=32, Hkv=16, D=128, cap=5.0),
        dict(L=160, H=32, Hkv=16, D=64, cap=5.0, docs=60, window=90, bias=True),
        dict(L=190, H=16, Hkv=16, D=96)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "L%d-H%d-D%d" % (c["L"], c["H"], c["D"]))
def test_many_heads(sc, dtype, case):
    print("case attn many heads %s %s" % (dtype, case), flush=True)
    c = dict(case)
    L = c.pop("L")
    run(sc, 40, L, L, c.pop("H"), c.pop("Hkv"), c.pop("D"), dtype, **c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_heads_over_a_cache(sc, dtype, D):
    print("case attn many heads cache %s D=%d" % (dtype, D), flush=True)
    kv_len = [(37 * b) % 300 for b in range(40)]   # also rows of length 0 and shorter than the queries
    run(sc, 40, 140, 299, 16, 16, D, dtype, kv_len=kv_len, window=120, bias=True)
