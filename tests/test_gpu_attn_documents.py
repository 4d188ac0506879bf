"""Attention over packed documents whose backward walk looks past the 64 stages it knows at once,
heads over 64 with documents, and documents in caches longer than the new tokens, against the
float64 reference.

A stage of the walk is 64 tokens for bfloat16 heads up to 64 and 32 otherwise."""
import numpy as np
import pytest
import torch

from oracle import layers as ref
from tests.layer_util import DEV, check, draw, f64
from tests.test_gpu_attn import documents, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def long_among_short(rng, B, L, lo, hi, pad):
    """One document lo .. hi - 1 among short ones; the last `pad` tokens are padding, and one inside."""
    d = documents(rng, B, L, 20, 0)
    for b in range(B):
        d[b, lo:hi] = lo
        at = hi
        while at < L:
            n = int(rng.integers(1, 40))
            d[b, at:at + n] = at
            at += n
        if pad:
            d[b, L - pad:] = L
            d[b, lo + 70] = L
    return d


def compare(sc, dtype, doc, H, Hkv, D, window=0, cap=0.0, bias=False, part=""):
    B, L = doc.shape
    rng = np.random.default_rng([L, H, D])
    q, qr = draw(rng, (B, L, H, D), dtype)
    k, kr = draw(rng, (B, L, Hkv, D), dtype)
    v, vr = draw(rng, (B, L, Hkv, D), dtype)
    do, dor = draw(rng, (B, L, H, D), dtype)
    slopes = np.asarray([2.0 ** (-8 * (h + 1) / H) for h in range(H)], np.float32) if bias else None
    dev = dict(window=window, cap=cap, doc_start=torch.from_numpy(doc).to(DEV),
               slopes=None if slopes is None else torch.from_numpy(slopes).to(DEV))
    o, lse = sc.causal_attention(q, k, v, lse=True, **dev)
    got = sc.causal_attention_bwd(do, q, k, v, o, lse, **dev)
    torch.cuda.synchronize()
    print("kernels done", flush=True)
    opt = dict(window=window, cap=cap, slopes=slopes, doc=doc, bf16=dtype == "bf16")
    scale = float(np.float32(D ** -0.5))
    (orf, lr), (bo, bl) = ref.attention(qr, kr, vr, scale, **opt)
    check(o, orf, bo, dtype, "o")
    check(lse, lr, bl, "f32", "lse")
    want, bound = ref.attention_bwd(dor, qr, kr, vr, f64(o), f64(lse), scale, **opt)
    for g, r, b, n in zip(got, want, bound, ("dq", "dk", "dv")):
        check(g, r, b, dtype, n)


@pytest.mark.parametrize("dtype,L,D", [("bf16", 4500, 64), ("bf16", 2300, 96), ("f32", 2300, 64), ("f32", 2300, 128)])
def test_documents_longer_than_the_stages_known_at_once(sc, dtype, L, D):
    print("case attn long documents %s L=%d D=%d" % (dtype, L, D), flush=True)
    doc = long_among_short(np.random.default_rng(L), 1, L, 300, L - 150, 20)
    compare(sc, dtype, doc, 2, 1, D, bias=True)


@pytest.mark.parametrize("dtype,D", [("bf16", 96), ("f32", 40)])
def test_two_heads_a_part(sc, dtype, D):
    # 34 heads on one key head and 34 key blocks: the heads are dealt out in twos, and the second
    # head of a part starts with what the first had looked up last
    print("case attn long documents, two heads a part %s" % dtype, flush=True)
    L = 2150
    doc = long_among_short(np.random.default_rng(7), 1, L, 200, L - 30, 10)
    compare(sc, dtype, doc, 34, 1, D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("docs,pad,window", [(1, 0, 0), (40, 20, 0), (70, 9, 30), (300, 130, 0)])
@pytest.mark.parametrize("D", [72, 96, 128])
def test_documents_with_larger_heads(sc, dtype, docs, pad, window, D):
    print("case attn documents %s D=%d %d %d %d" % (dtype, D, docs, pad, window), flush=True)
    run(sc, 2, 333, 333, 4, 2, D, dtype, docs=docs, pad=pad, window=window, bias=True, cap=6.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq,Lk,D", [(1, 200, 64), (7, 130, 128), (130, 257, 64), (90, 400, 96), (200, 333, 40)])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (6, 2)])
def test_documents_in_a_cache(sc, dtype, Lq, Lk, D, H, Hkv):
    # the rows' documents are read from their positions on, which differ from sequence to sequence
    print("case attn documents in a cache %s Lq=%d Lk=%d D=%d H=%d" % (dtype, Lq, Lk, D, H), flush=True)
    for kv_len in (None, [Lk, Lk - Lk // 3, max(Lq // 2, 1)]):
        run(sc, 3, Lq, Lk, H, Hkv, D, dtype, kv_len=kv_len, docs=50, pad=4, bias=True)
