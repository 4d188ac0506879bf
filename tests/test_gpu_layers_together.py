"""The layer calls as a program uses them: captured into a graph, over rows whose offsets pass 32
bits, and in the example stack (training and decoding)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layers as ref
from tests.layer_util import DEV, check, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sc():
    import fft_causal_long_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_captured_calls_follow_their_inputs(sc):
    # norm, attention over documents and a split cache, and a recurrence cut into segments, forward
    # and backward, replayed on changing inputs between eager work
    print("case layers captured", flush=True)
    B, L, H, D = 1, 3000, 2, 64
    C = H * D
    x = torch.randn(B, L, C, device=DEV).bfloat16()
    w, b = torch.randn(C, device=DEV).bfloat16(), torch.randn(C, device=DEV).bfloat16()
    doc = (torch.arange(L, device=DEV, dtype=torch.int32) // 700 * 700)[None]
    assert sc.sc_recur_workspace_bytes(sc.KIND_BF16, B, L, C) > 0

    def work():
        y, mean, rstd = sc.layer_norm(x, w, b, stats=True)
        q = y.view(B, L, H, D)
        o, lse = sc.causal_attention(q, q, q, window=256, doc_start=doc, lse=True)
        one = sc.causal_attention(q[:, :1], q, q)
        h, hT = sc.gated_recurrence(y, o.view(B, L, C))
        dz, du, dh0 = sc.gated_recurrence_bwd(y, y, o.view(B, L, C), h)
        dq, dk, dv = sc.causal_attention_bwd(du.view(B, L, H, D), q, q, q, o, lse, window=256, doc_start=doc)
        dx, dw, db = sc.layer_norm_bwd(dq.view(B, L, C), x, mean, rstd, w)
        return o, one, h, hT, dz, du, dh0, dk, dv, dx, dw, db

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for turn in range(4):
        x.copy_(torch.randn(B, L, C, device=DEV))
        graph.replay()
        got = [t.clone() for t in out]
        want = work()
        torch.cuda.synchronize()
        for i, (g, r) in enumerate(zip(got, want)):
            assert torch.equal(g, r), (turn, i)


def test_offsets_past_32_bits(sc):
    # rows 2^21 elements apart: element offsets reach 2^32 (8 GB of address space, few rows touched)
    print("case layers long offsets", flush=True)
    rng = np.random.default_rng(4)
    L, S = 2049, 1 << 21
    base = torch.empty((L - 1) * S + 4096, dtype=torch.bfloat16, device=DEV)
    rows = base.as_strided((L, 256), (S, 1))
    rows.copy_(torch.from_numpy(rng.standard_normal((L, 256)).astype(np.float32)))
    r = f64(rows)
    k, v = rows[:, :64].view(1, L, 1, 64), rows[:, 64:128].view(1, L, 1, 64)
    for Lq in (1, 40):
        q = torch.from_numpy(rng.standard_normal((1, Lq, 2, 64)).astype(np.float32)).to(DEV).bfloat16()
        o, lse = sc.causal_attention(q, k, v, lse=True)
        want, bound = ref.attention(f64(q), r[None, :, None, :64], r[None, :, None, 64:128], 0.125, bf16=True)
        check(o, want[0], bound[0], "bf16", "o Lq=%d" % Lq)
        check(lse, want[1], bound[1], "f32", "lse Lq=%d" % Lq)
    do = torch.randn(1, 40, 2, 64, device=DEV).bfloat16()
    got = sc.causal_attention_bwd(do, q, k, v, o, lse)
    want, bound = ref.attention_bwd(f64(do), f64(q), r[None, :, None, :64], r[None, :, None, 64:128], f64(o), f64(lse),
                                    0.125, bf16=True)
    for g, w_, b_, n in zip(got, want, bound, ("dq", "dk", "dv")):
        check(g, w_, b_, "bf16", n)
    z, u = rows[None, :, 128:160], rows[None, :, 160:192]
    h, hT = sc.gated_recurrence(z, u)
    (hr, hTr), (bh, bT) = ref.recurrence(r[None, :, 128:160], r[None, :, 160:192], np.zeros((1, 32)))
    check(h, hr, bh, "bf16", "h")
    check(hT, hTr, bT, "f32", "hT")
    y, mean, rstd = sc.layer_norm(rows[:, :192], out=None, stats=True)
    want, bound = ref.layernorm(r[:, :192], np.ones(192), np.zeros(192), 1e-5)
    check(y, want[0], bound[0], "bf16", "y")
    # an output that far out
    sc.layer_norm(rows[:, :64], out=rows[:, 192:256])
    want, bound = ref.layernorm(r[:, :64], np.ones(64), np.zeros(64), 1e-5)
    check(rows[:, 192:256], want[0], bound[0], "bf16", "y in place of columns")


def test_many_heads_share_a_key_head(sc):
    # the group's heads dealt out to several workgroups, whose parts are added in order
    print("case attn parts", flush=True)
    rng = np.random.default_rng(31)
    for H, D, dtype in ((7, 128, torch.bfloat16), (16, 40, torch.float32)):
        q, do = (torch.from_numpy(rng.standard_normal((1, 200, H, D)).astype(np.float32)).to(DEV, dtype) for _ in range(2))
        k, v = (torch.from_numpy(rng.standard_normal((1, 200, 1, D)).astype(np.float32)).to(DEV, dtype) for _ in range(2))
        o, lse = sc.causal_attention(q, k, v, lse=True, window=100)
        a = sc.causal_attention_bwd(do, q, k, v, o, lse, window=100)
        b = sc.causal_attention_bwd(do, q, k, v, o, lse, window=100)
        name = "bf16" if dtype == torch.bfloat16 else "f32"
        want, bound = ref.attention_bwd(f64(do), f64(q), f64(k), f64(v), f64(o), f64(lse), float(np.float32(D ** -0.5)),
                                        window=100, bf16=name == "bf16")
        for g, g2, w, bd, n in zip(a, b, want, bound, ("dq", "dk", "dv")):
            assert torch.equal(g, g2)
            check(g, w, bd, name, n)


def test_example_learns_and_decodes(example):
    print("case example", flush=True)
    model = example.Stack()
    losses = example.train(model, say=None)
    assert all(np.isfinite(losses))
    # more than half the way from the guess of one of 64 tokens to that of one of the sequence's four
    assert losses[-1] < 0.5 * (np.log(64) + np.log(4)), losses
    # one token at a time against the whole sequence, float32: the same sums in another order
    model = example.Stack(layout="ara", dtype=torch.float32)
    x, _ = example.task(3, 70, 64, torch.Generator().manual_seed(2))
    full = model(x).detach()
    state, lengths = model.start(3, 80)
    for t in range(x.shape[1]):
        logits = model.step(x[:, t], state, lengths)
        assert torch.allclose(logits, full[:, t], rtol=1e-4, atol=1e-3), t
