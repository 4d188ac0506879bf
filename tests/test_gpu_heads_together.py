"""The calls on heads as a serving program uses them: norm and rotation, the cache's write and its
attention one after the other, captured, on other streams, and in the example stack."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import heads as ref
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


def lengths(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


class Layer:
    """One attention layer's decoding: projections in, attention out."""

    def __init__(self, sc, code, B, H, Hkv, D, length, paged, gen):
        self.sc, self.H, self.Hkv = sc, H, Hkv
        N = -(-length // 64)
        table = torch.randperm(B * N + 2, generator=gen)[:B * N].view(B, N).int().to(DEV) if paged else None
        self.cache = sc.KVCache(B, length, Hkv, D, code, device=DEV, blocks=B * N + 2 if paged else None, table=table)
        self.freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).to(DEV)
        self.wq, self.wk = (torch.rand(D, generator=gen).add_(0.5).to(DEV).bfloat16() for _ in "qk")

    def __call__(self, qkv, n):
        q, k, v = qkv[:, :, :self.H], qkv[:, :, self.H:self.H + self.Hkv], qkv[:, :, self.H + self.Hkv:]
        q, k = self.sc.qk_norm_rotary(q, k, self.wq, self.wk, self.freq, kv_len=n)
        self.sc.cache_write(self.cache, k, v, n)
        return self.sc.cached_attention(q, self.cache, n, window=100, sinks=3, lse=True)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("paged", [False, True])
def test_a_prompt_and_its_continuation(sc, code, paged):
    # a prompt in two parts, then single tokens: every step against the model and the reference
    print("case heads serving", code, paged, flush=True)
    gen = torch.Generator().manual_seed(5)
    B, H, Hkv, D = 2, 6, 2, 64
    layer = Layer(sc, code, B, H, Hkv, D, 256, paged, gen)
    N = layer.cache.N
    m = ref.Cache(B, N, layer.cache.blocks, Hkv, D, code, None if not paged else layer.cache.table.cpu().numpy())
    lens = np.array([0, 0])
    eps = float(np.float32(1e-6))
    for L, more in ((130, (130, 71)), (40, (40, 40)), (1, (1, 1)), (1, (1, 1)), (3, (3, 0)), (1, (1, 1))):
        lens = lens + np.array(more)
        qkv = torch.randn(B, L, H + 2 * Hkv, D, generator=gen).to(DEV).bfloat16()
        o, lse = layer(qkv, lengths(*lens))
        # the rotated q and k as the layer computed them, checked by themselves
        pos = lens[:, None] - L + np.arange(L)
        q, k = sc.qk_norm_rotary(qkv[:, :, :H], qkv[:, :, H:H + Hkv], layer.wq, layer.wk, layer.freq, kv_len=lengths(*lens))
        check(q, *ref.qk_norm(f64(qkv[:, :, :H]), f64(layer.wq), pos, f64(layer.freq), False, eps), "bf16", "q")
        m.write(f64(k), f64(qkv[:, :, H + Hkv:]), lens)
        kx, vx, live = m.read(64 * N, [64 * N] * B)
        (ro, rl), (bo, bl) = ref.cached_attention(f64(q), kx, vx, lens, 0.125, 100, 3, live=live, bf16=True)
        check(o, ro, bo, "bf16", "o after %s" % lens)
        check(lse, rl, bl, "f32", "lse")


def test_captured_steps_move_on_with_their_lengths(sc):
    # a graph that lengthens the sequences, norms, writes and attends, replayed with eager work between;
    # and a second graph with a workspace of its own
    print("case heads captured", flush=True)
    gen = torch.Generator().manual_seed(6)
    B, H, Hkv, D = 3, 8, 2, 64
    layers = [Layer(sc, code, B, H, Hkv, D, 4096, True, torch.Generator().manual_seed(1)) for code in ("int8", "e4m3")]
    eager = [Layer(sc, code, B, H, Hkv, D, 4096, True, torch.Generator().manual_seed(1)) for code in ("int8", "e4m3")]
    x = torch.zeros(B, 1, H + 2 * Hkv, D, device=DEV, dtype=torch.bfloat16)
    prompt = torch.randn(B, 3000, H + 2 * Hkv, D, generator=gen).to(DEV).bfloat16()
    for l in layers + eager:
        l(prompt, lengths(3000, 1500, 10))
    ns = [lengths(3000, 1500, 10) for _ in layers]
    graphs, outs, kept = [], [], []      # (a graph's workspace lives as long as the graph)
    for l, n in zip(layers, ns):
        a = sc.sc_cached(1, H)
        a.scale = 0.125
        need = sc.sc_cached_attn_workspace_bytes(sc.KIND_BF16, l.cache._struct, a)
        assert need > 0
        ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
        ws = ws[(-ws.data_ptr()) % 256:][:need]
        kept.append(ws)

        def work(l=l, n=n, ws=ws):
            n.add_(1)
            q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
            q, k = sc.qk_norm_rotary(q, k, l.wq, l.wk, l.freq, kv_len=n)
            sc.cache_write(l.cache, k, v, n)
            return sc.cached_attention(q, l.cache, n, lse=True, workspace=ws), sc.cache_read(l.cache, 2, n)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work()
        torch.cuda.current_stream().wait_stream(side)
        n.copy_(lengths(3000, 1500, 10))      # (the step above wrote one token that the first replay writes again)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work())
        graphs.append(graph)
        n.copy_(lengths(3000, 1500, 10))
    n = lengths(3000, 1500, 10)
    for turn in range(5):
        x.copy_(torch.randn(B, 1, H + 2 * Hkv, D, generator=gen))
        n += 1
        for g in graphs:
            g.replay()
        for e, got in zip(eager, outs):
            q, k = sc.qk_norm_rotary(x[:, :, :H], x[:, :, H:H + Hkv], e.wq, e.wk, e.freq, kv_len=n)
            sc.cache_write(e.cache, k, x[:, :, H + Hkv:], n)
            want = sc.cached_attention(q, e.cache, n, lse=True), sc.cache_read(e.cache, 2, n)
            torch.cuda.synchronize()
            for g, w in zip(got[0] + got[1], want[0] + want[1]):
                assert torch.equal(g, w), turn


def test_backward_captured(sc):
    print("case heads backward captured", flush=True)
    x = torch.randn(2, 300, 4, 64, device=DEV).bfloat16()
    f = torch.rand(32, device=DEV)
    w = torch.ones(64, device=DEV).bfloat16()

    def work():
        y, z = sc.qk_norm_rotary(x[:, :, :3], x[:, :, 3:], w, w, f)
        return (y, z) + sc.qk_norm_rotary_bwd(y, z, x[:, :, :3], x[:, :, 3:], w, w, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for turn in range(4):
        x.copy_(torch.randn(2, 300, 4, 64, device=DEV))
        w.copy_(torch.rand(64, device=DEV) + 0.5)
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        for g, r in zip(out, want):
            assert torch.equal(g, r), turn


def test_two_streams_at_once(sc):
    # two caches served on two streams: the calls share nothing
    print("case heads streams", flush=True)
    gen = torch.Generator().manual_seed(8)
    layers = [Layer(sc, "int8", 2, 8, 2, 128, 2048, False, torch.Generator().manual_seed(2)) for _ in range(3)]
    xs = [torch.randn(2, L, 12, 128, generator=gen).to(DEV).bfloat16() for L in (1500, 1, 1, 1)]
    want = []
    n = [lengths(1500 + i, 900 + i) for i in range(4)]
    for x, m in zip(xs, n):
        want.append(layers[0](x, m))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for x, m in zip(xs, n):
        for s, l, g in zip(streams, layers[1:], got):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.append(l(x, m))
    torch.cuda.synchronize()
    for g in got:
        for (a, b), (c, d) in zip(g, want):
            assert torch.equal(a, c) and torch.equal(b, d)


def test_example_with_rotation_decodes_from_8_bits(example):
    print("case heads example", flush=True)
    # one token at a time against the whole sequence, float32 caches and the caches of codes
    model = example.Stack(layout="ara", dtype=torch.float32, rotary=True, window=1000)
    losses = example.train(model, steps=3, say=None)
    assert all(np.isfinite(losses))
    x, _ = example.task(3, 70, 64, torch.Generator().manual_seed(2))
    full = model(x).detach()
    state, n = model.start(3, 80)
    for t in range(x.shape[1]):
        logits = model.step(x[:, t], state, n)
        assert torch.allclose(logits, full[:, t], rtol=1e-4, atol=1e-3), t
    for code in ("int8", "e4m3"):
        state, n = model.start(3, 80, code)
        for t in range(x.shape[1]):
            logits = model.step(x[:, t], state, n, sinks=2)
        assert torch.isfinite(logits).all() and n.tolist() == [70] * 3
        # the layers' keys and values are those of the float caches to half a code's step
        k, v = example.sc.cache_read(state[0], 70, n, torch.float32)
        again, m = model.start(3, 80)
        for t in range(x.shape[1]):
            model.step(x[:, t], again, m)
        for got, want, scale in ((k, again[0][0][:, :70], state[0].k_scale), (v, again[0][1][:, :70], state[0].v_scale)):
            step = scale.view(3, 2, -1).repeat_interleave(64, 1)[:, :70, :, None]
            # int8: half a step, at most one rounding more for each of the doublings of its scale; e4m3:
            # 2^-4 of the value, or half the smallest step
            bound = step if code == "int8" else 2.0 ** -4 * want.abs() + 2.0 ** -10 * step
            assert ((got - want).abs() <= bound * 1.0001).all()


def test_example_gradients_with_rotation(example):
    # the loss's slope along the gradient, by differences in float32
    print("case heads example gradients", flush=True)
    model = example.Stack(layout="a", dtype=torch.float32, rotary=True)
    x, y = example.task(2, 40, 64, torch.Generator().manual_seed(3))

    def loss():
        return torch.nn.functional.cross_entropy(model(x).double().flatten(0, 1), y.flatten())
    loss().backward()
    for name in ("q_w", "k_w"):
        p = getattr(model, name)[0]
        g = p.grad.clone()
        d = torch.randn(64, generator=torch.Generator().manual_seed(4))[:p.numel()].to(DEV)
        eps = 1e-2
        with torch.no_grad():
            p += eps * d
            up = float(loss())
            p -= 2 * eps * d
            down = float(loss())
            p += eps * d
        want, got = (up - down) / (2 * eps), float((g.double() * d).sum())
        # float32 activations: about 2^-20 of a loss of log 64 over the step of 2e-2, and the curvature
        assert abs(want - got) <= 2.0 ** -20 * 4.2 / (2 * eps) + 0.02 * abs(want) + 1e-5, (name, want, got)
