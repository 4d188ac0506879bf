"""A small hybrid stack on the library's calls, trained and then decoded token by token.

Layers, each on layer-normalised activations with a residual connection, as the notes of
"Caracal: Causal Architecture via Spectral Mixing" arrange them: causal convolution layers
(v and a data-dependent gate stream from the same input), window attention with a distance bias
(positional encodings are removed), and a gated recurrence.  Projections are torch matmuls; the
mixing and the norms, forward and backward, are this library's kernels.

    python examples/hybrid_stack.py            # a few steps of training, then decoding
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fft_causal_long_amd as sc  # noqa: E402


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        y, mean, rstd = sc.layer_norm(x, w, b, stats=True)
        ctx.save_for_backward(x, w, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        return sc.layer_norm_bwd(dy.contiguous(), x, mean, rstd, w)


class CausalConv(torch.autograd.Function):
    """r = causal_conv(v, g) of channel-major (B, C, L) tensors."""

    @staticmethod
    def forward(ctx, v, g):
        ctx.save_for_backward(v, g)
        return sc.causal_conv(v, g)

    @staticmethod
    def backward(ctx, dr):
        return sc.causal_conv_bwd(dr.contiguous(), *ctx.saved_tensors)


class WindowAttention(torch.autograd.Function):
    """Attention of the q, k, v columns of one projection (B, L, (H + 2 Hkv) D)."""

    @staticmethod
    def forward(ctx, qkv, H, Hkv, window, slopes, doc_start):
        q, k, v = columns(qkv, H, Hkv)
        opt = dict(window=window, slopes=slopes, doc_start=doc_start)
        o, lse = sc.causal_attention(q, k, v, lse=True, **opt)
        ctx.save_for_backward(qkv, o, lse)
        ctx.args = H, Hkv, opt
        return o.flatten(2)

    @staticmethod
    def backward(ctx, do):
        qkv, o, lse = ctx.saved_tensors
        H, Hkv, opt = ctx.args
        dqkv = torch.empty_like(qkv)   # the gradients go to the projection's own columns
        dq, dk, dv = columns(dqkv, H, Hkv)
        sc.causal_attention_bwd(do.reshape(o.shape).contiguous(), *columns(qkv, H, Hkv), o, lse, dq=dq, dk=dk,
                                dv=dv, **opt)
        return dqkv, None, None, None, None, None


class Recurrence(torch.autograd.Function):
    """h of the z, u halves of one projection (B, L, 2 C)."""

    @staticmethod
    def forward(ctx, zu):
        C = zu.shape[-1] // 2
        h, _ = sc.gated_recurrence(zu[..., :C], zu[..., C:])
        ctx.save_for_backward(zu, h)
        return h

    @staticmethod
    def backward(ctx, dh):
        zu, h = ctx.saved_tensors
        C = h.shape[-1]
        dzu = torch.empty_like(zu)
        sc.gated_recurrence_bwd(dh.contiguous(), zu[..., :C], zu[..., C:], h, dz=dzu[..., :C], du=dzu[..., C:])
        return dzu


def columns(qkv, H, Hkv):
    x = qkv.unflatten(-1, (H + 2 * Hkv, -1))
    return x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]


class Stack(torch.nn.Module):
    """`layout`: one letter a layer, c convolution, a attention, r recurrence."""

    def __init__(self, vocab=64, C=128, heads=4, kv_heads=2, D=32, window=32, layout="ccar",
                 dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)
        self.layout, self.H, self.Hkv, self.D, self.window = layout, heads, kv_heads, D, window

        def par(*shape, scale):
            return torch.nn.Parameter((torch.randn(*shape, generator=gen) * scale).to(device, dtype))

        width = {"c": 2 * C, "a": (heads + 2 * kv_heads) * D, "r": 2 * C}
        mixed = {"c": C, "a": heads * D, "r": C}
        self.embed = par(vocab, C, scale=C ** -0.5)
        self.w_in = torch.nn.ParameterList([par(C, width[x], scale=C ** -0.5) for x in layout])
        self.w_out = torch.nn.ParameterList([par(mixed[x], C, scale=0.5 * mixed[x] ** -0.5) for x in layout])
        n = len(layout) + 1
        self.norm_w = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(C, dtype=dtype, device=device)) for _ in range(n)])
        self.norm_b = torch.nn.ParameterList([torch.nn.Parameter(torch.zeros(C, dtype=dtype, device=device)) for _ in range(n)])
        self.slopes = torch.tensor([2.0 ** (-8 * (h + 1) / heads) for h in range(heads)], device=device)

    def forward(self, tokens, doc_start=None):
        """Logits (B, L, vocab) in float32."""
        x = self.embed[tokens]
        for i, kind in enumerate(self.layout):
            p = LayerNorm.apply(x, self.norm_w[i], self.norm_b[i]) @ self.w_in[i]
            if kind == "c":
                v, s = p.transpose(1, 2).chunk(2, 1)
                m = CausalConv.apply(v.contiguous(), (torch.sigmoid(s) / tokens.shape[1] ** 0.5).contiguous()).transpose(1, 2)
            elif kind == "a":
                m = WindowAttention.apply(p, self.H, self.Hkv, self.window, self.slopes, doc_start)
            else:
                m = Recurrence.apply(p)
            x = x + m @ self.w_out[i]
        return (LayerNorm.apply(x, self.norm_w[-1], self.norm_b[-1]) @ self.embed.T).float()

    # ---- one token at a time (attention and recurrence layers: a convolution's output depends on
    # its whole past, it has no state of fixed size)

    def start(self, B, length):
        """The caches and states of an empty sequence of up to `length` tokens."""
        dev, dt = self.embed.device, self.embed.dtype
        state = []
        for kind in self.layout:
            if kind == "a":
                state.append(torch.zeros(2, B, length, self.Hkv, self.D, dtype=dt, device=dev))
            elif kind == "r":
                state.append(torch.zeros(B, self.embed.shape[1], device=dev))
            else:
                raise ValueError("convolution layers have no single-token form")
        return state, torch.zeros(B, dtype=torch.int32, device=dev)

    @torch.no_grad()
    def step(self, tokens, state, lengths):
        """Logits (B, vocab) of the next tokens (B,); caches, states and lengths move on."""
        x = self.embed[tokens][:, None]
        rows = torch.arange(len(tokens), device=tokens.device)
        at = lengths.long()
        lengths += 1
        for i, kind in enumerate(self.layout):
            p = sc.layer_norm(x, self.norm_w[i], self.norm_b[i]) @ self.w_in[i]
            if kind == "a":
                q, k, v = columns(p, self.H, self.Hkv)
                state[i][0][rows, at], state[i][1][rows, at] = k[:, 0], v[:, 0]
                m = sc.causal_attention(q, state[i][0], state[i][1], window=self.window, slopes=self.slopes,
                                        kv_len=lengths).flatten(2)
            else:
                C = p.shape[-1] // 2
                m, _ = sc.gated_recurrence(p[..., :C], p[..., C:], state[i], hT=state[i])
            x = x + m @ self.w_out[i]
        return (sc.layer_norm(x, self.norm_w[-1], self.norm_b[-1]) @ self.embed.T).float()[:, 0]


def task(B, L, vocab, gen, device="cuda"):
    """Sequences that each draw their tokens from four of their own: the next one is known to one of
    four (a loss of log 4) by a model that has looked at the past, to one of `vocab` by one that has not."""
    own = torch.rand(B, vocab, generator=gen).topk(4).indices
    out = own.gather(1, torch.randint(4, (B, L + 1), generator=gen))
    return out[:, :-1].to(device), out[:, 1:].to(device)


def train(model, steps=60, B=16, L=256, lr=3e-3, seed=1, say=print):
    """The losses of `steps` steps (torch's Adam on float32 copies of the weights)."""
    gen = torch.Generator().manual_seed(seed)
    params = list(model.parameters())
    master = [p.detach().float().requires_grad_() for p in params]
    opt = torch.optim.Adam(master, lr)
    losses = []
    for step in range(steps):
        x, y = task(B, L, model.embed.shape[0], gen, model.embed.device)
        loss = torch.nn.functional.cross_entropy(model(x).flatten(0, 1), y.flatten())
        model.zero_grad()
        loss.backward()
        for m, p in zip(master, params):
            m.grad = p.grad.float()
        opt.step()
        with torch.no_grad():
            for m, p in zip(master, params):
                p.copy_(m)
        losses.append(float(loss.detach()))
        if say and step % 10 == 0:
            say("step %3d  loss %.3f" % (step, losses[-1]))
    return losses


def main():
    losses = train(Stack())
    print("convolution, attention and recurrence layers: loss %.3f -> %.3f" % (losses[0], losses[-1]))
    model = Stack(layout="ara")
    train(model, say=None)
    x, _ = task(4, 64, 64, torch.Generator().manual_seed(9))
    state, lengths = model.start(4, 96)
    for t in range(x.shape[1]):
        logits = model.step(x[:, t], state, lengths)
    full = model(x).detach()[:, -1]
    print("after 64 tokens one at a time, logits within %.3g of the whole sequence's" % float((logits - full).abs().max()))


if __name__ == "__main__":
    main()
