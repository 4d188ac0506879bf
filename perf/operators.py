"""Cases that time the layer norm, causal attention and gated recurrence operators.

``own`` false: plain torch forms in 32 bits, rounded once to the storage type; ``own`` true:
the calls of this package.  Shapes are those of the models the library's workloads stand for
(12 and 16 heads of 64, contexts 1024, 4096 and 65536, attention window 256).
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-5


# --------------------------------------------------------------------------- cases

def _attn(**k):
    c = {"op": "attn", "dir": "fwd", "type": "bf16", "B": 1, "Lq": 1, "Lk": 1, "H": 1, "Hkv": 1,
         "D": 64, "window": 0, "cap": 0.0, "bias": False, "docs": 0, "ragged": False,
         "fused": False}
    c.update(k)
    return c


def listed():
    return [
        # layer norm of one decoding step of eight sequences: latency
        {"name": "ln-fwd-step", "op": "ln", "dir": "fwd", "type": "bf16", "rows": 8, "C": 768},
        # the Small model's activations, float32
        {"name": "ln-fwd-small", "op": "ln", "dir": "fwd", "type": "f32", "rows": 8192, "C": 768},
        # the Medium model's training step
        {"name": "ln-bwd-medium", "op": "ln", "dir": "bwd", "type": "bf16", "rows": 32768,
         "C": 1024},
        # one decoding step of eight sequences with their states: latency
        {"name": "rec-step", "op": "rec", "dir": "fwd", "type": "bf16", "B": 8, "L": 1, "C": 1024,
         "state": True, "strided": False},
        # the Medium model's forward pass, z and u the halves of one projection
        {"name": "rec-fwd-medium", "op": "rec", "dir": "fwd", "type": "bf16", "B": 8, "L": 4096,
         "C": 1024, "state": False, "strided": True},
        # the Small model's backward pass, float32
        {"name": "rec-bwd-small", "op": "rec", "dir": "bwd", "type": "f32", "B": 8, "L": 1024,
         "C": 768, "state": False, "strided": False},
        # one long document, few channels in flight at once
        {"name": "rec-fwd-long", "op": "rec", "dir": "fwd", "type": "f32", "B": 1, "L": 65536,
         "C": 1536, "state": True, "strided": False},
        # the Medium model's window attention layer, q, k, v from one projection
        _attn(name="attn-fwd-medium", B=8, Lq=4096, Lk=4096, H=16, Hkv=16, window=256, bias=True,
              fused=True),
        # a full causal layer with shared key heads over a long prompt
        _attn(name="attn-fwd-full", B=1, Lq=8192, Lk=8192, H=16, Hkv=4, D=128),
        # training the window layer on rows packed with documents
        _attn(name="attn-bwd-medium", dir="bwd", B=8, Lq=4096, Lk=4096, H=16, Hkv=16, window=256,
              bias=True, docs=700),
        # one new token a sequence over ragged long caches
        _attn(name="attn-decode", B=8, Lq=1, Lk=65536, H=16, Hkv=4, ragged=True),
        # float32 training of a capped layer on packed rows of an odd length
        _attn(name="attn-bwd-odd", dir="bwd", type="f32", B=2, Lq=1001, Lk=1001, H=12, Hkv=12,
              cap=30.0, bias=True, docs=300),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "rec", "attn", "attn"])
    ty = rng.choice(["f32", "bf16"])
    way = rng.choice(["fwd", "bwd"])
    if op == "ln":
        # a gradient over two or three channels is the rounding of terms that cancel
        C = rng.choice([_size(rng, 1 if way == "fwd" else 8, 16384), 8 * _size(rng, 8, 1024)])
        return {"op": "ln", "dir": way, "type": ty, "rows": _size(rng, 1, max(1, (1 << 25) // C)),
                "C": C}
    if op == "rec":
        C = rng.choice([_size(rng, 1, 4096), 64 * _size(rng, 1, 32)])
        B = _size(rng, 1, 16)
        top = max(1, min(65536, (3 << 24) // (B * C)))
        L = 1 if rng.random() < 0.15 else _size(rng, 1, top)
        return {"op": "rec", "dir": way, "type": ty, "B": B, "L": L, "C": C,
                "state": rng.random() < 0.5, "strided": rng.random() < 0.5}
    Hkv = rng.choice([1, 2, 4, 8, 12])
    G = rng.choice([1, 1, 2, 3, 4, 8]) if Hkv <= 8 else 1
    B = _size(rng, 1, 8)
    D = rng.choice([64, 64, 128, 40, 96])
    window = rng.choice([0, 256, _size(rng, 1, 1024)])
    cap = rng.choice([0.0, 0.0, 30.0])
    bias = rng.random() < 0.5
    docs = rng.choice([0, _size(rng, 20, 2000)])
    if rng.random() < 0.35:   # new tokens over a cache
        Lk = _size(rng, 1, max(1, (1 << 26) // (B * Hkv * D)))
        Lk = min(Lk, 262144)
        Lq = 1 if rng.random() < 0.6 else _size(rng, 1, min(Lk, 64))
        return _attn(type=ty, B=B, Lq=Lq, Lk=Lk, H=Hkv * G, Hkv=Hkv, D=D, window=window, cap=cap,
                     bias=bias, ragged=rng.random() < 0.7)
    L = _size(rng, 1, min(8192, int(math.sqrt((1 << 29) / (B * Hkv * G)))))
    if way == "bwd":   # a row that sees itself alone has the gradient 0, rounding aside
        L, window, docs = max(L, 48), max(window, 16) if window else 0, max(docs, 40) if docs else 0
    return _attn(dir=way, type=ty, B=B, Lq=L, Lk=L, H=Hkv * G, Hkv=Hkv, D=D, window=window,
                 cap=cap, bias=bias, docs=docs, ragged=rng.random() < 0.2,
                 fused=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs

def _doc_start(c):
    """Start of each token's document, (B, Lk); documents of varying length, the last twentieth
    of odd rows is padding (a start past the token: its row sees nothing)."""
    if not c["docs"]:
        return None
    r = np.random.default_rng([c["docs"], c["Lk"], c["B"]])
    out = np.zeros((c["B"], c["Lk"]), np.int32)
    for b in range(c["B"]):
        at = 0
        while at < c["Lk"]:
            n = max(1, int(c["docs"] * r.uniform(0.1, 1.9)))
            out[b, at:at + n] = at
            at += n
        if b % 2:
            out[b, c["Lk"] - c["Lk"] // 20:] = c["Lk"]
    return out


def _kv_len(c):
    if not c["ragged"]:
        return None
    return np.array([max(min(c["Lq"], c["Lk"]), c["Lk"] - (b * c["Lk"]) // (2 * c["B"]))
                     for b in range(c["B"])], np.int32)


def _slopes(c):
    return np.array([2.0 ** (-8.0 * (h + 1) / c["H"]) for h in range(c["H"])], np.float32)


def prepare(case, seed):
    c = case
    dt = DT[c["type"]]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape, mul=1.0, add=0.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(mul).add_(add).to(dt)

    def randn32(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = {"c": c}
    if c["op"] == "ln":
        s["x"] = randn(c["rows"], c["C"], mul=1.5, add=0.2)
        s["w"] = randn(c["C"], mul=0.2, add=1.0)
        s["b"] = randn(c["C"], mul=0.2)
        if c["dir"] == "bwd":
            s["dy"] = randn(c["rows"], c["C"])
            x = s["x"].float()
            s["mean"] = x.mean(-1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(-1) + EPS).rsqrt()
        return s
    if c["op"] == "rec":
        B, L, C = c["B"], c["L"], c["C"]
        if c["strided"]:
            zu = randn(B, L, 2 * C)
            zu[..., :C] += 2.0
            s["z"], s["u"] = zu[..., :C], zu[..., C:]
        else:
            s["z"], s["u"] = randn(B, L, C, add=2.0), randn(B, L, C)
        s["h0"] = randn32(B, C) if c["state"] else None
        if c["dir"] == "bwd":
            s["dh"] = randn(B, L, C)
            s["dhT"] = randn32(B, C) if c["state"] else None
            s["h"] = _rec_fwd(s)[0]
        return s
    B, Lq, Lk, H, Hkv, D = (c[k] for k in ("B", "Lq", "Lk", "H", "Hkv", "D"))
    if c["fused"]:
        qkv = randn(B, Lq, H + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    else:
        s["q"], s["k"], s["v"] = randn(B, Lq, H, D), randn(B, Lk, Hkv, D), randn(B, Lk, Hkv, D)
    doc, n = _doc_start(c), _kv_len(c)
    s["slopes"] = torch.from_numpy(_slopes(c)).to(DEV) if c["bias"] else None
    s["doc"] = None if doc is None else torch.from_numpy(doc).to(DEV)
    s["n"] = None if n is None else torch.from_numpy(n).to(DEV)
    if c["dir"] == "bwd":
        s["do"] = randn(B, Lq, H, D)
        s["o"], s["lse"] = _attn_fwd(s)
    return s


# --------------------------------------------------------------------------- plain forms

def _ln_fwd(s):
    dt = s["x"].dtype
    x = s["x"].float()
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = (d.square().mean(-1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["w"].float() + s["b"].float()
    return y.to(dt), mean, rstd


def _ln_bwd(s):
    dt = s["x"].dtype
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    e = dy * s["w"].float()
    dx = (e - e.mean(-1, keepdim=True) - xh * (e * xh).mean(-1, keepdim=True)) * s["rstd"][:, None]
    return dx.to(dt), (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, by doubling the span of each partial result."""
    step, L = 1, a.shape[1]
    while step < L:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _rec_fwd(s):
    z = s["z"].float()
    f, b = torch.sigmoid(z), torch.sigmoid(-z) * s["u"].float()
    if s["h0"] is not None:
        b[:, 0] += f[:, 0] * s["h0"]
    h = _scan(f, b)
    return h.to(s["z"].dtype), h[:, -1].clone()


def _rec_bwd(s):
    dt = s["z"].dtype
    z, u, h = s["z"].float(), s["u"].float(), s["h"].float()
    f, k = torch.sigmoid(z), torch.sigmoid(-z)
    dh = s["dh"].float()
    if s["dhT"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dhT"][:, None]], 1)
    a = torch.cat([torch.zeros_like(f[:, :1]), f[:, 1:].flip(1)], 1)
    g = _scan(a, dh.flip(1)).flip(1)
    first = torch.zeros_like(h[:, 0]) if s["h0"] is None else s["h0"]
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    dz = g * (before - u) * f * k
    return dz.to(dt), (k * g).to(dt), f[:, 0] * g[:, 0]


def _visible(s):
    c = s["c"]
    B, Lq, Lk = c["B"], c["Lq"], c["Lk"]
    n = s["n"].long() if s["n"] is not None else torch.full((B,), Lk, device=DEV)
    j = torch.arange(Lk, device=DEV)
    p = n[:, None] - Lq + torch.arange(Lq, device=DEV)           # (B, Lq)
    low = torch.zeros_like(p)
    live = torch.ones((B, Lk), dtype=torch.bool, device=DEV)
    if c["window"]:
        low = torch.maximum(low, p - c["window"] + 1)
    if s["doc"] is not None:
        low = torch.maximum(low, torch.gather(s["doc"].long(), 1, p.clamp(0, Lk - 1)))
        live = s["doc"] <= j
    see = (j >= low[:, :, None]) & (j <= p[:, :, None]) & live[:, None]
    return see[:, None], (p[:, :, None] - j)[:, None]            # (B, 1, Lq, Lk)


def _heads(x, G=1):
    return x.float().repeat_interleave(G, 2).transpose(1, 2).contiguous()


def _scores(s, q, k):
    c = s["c"]
    x = (q @ k.transpose(-1, -2)) * c["D"] ** -0.5
    t = None
    if c["cap"]:
        t = torch.tanh(x / c["cap"])
        x = c["cap"] * t
    see, far = _visible(s)
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * far
    return x.masked_fill(~see, -math.inf), t


def _attn_fwd(s):
    c = s["c"]
    G = c["H"] // c["Hkv"]
    x, _ = _scores(s, _heads(s["q"]), _heads(s["k"], G))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    o = (e @ _heads(s["v"], G)) / torch.where(l > 0, l, 1.0)
    return o.transpose(1, 2).contiguous().to(s["q"].dtype), (m + torch.log(l))[..., 0]


def _attn_bwd(s):
    c = s["c"]
    B, Lk, Hkv, D = c["B"], c["Lk"], c["Hkv"], c["D"]
    G, dt = c["H"] // Hkv, s["q"].dtype
    q, k, v, do = _heads(s["q"]), _heads(s["k"], G), _heads(s["v"], G), _heads(s["do"])
    x, t = _scores(s, q, k)
    lse = torch.where(torch.isinf(s["lse"]), 0.0, s["lse"])
    p = torch.exp(x - lse[..., None])
    delta = (do * _heads(s["o"])).sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - delta) * D ** -0.5
    if t is not None:
        ds = ds * (1 - t * t)
    dq = (ds @ k).transpose(1, 2)
    dk = (ds.transpose(-1, -2) @ q).view(B, Hkv, G, Lk, D).sum(2).transpose(1, 2)
    dv = (p.transpose(-1, -2) @ do).view(B, Hkv, G, Lk, D).sum(2).transpose(1, 2)
    return tuple(g.contiguous().to(dt) for g in (dq, dk, dv))


def run(state):
    s = state
    c = s["c"]
    if not own:
        return {"ln": {"fwd": _ln_fwd, "bwd": _ln_bwd}, "rec": {"fwd": _rec_fwd, "bwd": _rec_bwd},
                "attn": {"fwd": _attn_fwd, "bwd": _attn_bwd}}[c["op"]][c["dir"]](s)
    import fft_causal_long_amd as sc
    if c["op"] == "ln":
        if c["dir"] == "fwd":
            return sc.layer_norm(s["x"], s["w"], s["b"], eps=EPS, stats=True)
        return sc.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if c["op"] == "rec":
        if c["dir"] == "fwd":
            return sc.gated_recurrence(s["z"], s["u"], s["h0"])
        return sc.gated_recurrence_bwd(s["dh"], s["z"], s["u"], s["h"], s["h0"], s["dhT"])
    opt = dict(window=c["window"], cap=c["cap"], slopes=s["slopes"], doc_start=s["doc"],
               kv_len=s["n"])
    if c["dir"] == "fwd":
        return sc.causal_attention(s["q"], s["k"], s["v"], lse=True, **opt)
    return sc.causal_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **opt)


# --------------------------------------------------------------------------- counts

def _ranges(c):
    """First visible key and position of each query row, (B, Lq), and the live keys (B, Lk)."""
    n = _kv_len(c)
    n = np.full(c["B"], c["Lk"]) if n is None else n
    p = n[:, None].astype(np.int64) - c["Lq"] + np.arange(c["Lq"])
    low = np.zeros_like(p)
    live = np.ones((c["B"], c["Lk"]), bool)
    if c["window"]:
        low = np.maximum(low, p - c["window"] + 1)
    doc = _doc_start(c)
    if doc is not None:
        low = np.maximum(low, np.take_along_axis(doc, np.clip(p, 0, c["Lk"] - 1), 1))
        live = doc <= np.arange(c["Lk"])
    return low, p, live


def work(case):
    c = case
    e = 4 if c["type"] == "f32" else 2
    if c["op"] == "ln":
        n = c["rows"] * c["C"]
        if c["dir"] == "fwd":
            return {"bytes": 2 * n * e + 2 * c["C"] * e + 8 * c["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * c["C"] * e + 8 * c["rows"], "flops": 14 * n}
    if c["op"] == "rec":
        n, st = c["B"] * c["L"] * c["C"], c["B"] * c["C"] * 4
        if c["dir"] == "fwd":
            return {"bytes": 3 * n * e + st * (2 if c["state"] else 1), "flops": 10 * n}
        return {"bytes": 6 * n * e + st * (3 if c["state"] else 1), "flops": 14 * n}
    low, p, live = _ranges(c)
    seen = np.concatenate([np.zeros((c["B"], 1), np.int64), np.cumsum(live, 1)], 1)
    lo, hi = np.clip(low, 0, c["Lk"]), np.clip(p + 1, 0, c["Lk"])
    pairs = int(np.maximum(np.take_along_axis(seen, np.maximum(hi, lo), 1)
                           - np.take_along_axis(seen, lo, 1), 0).sum())
    # keys some row sees: from the lowest start to the end of the sequence
    keys = int(sum(hi[b].max() - min(lo[b].min(), hi[b].max()) for b in range(c["B"])))
    q = c["B"] * c["Lq"] * c["H"] * c["D"] * e
    kv = keys * c["Hkv"] * c["D"] * e
    whole = c["B"] * c["Lk"] * c["Hkv"] * c["D"] * e
    stat = c["B"] * c["Lq"] * c["H"] * 4
    if c["dir"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * c["D"] * pairs * c["H"]}
    return {"bytes": 4 * q + 2 * kv + 2 * whole + stat, "flops": 10 * c["D"] * pairs * c["H"]}


# --------------------------------------------------------------------------- 64 bits

def _exact_ln(s):
    d = {k: s[k].double() for k in ("x", "w", "b")}
    C = d["x"].shape[1]
    if s["c"]["dir"] == "fwd":
        mean = d["x"].sum(1) / C
        var = (d["x"] - mean[:, None]).pow(2).sum(1) / C
        y = (d["x"] - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * d["w"] + d["b"]
        return y, mean, 1 / torch.sqrt(var + EPS)
    dy, r = s["dy"].double(), s["rstd"].double()[:, None]
    xh = (d["x"] - s["mean"].double()[:, None]) * r
    e = dy * d["w"]
    dx = r * (e - e.sum(1, keepdim=True) / C - xh * ((e * xh).sum(1, keepdim=True) / C))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _exact_rec(s):
    z, u = s["z"].double(), s["u"].double()
    B, L, C = z.shape
    first = torch.zeros(B, C, dtype=torch.float64, device=DEV)
    if s["h0"] is not None:
        first = s["h0"].double()
    if s["c"]["dir"] == "fwd":
        h, st = torch.empty_like(z), first
        for t in range(L):
            f = 1 / (1 + torch.exp(-z[:, t]))
            st = f * st + u[:, t] / (1 + torch.exp(z[:, t]))
            h[:, t] = st
        return h, h[:, -1].clone()
    dh, h = s["dh"].double(), s["h"].double()
    dz, du = torch.empty_like(z), torch.empty_like(z)
    carry = torch.zeros_like(first) if s["dhT"] is None else s["dhT"].double()
    for t in reversed(range(L)):
        f, k = 1 / (1 + torch.exp(-z[:, t])), 1 / (1 + torch.exp(z[:, t]))
        g = dh[:, t] + carry
        du[:, t] = k * g
        dz[:, t] = g * ((h[:, t - 1] if t else first) - u[:, t]) * f * k
        carry = f * g
    return dz, du, carry


def _exact_attn(s):
    c = s["c"]
    G = c["H"] // c["Hkv"]
    low, p, live = _ranges(c)
    bwd = c["dir"] == "bwd"
    outs = {k: torch.zeros_like(s[k], dtype=torch.float64) for k in (("q", "k", "v") if bwd else ("q",))}
    lse = torch.full((c["B"], c["H"], c["Lq"]), -math.inf, dtype=torch.float64, device=DEV)
    slopes = _slopes(c)
    j = torch.arange(c["Lk"], device=DEV)
    for b in range(c["B"]):
        lb, pb = (torch.from_numpy(x[b]).to(DEV)[:, None] for x in (low, p))
        hide = (j < lb) | (j > pb) | ~torch.from_numpy(live[b]).to(DEV)
        empty = hide.all(1)
        for h in range(c["H"]):
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, h // G].double(), s["v"][b, :, h // G].double()
            x = q @ k.T / math.sqrt(c["D"])
            if c["cap"]:
                th = torch.tanh(x / c["cap"])
                x = th * c["cap"]
            if c["bias"]:
                x -= float(slopes[h]) * (pb - j)
            x[hide] = -math.inf
            if not bwd:
                lse[b, h] = torch.logsumexp(x, 1)
                pr = torch.exp(x - torch.where(empty, 0.0, lse[b, h])[:, None])
                outs["q"][b, :, h] = pr @ v
                continue
            do = s["do"][b, :, h].double()
            pr = torch.exp(x - torch.where(empty, 0.0, s["lse"][b, h].double())[:, None])
            g = pr * (do @ v.T - (do * s["o"][b, :, h].double()).sum(1, keepdim=True))
            if c["cap"]:
                g *= 1 - th ** 2
            g /= math.sqrt(c["D"])
            outs["q"][b, :, h] = g @ k
            outs["k"][b, :, h // G] += g.T @ q
            outs["v"][b, :, h // G] += pr.T @ do
    if bwd:
        return tuple(outs[k].contiguous() for k in ("q", "k", "v"))
    return outs["q"].contiguous(), lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "rec": _exact_rec, "attn": _exact_attn}[case["op"]](s)
