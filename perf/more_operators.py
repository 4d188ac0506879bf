"""Cases that time the norm and rotation of queries and keys, the 8-bit cache and its attention.

``own`` false: plain torch forms in 32 bits, rounded once to the storage type; ``own`` true: the
calls of this package.  Shapes are those of the models the library's workloads stand for (12 and 16
heads of 64, contexts 1024, 4096 and 65536, attention window 256).

A cache holds 64 tokens of a head a block, at one scale: the smallest power of two that brings the
block's values into the code's range.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6
BLOCK = 64
LOW, HIGH = -60, 60   # exponents of a block's scale


# --------------------------------------------------------------------------- cases

def _qk(**k):
    c = {"op": "qk", "dir": "fwd", "type": "bf16", "B": 1, "L": 1, "H": 16, "Hkv": 16, "D": 64,
         "R": 64, "pairs": False, "pos": "row", "far": 0, "fused": False}
    c.update(k)
    return c


def _cache(**k):
    c = {"op": "cache", "type": "bf16", "code": "int8", "B": 1, "T": 1, "L": 1, "back": 1,
         "Hkv": 4, "D": 64, "ragged": False, "paged": False}
    c.update(k)
    return c


def _attn(**k):
    c = {"op": "attn", "type": "bf16", "code": "int8", "B": 1, "L": 1, "T": 1, "H": 16, "Hkv": 4,
         "D": 64, "window": 0, "sinks": 0, "cap": 0.0, "bias": False, "ragged": False,
         "paged": False}
    c.update(k)
    return c


def listed():
    return [
        # one new token of eight sequences far into their contexts: latency
        _qk(name="qk-step", B=8, L=1, Hkv=4, pos="len", far=60000),
        # the Medium model's forward pass, q and k columns of one projection
        _qk(name="qk-fwd-medium", B=8, L=4096, fused=True),
        # float32, an odd length, half of each head turned, neighbours as pairs, packed positions
        _qk(name="qk-fwd-odd", type="f32", B=2, L=1001, H=12, Hkv=12, R=32, pairs=True, pos="list",
            far=500000),
        # the Medium model's training step
        _qk(name="qk-bwd-medium", dir="bwd", B=8, L=4096, fused=True),
        # float32 training of shared key heads over a long prompt
        _qk(name="qk-bwd-long", dir="bwd", type="f32", B=1, L=8192, Hkv=4, D=128, R=128),
        # one token a sequence appended to a block that holds others, the block read back
        _cache(name="cache-step", B=8, T=4096, L=1, back=64, ragged=True),
        # the Medium model's prompts stored and read back
        _cache(name="cache-prompt", code="e4m3", B=8, T=4096, L=4096, back=4096, Hkv=16),
        # a part of a prompt that ends inside blocks of a shared pool, float32, heads of 128
        _cache(name="cache-part", type="f32", B=3, T=2501, L=777, back=1000, D=128, ragged=True,
               paged=True),
        # one new token a sequence over ragged long caches
        _attn(name="attn8-decode", B=8, T=65536, ragged=True),
        # decoding the Medium model's window layer, the first tokens kept visible
        _attn(name="attn8-window", code="e4m3", B=32, T=4096, Hkv=16, window=256, sinks=4,
              bias=True, ragged=True, paged=True),
        # the last quarter of a long prompt over all that is stored of it
        _attn(name="attn8-prompt", B=1, L=2048, T=8192, D=128),
        # a few proposed tokens checked at once, float32, capped scores, an odd length
        _attn(name="attn8-few", type="f32", code="e4m3", B=4, L=5, T=10007, H=12, Hkv=12, cap=30.0,
              ragged=True, paged=True),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "cache", "attn", "attn"])
    ty = rng.choice(["f32", "bf16"])
    code = rng.choice(["int8", "e4m3"])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    G = rng.choice([1, 1, 2, 3, 4, 8]) if Hkv <= 8 else 1
    B = _size(rng, 1, 8)
    if op == "qk":
        D = rng.choice([64, 64, 128, 40, 80, 96])
        R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        top = max(1, min(65536, (1 << 25) // (B * Hkv * (G + 1) * D)))
        return _qk(dir=rng.choice(["fwd", "bwd"]), type=ty, B=B, L=_size(rng, 1, top), H=Hkv * G,
                   Hkv=Hkv, D=D, R=R, pairs=rng.random() < 0.4, pos=rng.choice(["row", "len", "list"]),
                   far=rng.choice([0, _size(rng, 1, 1 << 20)]), fused=rng.random() < 0.5)
    D = rng.choice([64, 64, 128, 32, 80, 96])
    ragged, paged = rng.random() < 0.6, rng.random() < 0.5
    if op == "cache":
        T = _size(rng, 1, min(65536, (1 << 24) // (B * Hkv * D)))
        L = 1 if rng.random() < 0.2 else _size(rng, 1, T)
        return _cache(type=ty, code=code, B=B, T=T, L=L, back=_size(rng, 1, T), Hkv=Hkv, D=D,
                      ragged=ragged, paged=paged)
    opt = dict(type=ty, code=code, B=B, H=Hkv * G, Hkv=Hkv, D=D, ragged=ragged, paged=paged,
               window=rng.choice([0, 256, _size(rng, 1, 1024)]), cap=rng.choice([0.0, 0.0, 30.0]),
               sinks=rng.choice([0, 4, _size(rng, 1, 200)]), bias=rng.random() < 0.5)
    if rng.random() < 0.6:   # few new tokens over a long cache
        T = min(262144, _size(rng, 1, max(1, (1 << 26) // (B * Hkv * D))))
        return _attn(T=T, L=1 if rng.random() < 0.6 else _size(rng, 1, min(T, 64)), **opt)
    T = _size(rng, 1, min(8192, int(math.sqrt((1 << 28) / (B * Hkv * G)))))
    return _attn(T=T, L=_size(rng, max(1, T // 8), T), **opt)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def _lens(c):
    return np.array([max(min(c["L"], c["T"]), c["T"] - (b * c["T"]) // (2 * c["B"]))
                     if c["ragged"] else c["T"] for b in range(c["B"])], np.int32)


def _tokens(c, gen):
    """k and v (B, T, Hkv, D), the last token of each row its newest: keys with a few large
    channels, as projections have, values without."""
    shape = c["B"], c["T"], c["Hkv"], c["D"]
    wide = torch.randn(c["Hkv"], c["D"], generator=gen, device=DEV).mul_(0.5).exp_()
    k = torch.randn(*shape, generator=gen, device=DEV).mul_(wide).to(DT[c["type"]])
    return k, torch.randn(*shape, generator=gen, device=DEV).to(DT[c["type"]])


def _inv_freq(c):
    return torch.from_numpy(10000.0 ** (-2.0 * np.arange(c["R"] // 2) / max(c["R"], 1))).float().to(DEV)


def _positions(c):
    """(positions, kv_len) of a qk case: where each token stands."""
    if c["pos"] == "list":   # documents packed behind each other
        step = max(1, c["L"] // 3)
        p = (np.arange(c["L"]) % step)[None] + c["far"] + 7 * np.arange(c["B"])[:, None]
        return torch.from_numpy(p.astype(np.int32)).to(DEV), None
    if c["pos"] == "len":
        n = c["L"] + c["far"] + 31 * np.arange(c["B"])
        return None, torch.from_numpy(n.astype(np.int32)).to(DEV)
    return None, None


def _slopes(c):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / c["H"]) for h in range(c["H"])], device=DEV)


def prepare(case, seed):
    c, gen = case, _gen(seed)
    dt = DT[c["type"]]
    B, L = c["B"], c["L"]
    s = {"c": c}
    if c["op"] == "qk":
        H, Hkv, D = c["H"], c["Hkv"], c["D"]

        def both():
            x = torch.randn(B, L, H + 2 * Hkv if c["fused"] else H + Hkv, D, generator=gen, device=DEV)
            x = x.mul_(1.5).add_(0.2).to(dt)
            return x[:, :, :H], x[:, :, H:H + Hkv]
        s["q"], s["k"] = (x if c["fused"] else x.contiguous() for x in both())
        s["wq"], s["wk"] = (torch.randn(D, generator=gen, device=DEV).mul_(0.2).add_(1.0).to(dt) for _ in "qk")
        s["f"] = _inv_freq(c)
        s["pos"], s["n"] = _positions(c)
        if c["dir"] == "bwd":
            s["gq"], s["gk"] = (x.contiguous() for x in both())
        return s
    n = torch.from_numpy(_lens(c)).to(DEV)
    s["n"] = n
    N = -(-c["T"] // BLOCK)
    k, v = _tokens(c, gen)
    if c["op"] == "attn":
        s["q"] = torch.randn(B, L, c["H"], c["D"], generator=gen, device=DEV).to(dt)
        s["slopes"] = _slopes(c) if c["bias"] else None
        fresh = c["T"]   # everything is stored by one call
    else:
        s["k"], s["v"] = k[:, c["T"] - L:].contiguous(), v[:, c["T"] - L:].contiguous()
        fresh = c["T"] - L
        k, v, n = k[:, :fresh], v[:, :fresh], n - L
    table = None
    if c["paged"]:
        table = torch.randperm(B * N + 3, generator=gen, device=DEV)[:B * N].view(B, N).int()
    if own:
        import fft_causal_long_amd as sc
        s["cache"] = sc.KVCache(B, N * BLOCK, c["Hkv"], c["D"], c["code"],
                                device=DEV, blocks=B * N + 3 if c["paged"] else None, table=table)
        if fresh:
            sc.cache_write(s["cache"], k.contiguous(), v.contiguous(), n)
        return s
    for name, x in (("k", k), ("v", v)):
        at = torch.arange(N * BLOCK, device=DEV)[None] - n[:, None].long() + fresh   # token of a position
        full = torch.zeros(B, N * BLOCK, c["Hkv"], c["D"], device=DEV)
        if fresh:
            here = (at >= 0) & (at < fresh)
            rows = torch.arange(B, device=DEV)[:, None]
            full = torch.where(here[:, :, None, None], x[rows, at.clamp(0, fresh - 1)].float(), full)
        s["code_" + name], s["scale_" + name] = _quantise(full, c["code"])
    return s


# --------------------------------------------------------------------------- plain forms

def _angles(s, L):
    c = s["c"]
    if s["pos"] is not None:
        p = s["pos"].double()
    else:
        p = torch.arange(L, device=DEV, dtype=torch.float64)[None].expand(c["B"], L)
        if s["n"] is not None:
            p = p + (s["n"].double() - L)[:, None]
    a = p[:, :, None] * s["f"].double()
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _turn(c, x, cos, sin):
    R = c["R"]
    y = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if c["pairs"] else (slice(0, R // 2), slice(R // 2, R))
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def _qk_fwd(s):
    cos, sin = _angles(s, s["c"]["L"])
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x32 = x.float()
        y = x32 * (x32.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
        out.append(_turn(s["c"], y, cos, sin).to(x.dtype))
    return out


def _qk_bwd(s):
    cos, sin = _angles(s, s["c"]["L"])
    dx, dw = [], []
    for x, w, g in ((s["q"], s["wq"], s["gq"]), (s["k"], s["wk"], s["gk"])):
        x32 = x.float()
        r = (x32.square().mean(-1, keepdim=True) + EPS).rsqrt()
        e, xh = _turn(s["c"], g.float(), cos, -sin), x32 * r
        ew = e * w.float()
        dx.append(((ew - xh * (ew * xh).mean(-1, keepdim=True)) * r).to(x.dtype))
        dw.append((e * xh).flatten(0, 2).sum(0, dtype=torch.float64).to(x.dtype))
    return dx + dw


def _power(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _scale(top, code):
    """The smallest power of two that brings `top` to 127 or 448."""
    m, e = torch.frexp(top)
    e = e - 7 + (m > 127 / 128).int() if code == "int8" else e - 9 + (m > 0.875).int()
    return _power(torch.where(top > 0, e, LOW).clamp(LOW, HIGH))


def _round(x, code):
    if code == "int8":
        return torch.round(x).clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _each(scale):
    """(B, N, H) scales to (B, N * BLOCK, H, 1)."""
    return scale.repeat_interleave(BLOCK, 1)[..., None]


def _quantise(x, code):
    B, n, H, D = x.shape
    scale = _scale(x.view(B, n // BLOCK, BLOCK, H, D).abs().amax((2, 4)), code)
    return _round(x / _each(scale), code), scale


def _plain_cache(s):
    c = s["c"]
    B, L, cap = c["B"], c["L"], s["code_k"].shape[1]
    n = s["n"].long()
    rows = torch.arange(B, device=DEV)[:, None]
    base = (n - L).clamp(min=0) // BLOCK * BLOCK
    p = base[:, None] + torch.arange(-(-L // BLOCK) * BLOCK + BLOCK, device=DEV)   # the blocks that change
    there = p < cap
    new = there & (p >= (n - L)[:, None]) & (p < n[:, None])
    new4 = new[:, :, None, None]
    old = base < n - L
    pb = p[:, ::BLOCK] // BLOCK
    thereb = pb < cap // BLOCK
    out = []
    for name in "kv":
        code, scale = s["code_" + name], s["scale_" + name]
        x = torch.where(new4, s[name][rows, (p - (n - L)[:, None]).clamp(0, L - 1)].float(), 0.0)
        was = scale[rows, pb.clamp(max=cap // BLOCK - 1)]
        held = code[rows, p.clamp(max=cap - 1)].float()
        fresh = _scale(x.view(B, -1, BLOCK, c["Hkv"], c["D"]).abs().amax((2, 4)), c["code"])
        keeps = (old[:, None] & (torch.arange(pb.shape[1], device=DEV) == 0))[:, :, None]
        now = torch.where(keeps, torch.maximum(was, fresh), fresh)
        y = _round(torch.where(new4, x / _each(now), held * _each(was / now)), c["code"])
        touched = thereb & new.view(B, -1, BLOCK).any(2)
        t = touched.repeat_interleave(BLOCK, 1)
        bi, ti = t.nonzero(as_tuple=True)
        code[bi, p[bi, ti]] = y[bi, ti]
        bi, ti = touched.nonzero(as_tuple=True)
        scale[bi, pb[bi, ti]] = now[bi, ti]
        r = n[:, None] - c["back"] + torch.arange(c["back"], device=DEV)
        at = r.clamp(min=0)
        y = code[rows, at].float() * scale[rows, at // BLOCK][..., None]
        out.append(torch.where((r >= 0)[:, :, None, None], y, 0.0).to(DT[c["type"]]))
    return out


def _plain_attn(s):
    c = s["c"]
    G, cap, D = c["H"] // c["Hkv"], s["code_k"].shape[1], c["D"]
    n = s["n"].long()

    def heads(x, G=1):
        return x.float().repeat_interleave(G, 2).transpose(1, 2).contiguous()
    k, v = (heads(s["code_" + x].float() * _each(s["scale_" + x]), G) for x in "kv")
    x = (heads(s["q"]) @ k.transpose(-1, -2)) * D ** -0.5
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j = torch.arange(cap, device=DEV)
    p = (n[:, None] - c["L"] + torch.arange(c["L"], device=DEV))[:, :, None]
    see = j <= p
    if c["window"]:
        see &= (j > p - c["window"]) | (j < c["sinks"])
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (p - j)[:, None]
    x = x.masked_fill(~see[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(l > 0, l, 1.0)
    return o.transpose(1, 2).contiguous().to(s["q"].dtype), (m + torch.log(l))[..., 0]


def run(state):
    s = state
    c = s["c"]
    if not own:
        if c["op"] == "qk":
            return _qk_fwd(s) if c["dir"] == "fwd" else _qk_bwd(s)
        return _plain_cache(s) if c["op"] == "cache" else _plain_attn(s)
    import fft_causal_long_amd as sc
    if c["op"] == "qk":
        opt = dict(positions=s["pos"], kv_len=s["n"], interleaved=c["pairs"], eps=EPS)
        if c["dir"] == "fwd":
            return sc.qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["f"], **opt)
        return sc.qk_norm_rotary_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["f"], **opt)
    if c["op"] == "cache":
        sc.cache_write(s["cache"], s["k"], s["v"], s["n"])
        return sc.cache_read(s["cache"], c["back"], s["n"], DT[c["type"]])
    return sc.cached_attention(s["q"], s["cache"], s["n"], window=c["window"], sinks=c["sinks"],
                               cap=c["cap"], slopes=s["slopes"], lse=True)


# --------------------------------------------------------------------------- counts

def work(case):
    c = case
    e = 4 if c["type"] == "f32" else 2
    if c["op"] == "qk":
        n = c["B"] * c["L"] * (c["H"] + c["Hkv"]) * c["D"]
        side = 2 * c["D"] * e + 2 * c["R"] + (4 * c["B"] * c["L"] if c["pos"] == "list" else 0)
        if c["dir"] == "fwd":
            return {"bytes": 2 * n * e + side, "flops": 8 * n}
        return {"bytes": 3 * n * e + side + 2 * c["D"] * e, "flops": 16 * n}
    n = _lens(c).astype(np.int64)
    wide = 2 * c["Hkv"] * c["D"]   # k and v of a token
    if c["op"] == "cache":
        new, back = int(np.minimum(n, c["L"]).sum()), int(np.minimum(n, c["back"]).sum())
        return {"bytes": wide * (new * (e + 1) + back + c["B"] * c["back"] * e), "flops": 4 * wide * (new + back)}
    p = n[:, None] - c["L"] + np.arange(c["L"])
    low = np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p)
    pairs = int(np.where(p >= 0, p - low + 1 + np.minimum(c["sinks"] if c["window"] else 0, low), 0).sum())
    first = np.where(p >= 0, low, 1 << 40).min(1)
    keys = int((n - first + np.minimum(c["sinks"] if c["window"] else 0, first)).sum())
    rows = c["B"] * c["L"] * c["H"]
    return {"bytes": 2 * rows * c["D"] * e + 4 * rows + keys * wide + keys // BLOCK * 8 * c["Hkv"],
            "flops": 4 * c["D"] * pairs * c["H"]}


# --------------------------------------------------------------------------- 64 bits

def _exact_qk(s):
    c = s["c"]
    B, L, D, R = c["B"], c["L"], c["D"], c["R"]
    pos = torch.arange(L, device=DEV, dtype=torch.float64).repeat(B, 1)
    if s["n"] is not None:
        pos += s["n"].double().view(B, 1) - L
    if s["pos"] is not None:
        pos = s["pos"].double()
    theta = (pos.view(B, L, 1, 1) * s["f"].double().view(1, 1, 1, -1))
    z = torch.polar(torch.ones_like(theta), theta)

    def turn(x, z):
        a = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) if c["pairs"] else torch.complex(x[..., :R // 2], x[..., R // 2:R])
        a = a * z
        parts = torch.stack([a.real, a.imag], -1).flatten(-2) if c["pairs"] else torch.cat([a.real, a.imag], -1)
        return torch.cat([parts, x[..., R:]], -1)
    outs, sums = [], []
    for x, w in (("q", "wq"), ("k", "wk")):
        w, g = s[w].double(), s.get("g" + x)
        x = s[x].double()
        norm = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
        if g is None:
            outs.append(turn(norm * w, z))
            continue
        e = turn(g.double(), z.conj())
        inner = (e * w * norm).sum(-1, keepdim=True) / D
        outs.append((e * w - norm * inner) / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS))
        sums.append((e * norm).sum((0, 1, 2)))
    return outs + sums


def _exact_exponent(top, code):
    q = 127.0 if code == "int8" else 448.0
    e = torch.full(top.shape, LOW, dtype=torch.int64, device=DEV)
    for _ in range(HIGH - LOW):
        e = torch.where(top > q * _exact_power(e), e + 1, e)
    return e.clamp(max=HIGH)


def _exact_power(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_round(x, code):
    if code == "int8":
        return x.round().clamp(-127, 127)
    a = x.abs().clamp(max=448.0)
    k = torch.floor(torch.log2(a.clamp(min=2.0 ** -9))).to(torch.int64)
    k = torch.where(a >= _exact_power(k + 1), k + 1, torch.where(a < _exact_power(k), k - 1, k)).clamp(min=-6)
    step = _exact_power(k - 3)
    return torch.sign(x) * (a / step).round() * step


def _exact_blocks(x, code):
    """Rounds the blocks of x (n, H, D) in place; the exponents of the last one."""
    n = x.shape[0]
    full = torch.zeros(-(-n // BLOCK) * BLOCK, *x.shape[1:], dtype=torch.float64, device=DEV)
    full[:n] = x
    full = full.view(-1, BLOCK, *x.shape[1:])
    e = _exact_exponent(full.abs().amax((1, 3)), code)
    u = _exact_power(e)[:, None, :, None]
    x.copy_((_exact_round(full / u, code) * u).flatten(0, 1)[:n])
    return e[-1]


def _exact_store(x, upto, code):
    """What the tokens x (n, H, D) of a row stand for, those before `upto` stored by an earlier call."""
    x, n = x.double(), x.shape[0]
    if upto:
        e = _exact_blocks(x[:upto], code)
    if upto % BLOCK and upto < n:   # a block that both calls write: its scale can only grow
        first, last = upto // BLOCK * BLOCK, min(upto // BLOCK * BLOCK + BLOCK, n)
        u = _exact_power(torch.maximum(e, _exact_exponent(x[upto:last].abs().amax((0, 2)), code)))[:, None]
        x[first:last] = _exact_round(x[first:last] / u, code) * u
        upto = last
    if upto < n:
        _exact_blocks(x[upto:], code)
    return x


def _exact_cache(c, seed):
    gen = _gen(seed)
    n = _lens(c)
    out = []
    for x in _tokens(c, gen):
        y = torch.zeros(c["B"], c["back"], c["Hkv"], c["D"], dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            m = int(n[b])
            got = _exact_store(x[b, c["T"] - m:], m - min(c["L"], m), c["code"])
            keep = min(m, c["back"])
            y[b, c["back"] - keep:] = got[m - keep:]
        out.append(y)
    return out


def _exact_attn(c, seed):
    gen = _gen(seed)
    k, v = _tokens(c, gen)
    q = torch.randn(c["B"], c["L"], c["H"], c["D"], generator=gen, device=DEV).to(DT[c["type"]])
    G, n = c["H"] // c["Hkv"], _lens(c)
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["H"], c["L"]), -math.inf, dtype=torch.float64, device=DEV)
    slopes = _slopes(c).double()
    for b in range(c["B"]):
        m = int(n[b])
        kb, vb = (_exact_store(x[b, c["T"] - m:], m, c["code"]) for x in (k, v))
        j = torch.arange(m, device=DEV)
        p = torch.arange(m - c["L"], m, device=DEV)[:, None]
        hide = j > p
        if c["window"]:
            hide = hide | ((p - j >= c["window"]) & (j >= c["sinks"]))
        empty = hide.all(1)
        for h in range(c["H"]):
            x = q[b, :, h].double() @ kb[:, h // G].T / math.sqrt(c["D"])
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if c["bias"]:
                x = x - slopes[h] * (p - j)
            x[hide] = -math.inf
            lse[b, h] = torch.logsumexp(x, 1)
            o[b, :, h] = torch.exp(x - torch.where(empty, 0.0, lse[b, h])[:, None]) @ vb[:, h // G]
    return o, lse


def exact(case, seed):
    if case["op"] == "qk":
        return _exact_qk(prepare(case, seed))
    return _exact_cache(case, seed) if case["op"] == "cache" else _exact_attn(case, seed)
