// Host layer of the calls on heads: norm and rotation of q and k, the 8-bit cache and attention over
// it.  Argument checks, workspaces and launches behind the C ABI declared in include/specconv.h.
#include "specconv.h"

#include <algorithm>
#include <climits>
#include <cmath>

#include "sc_checks.h"
#include "sc_internal.h"

namespace {

using namespace sc::checks;

Array flat(const void* p, int64_t n, int64_t es) { return rows_of(p, 1, n, n, es); }

// ------------------------------------------------------------------ norm and rotation

constexpr int64_t kMaxHead = 512;

// A (batch, token, head) tensor whose rows may start anywhere.
bool loose(const Tensor& t)
{
    const int64_t n[3] = {t.B, t.L, t.H};
    __int128 all = t.D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] < 2) continue;
        if (t.s[i] < 0 || t.s[i] > INT64_MAX / 16) return false;
        all += (__int128)(n[i] - 1) * t.s[i];
    }
    return t.p && (uintptr_t)t.p % t.es == 0 && all * t.es <= (__int128)INT64_MAX;
}

bool vectors(const Tensor& t)
{
    const int64_t n[3] = {t.B, t.L, t.H};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && t.s[i] * t.es % 16) return false;
    return (uintptr_t)t.p % 16 == 0;
}

bool same(const Tensor& x, const Tensor& y)
{
    const int64_t n[3] = {x.B, x.L, x.H};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && x.s[i] != y.s[i]) return false;
    return x.p == y.p;
}

// *empty: no rows (the backward call still writes dw).
sc_status qk_shape(sc_kind kind, const sc_qk* a, sc::QkArgs* x, bool* empty)
{
    if (!a || !float_kind(kind)) return SC_ERR_INVALID_ARGUMENT;
    if (a->B < 0 || a->L < 0 || a->H < 0 || a->Hkv < 0 || a->D < 0 || a->R < 0 || a->R > a->D || a->R % 2)
        return SC_ERR_INVALID_ARGUMENT;
    if (!(a->eps >= 0.f) || std::isinf(a->eps) || (a->interleaved != 0 && a->interleaved != 1)) return SC_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->inv_freq | (uintptr_t)a->positions | (uintptr_t)a->kv_len) % 4) return SC_ERR_INVALID_ARGUMENT;
    if (a->positions && a->kv_len) return SC_ERR_INVALID_ARGUMENT;
    if ((__int128)a->B * a->L > kMaxDim * 64 || a->L > kMaxDim) return SC_ERR_UNSUPPORTED;
    if (a->D > kMaxHead || a->H > kMaxDim / 256 || a->Hkv > kMaxDim / 256) return SC_ERR_UNSUPPORTED;
    *empty = a->B * a->L == 0 || a->H + a->Hkv == 0 || a->D == 0;
    if (!*empty && a->R > 0 && !a->inv_freq) return SC_ERR_INVALID_ARGUMENT;
    *x = sc::QkArgs{};
    x->B = a->B;
    x->L = a->L;
    x->tokens = *empty ? 0 : a->B * a->L;
    x->H[0] = (int)a->H;
    x->H[1] = (int)a->Hkv;
    x->D = (int)a->D;
    x->R = (int)a->R;
    x->eps = a->eps;
    x->pairs = a->interleaved;
    x->freq = a->inv_freq;
    x->pos = a->positions;
    x->len = a->kv_len;
    return SC_OK;
}

sc_status qk_run(sc_kind kind, const sc_qk* a, const void* q, const void* k, const void* wq, const void* wk,
                 void* qo, void* ko, hipStream_t stream)
{
    sc::QkArgs x;
    bool empty;
    sc_status st = qk_shape(kind, a, &x, &empty);
    if (st != SC_OK || empty) return st;
    const int64_t es = elt(kind);
    const Tensor in[2] = {{q, a->q, a->B, a->L, a->H, a->D, es}, {k, a->k, a->B, a->L, a->Hkv, a->D, es}};
    const Tensor out[2] = {{qo, a->q_out, a->B, a->L, a->H, a->D, es}, {ko, a->k_out, a->B, a->L, a->Hkv, a->D, es}};
    const void* w[2] = {wq, wk};
    const Array none = rows_of(nullptr, 0, 0, 0, 1);
    Array src[2] = {none, none}, dst[2] = {none, none};
    x.whole = true;
    for (int i = 0; i < 2; ++i) {
        if ((uintptr_t)w[i] % es) return SC_ERR_INVALID_ARGUMENT;
        if (in[i].H == 0) continue;
        if (!loose(in[i]) || !loose(out[i]) || !out[i].distinct()) return SC_ERR_INVALID_ARGUMENT;
        src[i] = in[i].array();
        dst[i] = out[i].array();
        x.whole = x.whole && vectors(in[i]) && vectors(out[i]) && (uintptr_t)w[i] % 16 == 0;
        x.x[i] = in[i].p;
        x.y[i] = const_cast<void*>(out[i].p);
        x.w[i] = w[i];
        std::copy(in[i].s, in[i].s + 3, x.xs[i]);
        std::copy(out[i].s, out[i].s + 3, x.ys[i]);
    }
    // a result may take the very place of its input: a row is read before it is written
    const int64_t np = a->positions ? a->B * a->L : 0, nl = a->kv_len ? a->B : 0;
    for (int i = 0; i < 2; ++i) {
        const bool place = in[i].H > 0 && same(in[i], out[i]);
        const Array others[] = {place ? none : src[i], src[1 - i], flat(wq, a->D, es), flat(wk, a->D, es),
                                flat(a->inv_freq, a->R / 2, 4), flat(a->positions, np, 4), flat(a->kv_len, nl, 4)};
        const Array mine[] = {dst[i]};
        if (!apart(others, mine)) return SC_ERR_INVALID_ARGUMENT;
    }
    if (share(dst[0], dst[1])) return SC_ERR_INVALID_ARGUMENT;
    return of(sc::launch_qk(store(kind), x, stream));
}

sc_status qk_bwd_run(sc_kind kind, const sc_qk* a, const void* dqo, const void* dko, const void* q, const void* k,
                     const void* wq, const void* wk, void* dq, void* dk, void* dwq, void* dwk, void* ws,
                     size_t ws_bytes, hipStream_t stream)
{
    sc::QkArgs x;
    bool empty;
    sc_status st = qk_shape(kind, a, &x, &empty);
    if (st != SC_OK) return st;
    if (a->D == 0 || (empty && !dwq && !dwk)) return SC_OK;
    const int64_t es = elt(kind);
    const Tensor in[2] = {{q, a->q, a->B, a->L, a->H, a->D, es}, {k, a->k, a->B, a->L, a->Hkv, a->D, es}};
    const Tensor g[2] = {{dqo, a->q_out, a->B, a->L, a->H, a->D, es}, {dko, a->k_out, a->B, a->L, a->Hkv, a->D, es}};
    const Tensor out[2] = {{dq, a->dq, a->B, a->L, a->H, a->D, es}, {dk, a->dk, a->B, a->L, a->Hkv, a->D, es}};
    const void* w[2] = {wq, wk};
    void* dw[2] = {dwq, dwk};
    const Array none = rows_of(nullptr, 0, 0, 0, 1);
    Array src[2] = {none, none}, grad[2] = {none, none}, dst[2] = {none, none};
    x.whole = true;
    for (int i = 0; i < 2; ++i) {
        if (((uintptr_t)w[i] | (uintptr_t)dw[i]) % es) return SC_ERR_INVALID_ARGUMENT;
        x.dw[i] = dw[i];
        if (empty || in[i].H == 0) continue;
        if (!loose(in[i]) || !loose(g[i]) || !loose(out[i]) || !out[i].distinct()) return SC_ERR_INVALID_ARGUMENT;
        src[i] = in[i].array();
        grad[i] = g[i].array();
        dst[i] = out[i].array();
        x.whole = x.whole && vectors(in[i]) && vectors(g[i]) && vectors(out[i]) && (uintptr_t)w[i] % 16 == 0;
        x.x[i] = in[i].p;
        x.dy[i] = g[i].p;
        x.y[i] = const_cast<void*>(out[i].p);
        x.w[i] = w[i];
        std::copy(in[i].s, in[i].s + 3, x.xs[i]);
        std::copy(g[i].s, g[i].s + 3, x.dys[i]);
        std::copy(out[i].s, out[i].s + 3, x.ys[i]);
    }
    const size_t need = dwq || dwk ? sc::qk_bwd_bytes(store(kind), x) : 0;
    const int64_t np = a->positions ? a->B * a->L : 0, nl = a->kv_len ? a->B : 0;
    const Array ins[] = {src[0], src[1], grad[0], grad[1], flat(wq, a->D, es), flat(wk, a->D, es),
                         flat(a->inv_freq, a->R / 2, 4), flat(a->positions, np, 4), flat(a->kv_len, nl, 4)};
    const Array outs[] = {dst[0], dst[1], flat(dwq, a->D, es), flat(dwk, a->D, es), flat(ws, (int64_t)need, 1)};
    if (!apart(ins, outs)) return SC_ERR_INVALID_ARGUMENT;
    return with_ws(need, ws, ws_bytes, stream, [&](void* p) { return of(sc::launch_qk_bwd(store(kind), x, p, stream)); });
}

// ------------------------------------------------------------------ the cache

bool code_ok(int32_t c) { return c == SC_CODE_I8 || c == SC_CODE_E4M3; }
sc::Code code_of(const sc_cache* c) { return c->code == SC_CODE_I8 ? sc::Code::I8 : sc::Code::E4M3; }

struct CacheArrays {
    Array k, v, ks, vs, table;
};

// *held: there is a block that a row can have.
sc_status cache_shape(const sc_cache* c, sc::CacheArgs* x, CacheArrays* arrays, bool* held)
{
    if (!c || !code_ok(c->code)) return SC_ERR_INVALID_ARGUMENT;
    if (c->B < 0 || c->N < 0 || c->P < 0 || c->Hkv < 0 || c->D < 0) return SC_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)c->k | (uintptr_t)c->v) % 16 || ((uintptr_t)c->k_scale | (uintptr_t)c->v_scale | (uintptr_t)c->table) % 4)
        return SC_ERR_INVALID_ARGUMENT;
    if (c->D % 16 || c->D > 128) return SC_ERR_UNSUPPORTED;
    if (c->N > kMaxDim / SC_CACHE_BLOCK || c->P > INT32_MAX || (__int128)c->B * std::max<int64_t>(c->Hkv, 1) > INT32_MAX)
        return SC_ERR_UNSUPPORTED;
    const __int128 bytes = (__int128)c->P * c->Hkv * SC_CACHE_BLOCK * c->D;
    if (bytes > (__int128)INT64_MAX) return SC_ERR_INVALID_ARGUMENT;
    if (!c->table && (__int128)c->B * c->N > c->P) return SC_ERR_INVALID_ARGUMENT;
    *held = c->B > 0 && c->N > 0 && c->P > 0 && c->Hkv > 0 && c->D > 0;
    if (*held && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return SC_ERR_INVALID_ARGUMENT;
    *x = sc::CacheArgs{c->k, c->v, c->k_scale, c->v_scale, c->table, (int)c->B, *held ? (int)c->N : 0, (int)c->P,
                       (int)c->Hkv, (int)c->D};
    const int64_t n = *held ? (int64_t)bytes : 0, s = *held ? c->P * c->Hkv : 0;
    *arrays = {flat(c->k, n, 1), flat(c->v, n, 1), flat(c->k_scale, s, 4), flat(c->v_scale, s, 4),
               flat(c->table, *held ? c->B * c->N : 0, 4)};
    return SC_OK;
}

sc_status cache_run(sc_kind kind, const sc_cache* c, const void* k, const int64_t* ks, const void* v,
                    const int64_t* vs, int64_t L, const int32_t* len, bool put, hipStream_t stream)
{
    if (!float_kind(kind) || L < 0 || !ks || !vs) return SC_ERR_INVALID_ARGUMENT;
    sc::CacheArgs x;
    CacheArrays ca;
    bool held;
    sc_status st = cache_shape(c, &x, &ca, &held);
    if (st != SC_OK) return st;
    if (L > kMaxDim) return SC_ERR_UNSUPPORTED;
    if (c->B == 0 || c->Hkv == 0 || c->D == 0 || L == 0) return SC_OK;
    const int64_t es = elt(kind);
    const Tensor tk{k, ks, c->B, L, c->Hkv, c->D, es}, tv{v, vs, c->B, L, c->Hkv, c->D, es};
    if (!tk.ok() || !tv.ok() || !len || (uintptr_t)len % 4) return SC_ERR_INVALID_ARGUMENT;
    if (!put && (!tk.distinct() || !tv.distinct())) return SC_ERR_INVALID_ARGUMENT;
    const Array l = flat(len, c->B, 4);
    bool ok;
    if (put) {
        const Array in[] = {tk.array(), tv.array(), l, ca.table}, out[] = {ca.k, ca.v, ca.ks, ca.vs};
        ok = apart(in, out);
    } else {
        const Array in[] = {ca.k, ca.v, ca.ks, ca.vs, l, ca.table}, out[] = {tk.array(), tv.array()};
        ok = apart(in, out);
    }
    if (!ok) return SC_ERR_INVALID_ARGUMENT;
    if (put && !held) return SC_OK;
    sc::CacheIo io{};
    if (put) {
        io.k = k;
        io.v = v;
    } else {
        io.ko = const_cast<void*>(k);
        io.vo = const_cast<void*>(v);
    }
    std::copy(ks, ks + 3, io.kst);
    std::copy(vs, vs + 3, io.vst);
    io.len = len;
    io.L = (int)L;
    return of(put ? sc::launch_cache_write(store(kind), code_of(c), x, io, stream)
                  : sc::launch_cache_read(store(kind), code_of(c), x, io, stream));
}

// ------------------------------------------------------------------ attention over it

struct Attn8 {
    sc::AttnArgs a;
    sc::CacheArgs c;
    CacheArrays arrays;
    int sinks;
    bool empty;
};

sc_status attn8_shape(sc_kind kind, const sc_cache* c, const sc_cached* q, Attn8* x)
{
    if (!q || !float_kind(kind)) return SC_ERR_INVALID_ARGUMENT;
    bool held;
    sc_status st = cache_shape(c, &x->c, &x->arrays, &held);
    if (st != SC_OK) return st;
    if (q->Lq < 0 || q->H < 0 || q->window < 0 || q->sinks < 0) return SC_ERR_INVALID_ARGUMENT;
    if (!(q->scale > 0.f) || std::isinf(q->scale) || !(q->cap >= 0.f) || std::isinf(q->cap)) return SC_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)q->slopes | (uintptr_t)q->kv_len) % 4) return SC_ERR_INVALID_ARGUMENT;
    x->empty = c->B == 0 || c->D == 0 || q->H == 0 || q->Lq == 0;
    if (x->empty) return SC_OK;
    if (c->Hkv == 0 || q->H % c->Hkv) return SC_ERR_UNSUPPORTED;
    const int64_t G = q->H / c->Hkv;
    if (G > kMaxDim || q->Lq > kMaxDim / G) return SC_ERR_UNSUPPORTED;
    sc::AttnArgs& a = x->a;
    a = sc::AttnArgs{};
    a.B = (int)c->B;
    a.H = (int)q->H;
    a.Hkv = (int)c->Hkv;
    a.G = (int)G;
    a.D = (int)c->D;
    a.Lq = (int)q->Lq;
    a.Lk = held ? (int)(c->N * SC_CACHE_BLOCK) : 0;
    a.scale = q->scale;
    a.cap = q->cap;
    a.window = q->window == 0 || q->window > INT_MAX ? INT_MAX : (int)q->window;
    a.slopes = q->slopes;
    a.kv_len = q->kv_len;
    a.nrow = (int)(q->Lq * G);
    a.nbh = (int)(c->B * c->Hkv);
    std::copy(q->q, q->q + 3, a.qs);
    std::copy(q->o, q->o + 3, a.os);
    x->sinks = (int)std::min<int64_t>(q->sinks, kMaxDim);
    return SC_OK;
}

sc_status attn8_run(sc_kind kind, const sc_cache* c, const sc_cached* p, const void* q, void* o, float* lse, void* ws,
                    size_t ws_bytes, hipStream_t stream)
{
    Attn8 x;
    sc_status st = attn8_shape(kind, c, p, &x);
    if (st != SC_OK || x.empty) return st;
    const int64_t es = elt(kind), nl = c->B * p->H * p->Lq;
    const Tensor tq{q, p->q, c->B, p->Lq, p->H, c->D, es}, to{o, p->o, c->B, p->Lq, p->H, c->D, es};
    if (!tq.ok() || !to.ok() || !to.distinct() || !p->kv_len || (uintptr_t)lse % 4) return SC_ERR_INVALID_ARGUMENT;
    const size_t need = sc::cached_attn_bytes(x.a, x.sinks);
    const Array in[] = {tq.array(), x.arrays.k, x.arrays.v, x.arrays.ks, x.arrays.vs, x.arrays.table,
                        flat(p->slopes, p->H, 4), flat(p->kv_len, c->B, 4)};
    const Array out[] = {to.array(), flat(lse, nl, 4), flat(ws, (int64_t)need, 1)};
    if (!apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    x.a.q = q;
    x.a.o = o;
    x.a.lse = lse;
    return with_ws(need, ws, ws_bytes, stream, [&](void* w) {
        return of(sc::launch_cached_attn(store(kind), code_of(c), x.a, x.c, x.sinks, w, stream));
    });
}

}  // namespace

extern "C" {

sc_status sc_qk_norm_rotary(sc_kind kind, const sc_qk* a, const void* q, const void* k, const void* wq,
                            const void* wk, void* q_out, void* k_out, hipStream_t stream)
{
    return guarded([&] { return qk_run(kind, a, q, k, wq, wk, q_out, k_out, stream); });
}

size_t sc_qk_norm_rotary_workspace_bytes(sc_kind kind, const sc_qk* a)
{
    sc::QkArgs x;
    bool empty;
    if (qk_shape(kind, a, &x, &empty) != SC_OK || empty) return 0;
    return sc::qk_bwd_bytes(store(kind), x);
}

sc_status sc_qk_norm_rotary_bwd(sc_kind kind, const sc_qk* a, const void* dq_out, const void* dk_out, const void* q,
                                const void* k, const void* wq, const void* wk, void* dq, void* dk, void* dwq,
                                void* dwk, void* ws, size_t ws_bytes, hipStream_t stream)
{
    return guarded([&] {
        return qk_bwd_run(kind, a, dq_out, dk_out, q, k, wq, wk, dq, dk, dwq, dwk, ws, ws_bytes, stream);
    });
}

sc_status sc_cache_write(sc_kind kind, const sc_cache* c, const void* k, const int64_t k_strides[3], const void* v,
                         const int64_t v_strides[3], int64_t L, const int32_t* kv_len, hipStream_t stream)
{
    return guarded([&] { return cache_run(kind, c, k, k_strides, v, v_strides, L, kv_len, true, stream); });
}

sc_status sc_cache_read(sc_kind kind, const sc_cache* c, void* k, const int64_t k_strides[3], void* v,
                        const int64_t v_strides[3], int64_t L, const int32_t* kv_len, hipStream_t stream)
{
    return guarded([&] { return cache_run(kind, c, k, k_strides, v, v_strides, L, kv_len, false, stream); });
}

size_t sc_cached_attn_workspace_bytes(sc_kind kind, const sc_cache* c, const sc_cached* a)
{
    Attn8 x;
    if (attn8_shape(kind, c, a, &x) != SC_OK || x.empty) return 0;
    return sc::cached_attn_bytes(x.a, x.sinks);
}

sc_status sc_cached_attn(sc_kind kind, const sc_cache* c, const sc_cached* a, const void* q, void* o, float* lse,
                         void* ws, size_t ws_bytes, hipStream_t stream)
{
    return guarded([&] { return attn8_run(kind, c, a, q, o, lse, ws, ws_bytes, stream); });
}

}  // extern "C"
