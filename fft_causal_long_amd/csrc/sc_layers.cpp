// Host layer of the calls beside the convolution (layer norm, gated recurrence, attention):
// argument checks, workspaces and launches behind the C ABI declared in include/specconv.h.
#include "specconv.h"

#include <algorithm>
#include <climits>
#include <cmath>

#include "sc_checks.h"
#include "sc_internal.h"

namespace {

using namespace sc::checks;

// ------------------------------------------------------------------ layer norm

sc_status ln_shape(sc_kind kind, int64_t rows, int64_t C)
{
    if (!float_kind(kind) || rows < 0 || C < 0) return SC_ERR_INVALID_ARGUMENT;
    return C > kMaxDim ? SC_ERR_UNSUPPORTED : SC_OK;
}

sc_status ln_run(sc_kind kind, const void* x, const void* w, const void* b, void* y, float* mean,
                 float* rstd, int64_t rows, int64_t C, int64_t xs, int64_t ys, float eps,
                 hipStream_t stream)
{
    sc_status st = ln_shape(kind, rows, C);
    if (st != SC_OK) return st;
    if (xs < 0 || ys < C || !(eps >= 0.f) || std::isinf(eps)) return SC_ERR_INVALID_ARGUMENT;
    if (rows == 0 || C == 0) return SC_OK;
    const int64_t es = elt(kind);
    if (!x || !y || ((uintptr_t)x | (uintptr_t)y | (uintptr_t)w | (uintptr_t)b) % es ||
        ((uintptr_t)mean | (uintptr_t)rstd) % 4)
        return SC_ERR_INVALID_ARGUMENT;
    const Array in[] = {rows_of(x, rows, xs, C, es), rows_of(w, 1, C, C, es), rows_of(b, 1, C, C, es)};
    const Array out[] = {rows_of(y, rows, ys, C, es), rows_of(mean, 1, rows, rows, 4),
                         rows_of(rstd, 1, rows, rows, 4)};
    if (!fits(in[0]) || !fits(out[0]) || !apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    return of(sc::launch_layernorm(store(kind), x, w, b, y, mean, rstd, rows, (int)C, xs, ys, eps, stream));
}

sc_status ln_bwd_run(sc_kind kind, const void* dy, const void* x, const void* w, const float* mean,
                     const float* rstd, void* dx, void* dw, void* db, int64_t rows, int64_t C,
                     int64_t dys, int64_t xs, int64_t dxs, void* ws, size_t ws_bytes,
                     hipStream_t stream)
{
    sc_status st = ln_shape(kind, rows, C);
    if (st != SC_OK) return st;
    if (xs < 0 || dys < 0 || dxs < C) return SC_ERR_INVALID_ARGUMENT;
    if (C == 0 || (rows == 0 && !dw && !db)) return SC_OK;
    const int64_t es = elt(kind);
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return SC_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)dy | (uintptr_t)x | (uintptr_t)w | (uintptr_t)dx | (uintptr_t)dw | (uintptr_t)db) % es ||
        ((uintptr_t)mean | (uintptr_t)rstd) % 4)
        return SC_ERR_INVALID_ARGUMENT;
    const size_t need = dw || db ? sc::layernorm_bwd_bytes(store(kind), rows, (int)C) : 0;
    const Array in[] = {rows_of(dy, rows, dys, C, es), rows_of(x, rows, xs, C, es),
                        rows_of(w, 1, C, C, es), rows_of(mean, 1, rows, rows, 4),
                        rows_of(rstd, 1, rows, rows, 4)};
    const Array out[] = {rows_of(dx, rows, dxs, C, es), rows_of(dw, 1, C, C, es),
                         rows_of(db, 1, C, C, es), rows_of(ws, 1, (int64_t)need, (int64_t)need, 1)};
    if (!fits(in[0]) || !fits(in[1]) || !fits(out[0]) || !apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    return with_ws(need, ws, ws_bytes, stream, [&](void* p) {
        return of(sc::launch_layernorm_bwd(store(kind), dy, x, w, mean, rstd, dx, dw, db, rows, (int)C,
                                           dys, xs, dxs, p, stream));
    });
}

// ------------------------------------------------------------------ gated recurrence

sc_status recur_shape(sc_kind kind, int64_t B, int64_t L, int64_t C)
{
    if (!float_kind(kind) || B < 0 || L < 0 || C < 0) return SC_ERR_INVALID_ARGUMENT;
    if ((__int128)B * L * C * 4 > (__int128)INT64_MAX || (__int128)B * C * 4 > (__int128)INT64_MAX)
        return SC_ERR_INVALID_ARGUMENT;
    return C > kMaxDim || B > INT32_MAX ? SC_ERR_UNSUPPORTED : SC_OK;
}

// the state of an empty sequence: dst = src, or zero
sc_status copy_state(const float* src, float* dst, int64_t n, hipStream_t stream)
{
    if (!dst || dst == src || n == 0) return SC_OK;
    if (!src) return of(sc::launch_zero16(dst, n * 2, stream));
    return hipMemcpyAsync(dst, src, (size_t)n * 4, hipMemcpyDeviceToDevice, stream) == hipSuccess ? SC_OK
                                                                                                 : SC_ERR_HIP;
}

sc_status recur_run(sc_kind kind, const void* z, const void* u, const float* h0, void* h, float* hT,
                    int64_t B, int64_t L, int64_t C, int64_t zs, int64_t us, int64_t hs, void* ws,
                    size_t ws_bytes, hipStream_t stream)
{
    sc_status st = recur_shape(kind, B, L, C);
    if (st != SC_OK) return st;
    if (zs < 0 || us < 0 || hs < C) return SC_ERR_INVALID_ARGUMENT;
    if (B == 0 || C == 0) return SC_OK;
    const int64_t es = elt(kind), R = B * L;
    if (((uintptr_t)h0 | (uintptr_t)hT) % 4) return SC_ERR_INVALID_ARGUMENT;
    const size_t need = sc::recur_bytes(B, L, (int)C);
    const Array same = rows_of(h0 == hT ? nullptr : h0, 1, B * C, B * C, 4);
    const Array in[] = {rows_of(z, R, zs, C, es), rows_of(u, R, us, C, es), same};
    const Array out[] = {rows_of(h, R, hs, C, es), rows_of(hT, 1, B * C, B * C, 4),
                         rows_of(ws, 1, (int64_t)need, (int64_t)need, 1)};
    if (L > 0 && (!z || !u || !h || ((uintptr_t)z | (uintptr_t)u | (uintptr_t)h) % es))
        return SC_ERR_INVALID_ARGUMENT;
    if (!fits(in[0]) || !fits(in[1]) || !fits(out[0]) || !apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    // h0 with hT the same memory: still apart from h and ws
    if (share(rows_of(h0, 1, B * C, B * C, 4), out[0]) || share(rows_of(h0, 1, B * C, B * C, 4), out[2]))
        return SC_ERR_INVALID_ARGUMENT;
    if (L == 0) return copy_state(h0, hT, B * C, stream);
    sc::RecurFwd r{z, u, h, h0, hT, zs, us, hs,
                   aligned(z, zs, es) && aligned(u, us, es) && aligned(h, hs, es)};
    return with_ws(need, ws, ws_bytes, stream,
                   [&](void* p) { return of(sc::launch_recur(store(kind), r, B, L, (int)C, p, stream)); });
}

sc_status recur_bwd_run(sc_kind kind, const void* dh, const void* z, const void* u, const void* h,
                        const float* h0, const float* dhT, void* dz, void* du, float* dh0, int64_t B,
                        int64_t L, int64_t C, const int64_t (&s)[6], void* ws, size_t ws_bytes,
                        hipStream_t stream)
{
    sc_status st = recur_shape(kind, B, L, C);
    if (st != SC_OK) return st;
    if (s[0] < 0 || s[1] < 0 || s[2] < 0 || s[3] < 0 || s[4] < C || s[5] < C) return SC_ERR_INVALID_ARGUMENT;
    if (B == 0 || C == 0) return SC_OK;
    const int64_t es = elt(kind), R = B * L, n = B * C;
    if (((uintptr_t)h0 | (uintptr_t)dhT | (uintptr_t)dh0) % 4) return SC_ERR_INVALID_ARGUMENT;
    if (L > 0) {
        const void* all[] = {dh, z, u, h, dz, du};
        for (const void* p : all)
            if (!p || (uintptr_t)p % es) return SC_ERR_INVALID_ARGUMENT;
    }
    const size_t need = sc::recur_bytes(B, L, (int)C);
    const Array in[] = {rows_of(dh, R, s[0], C, es), rows_of(z, R, s[1], C, es),
                        rows_of(u, R, s[2], C, es), rows_of(h, R, s[3], C, es),
                        rows_of(h0, 1, n, n, 4), rows_of(dhT == dh0 ? nullptr : dhT, 1, n, n, 4)};
    const Array out[] = {rows_of(dz, R, s[4], C, es), rows_of(du, R, s[5], C, es),
                         rows_of(dh0, 1, n, n, 4), rows_of(ws, 1, (int64_t)need, (int64_t)need, 1)};
    for (const Array& a : in)
        if (!fits(a)) return SC_ERR_INVALID_ARGUMENT;
    if (!fits(out[0]) || !fits(out[1]) || !apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    const Array last = rows_of(dhT, 1, n, n, 4);
    if (share(last, out[0]) || share(last, out[1]) || share(last, out[3])) return SC_ERR_INVALID_ARGUMENT;
    if (L == 0) return copy_state(dhT, dh0, n, stream);
    sc::RecurBwd r{dh, z, u, h, dz, du, h0, dhT, dh0, s[0], s[1], s[2], s[3], s[4], s[5],
                   aligned(dh, s[0], es) && aligned(z, s[1], es) && aligned(u, s[2], es) &&
                       aligned(h, s[3], es) && aligned(dz, s[4], es) && aligned(du, s[5], es)};
    return with_ws(need, ws, ws_bytes, stream, [&](void* p) {
        return of(sc::launch_recur_bwd(store(kind), r, B, L, (int)C, p, stream));
    });
}

// ------------------------------------------------------------------ attention

// Shape checks; *x receives everything but the pointers.  *empty: no output to write (the backward
// call without query heads still writes dk and dv).
sc_status attn_shape(sc_kind kind, const sc_attn* a, bool backward, sc::AttnArgs* x, bool* empty)
{
    if (!a || !float_kind(kind)) return SC_ERR_INVALID_ARGUMENT;
    if (a->B < 0 || a->Lq < 0 || a->Lk < 0 || a->H < 0 || a->Hkv < 0 || a->D < 0 || a->window < 0)
        return SC_ERR_INVALID_ARGUMENT;
    if (!(a->scale > 0.f) || std::isinf(a->scale) || !(a->cap >= 0.f) || std::isinf(a->cap))
        return SC_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->slopes | (uintptr_t)a->kv_len | (uintptr_t)a->doc_start) % 4)
        return SC_ERR_INVALID_ARGUMENT;
    *empty = a->B == 0 || a->D == 0 || (a->H == 0 && (!backward || a->Hkv == 0));
    if (*empty) return SC_OK;
    if (a->Hkv == 0 || a->H % a->Hkv) return SC_ERR_UNSUPPORTED;
    if (a->D % 8 || a->D > 128) return SC_ERR_UNSUPPORTED;
    const int64_t G = a->H / a->Hkv;
    if (a->Lk > kMaxDim || a->Lq > kMaxDim / std::max<int64_t>(G, 1) || G > kMaxDim) return SC_ERR_UNSUPPORTED;
    if ((__int128)a->B * a->Hkv > (__int128)INT32_MAX) return SC_ERR_UNSUPPORTED;
    *x = sc::AttnArgs{};
    x->B = (int)a->B;
    x->H = (int)a->H;
    x->Hkv = (int)a->Hkv;
    x->G = (int)G;
    x->D = (int)a->D;
    x->Lq = (int)a->Lq;
    x->Lk = (int)a->Lk;
    x->scale = a->scale;
    x->cap = a->cap;
    x->window = a->window == 0 || a->window > INT_MAX ? INT_MAX : (int)a->window;
    x->slopes = a->slopes;
    x->kv_len = a->kv_len;
    x->doc = a->doc_start;
    x->nrow = (int)(a->Lq * G);
    x->nbh = (int)(a->B * a->Hkv);
    for (int i = 0; i < 3; ++i) {
        x->qs[i] = a->q[i];
        x->ks[i] = a->k[i];
        x->vs[i] = a->v[i];
        x->os[i] = a->o[i];
        x->dos[i] = a->dout[i];
        x->dqs[i] = a->dq[i];
        x->dks[i] = a->dk[i];
        x->dvs[i] = a->dv[i];
    }
    return SC_OK;
}

sc_status attn_run(sc_kind kind, const sc_attn* a, const void* q, const void* k, const void* v,
                   void* o, float* lse, void* ws, size_t ws_bytes, hipStream_t stream)
{
    sc::AttnArgs x;
    bool empty;
    sc_status st = attn_shape(kind, a, false, &x, &empty);
    if (st != SC_OK) return st;
    if (empty || a->Lq == 0) return SC_OK;
    const int64_t es = elt(kind);
    const Tensor tq{q, a->q, a->B, a->Lq, a->H, a->D, es}, to{o, a->o, a->B, a->Lq, a->H, a->D, es};
    const Tensor tk{k, a->k, a->B, a->Lk, a->Hkv, a->D, es}, tv{v, a->v, a->B, a->Lk, a->Hkv, a->D, es};
    if (!tq.ok() || !to.ok() || !to.distinct() || (a->Lk > 0 && (!tk.ok() || !tv.ok())) || (uintptr_t)lse % 4)
        return SC_ERR_INVALID_ARGUMENT;
    const size_t need = sc::attn_fwd_bytes(x);
    const int64_t nl = a->B * a->H * a->Lq;
    const Array none = rows_of(nullptr, 0, 0, 0, 1);
    const Array in[] = {tq.array(), a->Lk ? tk.array() : none, a->Lk ? tv.array() : none,
                        rows_of(a->slopes, 1, a->H, a->H, 4), rows_of(a->kv_len, 1, a->B, a->B, 4),
                        rows_of(a->doc_start, 1, a->B * a->Lk, a->B * a->Lk, 4)};
    const Array out[] = {to.array(), rows_of(lse, 1, nl, nl, 4),
                         rows_of(ws, 1, (int64_t)need, (int64_t)need, 1)};
    if (!apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    x.q = q;
    x.k = k;
    x.v = v;
    x.o = o;
    x.lse = lse;
    return with_ws(need, ws, ws_bytes, stream,
                   [&](void* p) { return of(sc::launch_attn(store(kind), x, p, stream)); });
}

sc_status attn_bwd_run(sc_kind kind, const sc_attn* a, const void* dout, const void* q, const void* k,
                       const void* v, const void* o, const float* lse, void* dq, void* dk, void* dv,
                       void* ws, size_t ws_bytes, hipStream_t stream)
{
    sc::AttnArgs x;
    bool empty;
    sc_status st = attn_shape(kind, a, true, &x, &empty);
    if (st != SC_OK) return st;
    if (empty || ((a->Lq == 0 || a->H == 0) && a->Lk == 0)) return SC_OK;
    const int64_t es = elt(kind);
    const Tensor tq{q, a->q, a->B, a->Lq, a->H, a->D, es}, to{o, a->o, a->B, a->Lq, a->H, a->D, es};
    const Tensor tg{dout, a->dout, a->B, a->Lq, a->H, a->D, es}, tdq{dq, a->dq, a->B, a->Lq, a->H, a->D, es};
    const Tensor tk{k, a->k, a->B, a->Lk, a->Hkv, a->D, es}, tv{v, a->v, a->B, a->Lk, a->Hkv, a->D, es};
    const Tensor tdk{dk, a->dk, a->B, a->Lk, a->Hkv, a->D, es}, tdv{dv, a->dv, a->B, a->Lk, a->Hkv, a->D, es};
    const bool nq = a->Lq == 0 || a->H == 0, nk = a->Lk == 0;
    if (!nq && (!tq.ok() || !to.ok() || !tg.ok() || !tdq.ok() || !tdq.distinct() || !lse || (uintptr_t)lse % 4))
        return SC_ERR_INVALID_ARGUMENT;
    if (!nk && (!tk.ok() || !tv.ok() || !tdk.ok() || !tdv.ok() || !tdk.distinct() || !tdv.distinct()))
        return SC_ERR_INVALID_ARGUMENT;
    const size_t need = sc::attn_bwd_bytes(x);
    const int64_t nl = a->B * a->H * a->Lq;
    const Array none = rows_of(nullptr, 0, 0, 0, 1);
    const Array in[] = {nq ? none : tq.array(), nq ? none : to.array(), nq ? none : tg.array(),
                        nk ? none : tk.array(), nk ? none : tv.array(),
                        rows_of(lse, 1, nl, nl, 4), rows_of(a->slopes, 1, a->H, a->H, 4),
                        rows_of(a->kv_len, 1, a->B, a->B, 4),
                        rows_of(a->doc_start, 1, a->B * a->Lk, a->B * a->Lk, 4)};
    const Array out[] = {nq ? none : tdq.array(), nk ? none : tdk.array(), nk ? none : tdv.array(),
                         rows_of(ws, 1, (int64_t)need, (int64_t)need, 1)};
    if (!apart(in, out)) return SC_ERR_INVALID_ARGUMENT;
    x.q = q;
    x.k = k;
    x.v = v;
    x.o = const_cast<void*>(o);
    x.lse = const_cast<float*>(lse);
    x.dout = dout;
    x.dq = dq;
    x.dk = dk;
    x.dv = dv;
    return with_ws(need, ws, ws_bytes, stream,
                   [&](void* p) { return of(sc::launch_attn_bwd(store(kind), x, p, stream)); });
}

}  // namespace

extern "C" {

sc_status sc_layernorm(sc_kind kind, const void* x, const void* w, const void* b, void* y,
                       float* mean, float* rstd, int64_t rows, int64_t C, int64_t x_stride,
                       int64_t y_stride, float eps, hipStream_t stream)
{
    return guarded([&] { return ln_run(kind, x, w, b, y, mean, rstd, rows, C, x_stride, y_stride, eps, stream); });
}

size_t sc_layernorm_bwd_workspace_bytes(sc_kind kind, int64_t rows, int64_t C)
{
    if (ln_shape(kind, rows, C) != SC_OK) return 0;
    return sc::layernorm_bwd_bytes(store(kind), rows, (int)C);
}

sc_status sc_layernorm_bwd(sc_kind kind, const void* dy, const void* x, const void* w,
                           const float* mean, const float* rstd, void* dx, void* dw, void* db,
                           int64_t rows, int64_t C, int64_t dy_stride, int64_t x_stride,
                           int64_t dx_stride, void* ws, size_t ws_bytes, hipStream_t stream)
{
    return guarded([&] {
        return ln_bwd_run(kind, dy, x, w, mean, rstd, dx, dw, db, rows, C, dy_stride, x_stride, dx_stride,
                          ws, ws_bytes, stream);
    });
}

size_t sc_recur_workspace_bytes(sc_kind kind, int64_t B, int64_t L, int64_t C)
{
    if (recur_shape(kind, B, L, C) != SC_OK || B == 0 || L == 0 || C == 0) return 0;
    return sc::recur_bytes(B, L, (int)C);
}

sc_status sc_recur(sc_kind kind, const void* z, const void* u, const float* h0, void* h, float* hT,
                   int64_t B, int64_t L, int64_t C, int64_t z_stride, int64_t u_stride,
                   int64_t h_stride, void* ws, size_t ws_bytes, hipStream_t stream)
{
    return guarded([&] {
        return recur_run(kind, z, u, h0, h, hT, B, L, C, z_stride, u_stride, h_stride, ws, ws_bytes, stream);
    });
}

sc_status sc_recur_bwd(sc_kind kind, const void* dh, const void* z, const void* u, const void* h,
                       const float* h0, const float* dhT, void* dz, void* du, float* dh0,
                       int64_t B, int64_t L, int64_t C, int64_t dh_stride, int64_t z_stride,
                       int64_t u_stride, int64_t h_stride, int64_t dz_stride, int64_t du_stride,
                       void* ws, size_t ws_bytes, hipStream_t stream)
{
    const int64_t s[6] = {dh_stride, z_stride, u_stride, h_stride, dz_stride, du_stride};
    return guarded([&] {
        return recur_bwd_run(kind, dh, z, u, h, h0, dhT, dz, du, dh0, B, L, C, s, ws, ws_bytes, stream);
    });
}

size_t sc_attn_workspace_bytes(sc_kind kind, const sc_attn* a, int backward)
{
    sc::AttnArgs x;
    bool empty;
    if (attn_shape(kind, a, backward, &x, &empty) != SC_OK || empty) return 0;
    return backward ? sc::attn_bwd_bytes(x) : sc::attn_fwd_bytes(x);
}

sc_status sc_causal_attn(sc_kind kind, const sc_attn* a, const void* q, const void* k,
                         const void* v, void* o, float* lse, void* ws, size_t ws_bytes,
                         hipStream_t stream)
{
    return guarded([&] { return attn_run(kind, a, q, k, v, o, lse, ws, ws_bytes, stream); });
}

sc_status sc_causal_attn_bwd(sc_kind kind, const sc_attn* a, const void* dout, const void* q,
                             const void* k, const void* v, const void* o, const float* lse,
                             void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                             hipStream_t stream)
{
    return guarded([&] {
        return attn_bwd_run(kind, a, dout, q, k, v, o, lse, dq, dk, dv, ws, ws_bytes, stream);
    });
}

}  // extern "C"
