// Argument checks and workspaces shared by the host layers of the calls beside the convolution.
#pragma once

#include "specconv.h"

#include <algorithm>
#include <climits>

#include "sc_internal.h"

namespace sc {
namespace checks {

constexpr int64_t kMaxDim = (int64_t)1 << 30;   // columns, tokens and packed rows held in 32 bits

inline bool float_kind(sc_kind k) { return k == SC_KIND_F32 || k == SC_KIND_BF16; }
inline int64_t elt(sc_kind k) { return k == SC_KIND_BF16 ? 2 : 4; }
inline sc::Store store(sc_kind k) { return k == SC_KIND_F32 ? sc::Store::F32 : sc::Store::BF16; }

inline sc_status of(hipError_t e)
{
    // the launchers return InvalidValue for a grid that a launch cannot hold
    return e == hipSuccess ? SC_OK : e == hipErrorInvalidValue ? SC_ERR_UNSUPPORTED : SC_ERR_HIP;
}

template <class F>
sc_status guarded(F&& f)
{
    try {
        return f();
    } catch (...) {
        return SC_ERR_HIP;
    }
}

// What the overlap checks know of an array: runs of `width` elements of es bytes, one for each index
// of the axes (n[i] places s[i] elements apart).
struct Array {
    const void* p;
    int64_t n[3], s[3], width, es;
    bool used() const { return p && n[0] > 0 && n[1] > 0 && n[2] > 0 && width > 0; }
    // bytes from the first to past the last; false if they do not fit 63 bits
    bool span(__int128* out) const
    {
        __int128 k = width;
        for (int i = 0; i < 3; ++i) k += (__int128)(n[i] - 1) * s[i];
        *out = k * es;
        return *out <= (__int128)INT64_MAX;
    }
};

inline Array rows_of(const void* p, int64_t rows, int64_t stride, int64_t width, int64_t es)
{
    return {p, {rows, 1, 1}, {stride, 0, 0}, width, es};
}

// An array in bytes from `at` on, the axes that have more than one place by descending stride.
struct Runs {
    __int128 at;
    int axes;
    __int128 n[3], s[3], width;
    explicit Runs(const Array& a) : at((uintptr_t)a.p), axes(0), width((__int128)a.width * a.es)
    {
        for (int i = 0; i < 3; ++i) {
            if (a.n[i] < 2) continue;
            int k = axes++;
            for (; k > 0 && s[k - 1] < (__int128)a.s[i] * a.es; --k) {
                n[k] = n[k - 1];
                s[k] = s[k - 1];
            }
            n[k] = a.n[i];
            s[k] = (__int128)a.s[i] * a.es;
        }
    }
    __int128 span(int from) const
    {
        __int128 k = width;
        for (int i = from; i < axes; ++i) k += (n[i] - 1) * s[i];
        return k;
    }
};

// May a from `pa` on with its axes ia.. share a byte with b from `pb` on with its axes ib..?  Not if
// their extents do not meet.  Else the larger of the two leading strides is taken as a period that
// both repeat with (the other array, if its stride is smaller, once); as long as what repeats is no
// longer than the period, repetitions i of a and j of b meet for at most two values of i - j, and what
// repeats is compared there.  Exact for axes that nest, as the parts of one dense array do; where they
// do not, the arrays count as sharing.
inline bool meet(const Runs& a, __int128 pa, int ia, const Runs& b, __int128 pb, int ib)
{
    if (pa >= pb + b.span(ib) || pb >= pa + a.span(ia)) return false;
    const __int128 sa = ia < a.axes ? a.s[ia] : 0, sb = ib < b.axes ? b.s[ib] : 0, period = std::max(sa, sb);
    if (period == 0) return true;
    const bool ta = sa == period, tb = sb == period;   // whose leading axis is taken
    const __int128 na = ta ? a.n[ia] : 1, nb = tb ? b.n[ib] : 1;
    ia += ta;
    ib += tb;
    if (a.span(ia) > period || b.span(ib) > period) return true;
    // a's repetition i begins at pa + i period, b's j at pb + j period: i - j = k
    const __int128 d = pb - pa, low = d >= 0 ? d / period : -((-d + period - 1) / period);
    for (__int128 k = low; k <= low + 1; ++k)
        if (k > -nb && k < na && meet(a, pa + k * period, ia, b, pb, ib)) return true;
    return false;
}

// May two arrays share a byte?  Rows of one period whose other axes are multiples of it are columns of
// one array, whatever those axes are: they share nothing if their columns do not.
inline bool share(const Array& x, const Array& y)
{
    if (!x.used() || !y.used()) return false;
    __int128 ex, ey;
    if (!x.span(&ex) || !y.span(&ey)) return true;
    const __int128 px = (uintptr_t)x.p, py = (uintptr_t)y.p;
    if (px >= py + ey || py >= px + ex) return false;   // almost always
    const Runs a(x), b(y);
    for (int ka = 0; ka < a.axes; ++ka)
        for (int kb = 0; kb < b.axes; ++kb) {
            const __int128 period = a.s[ka], wa = a.span(ka + 1), wb = b.span(kb + 1);
            if (period <= 0 || period != b.s[kb] || wa > period || wb > period) continue;
            bool multiples = true;
            for (int i = 0; i < ka; ++i) multiples &= a.s[i] % period == 0;
            for (int i = 0; i < kb; ++i) multiples &= b.s[i] % period == 0;
            if (!multiples) continue;
            const __int128 d = ((b.at - a.at) % period + period) % period;   // b's first column - a's
            if (d >= wa && d + wb <= period) return false;
        }
    return meet(a, a.at, 0, b, b.at, 0);
}

// Every output apart from every input and from the other outputs.
template <int NI, int NO>
bool apart(const Array (&in)[NI], const Array (&out)[NO])
{
    for (int i = 0; i < NO; ++i) {
        for (const Array& x : in)
            if (share(out[i], x)) return false;
        for (int k = 0; k < i; ++k)
            if (share(out[i], out[k])) return false;
    }
    return true;
}

inline bool fits(const Array& a)
{
    __int128 e;
    return !a.used() || a.span(&e);
}

inline bool aligned(const void* p, int64_t stride, int64_t es)
{
    return !((uintptr_t)p % 16) && !(stride * es % 16);
}

// Runs f(ws) with the caller's workspace or one of `need` bytes allocated on the stream.
template <class F>
sc_status with_ws(size_t need, void* ws, size_t ws_bytes, hipStream_t stream, F&& f)
{
    if (ws) {
        if ((uintptr_t)ws % 256) return SC_ERR_INVALID_ARGUMENT;
        if (ws_bytes < need) return SC_ERR_WORKSPACE;
        return f(ws);
    }
    if (ws_bytes) return SC_ERR_INVALID_ARGUMENT;
    if (!need) return f(nullptr);
    void* own = nullptr;
    if (hipMallocAsync(&own, need, stream) != hipSuccess) {
        (void)hipGetLastError();
        return SC_ERR_HIP;
    }
    sc_status st = f(own);
    if (hipFreeAsync(own, stream) != hipSuccess && st == SC_OK) st = SC_ERR_HIP;
    return st;
}

// A (batch, token, head) tensor.
struct Tensor {
    const void* p;
    const int64_t* s;
    int64_t B, L, H, D, es;
    Array array() const { return {p, {B, L, H}, {s[0], s[1], s[2]}, D, es}; }
    // sizes times strides in range, 16-byte steps
    bool ok() const
    {
        const int64_t n[3] = {B, L, H};
        __int128 all = D;
        for (int i = 0; i < 3; ++i) {
            if (n[i] < 2) continue;
            if (s[i] < 0 || s[i] * es % 16 || s[i] > INT64_MAX / 16) return false;
            all += (__int128)(n[i] - 1) * s[i];
        }
        return p && (uintptr_t)p % 16 == 0 && all * es <= (__int128)INT64_MAX;
    }
    // no element twice (outputs): the axes nest
    bool distinct() const
    {
        struct Axis { int64_t n, s; } ax[3] = {{B, s[0]}, {L, s[1]}, {H, s[2]}};
        std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.s < y.s; });
        __int128 span = D;
        for (const Axis& x : ax) {
            if (x.n < 2) continue;
            if (x.s < span) return false;
            span += (__int128)(x.n - 1) * x.s;
        }
        return true;
    }
};

}  // namespace checks
}  // namespace sc
