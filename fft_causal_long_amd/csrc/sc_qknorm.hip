// Norm of each head of q and k with the rotation of positions, forward and backward (gfx950).
//
// Row x of D values (a head of a token), weight w, first R values turned in pairs (a, b) by the
// angle p f_i of the token's position p:
//
//     rstd = (mean x^2 + eps)^-1/2,  n = x rstd w,   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin
//
// and for the output gradient dy, with e = the rotation of dy by -p f_i:
//
//     dx = rstd (e w - x rstd^2 mean(e w x)),   dw = sum over rows of e x rstd
//
// Bound by memory: two elements a value move forward, three backward.  A lane holds the pairs it turns:
// V values at l V and V at R/2 + l V of a row, or 2 V neighbours where neighbours are pairs, so a row is
// read once and turned without an exchange, and its sums are a few additions between neighbouring lanes.
// Rows that are not such vectors are read in shorter ones, or value by value.  The angles of a token are
// the same for all its heads: a workgroup makes those of its tokens once, in LDS, while its first rows are
// on their way.  q's rows and k's have workgroups of their own: one chain of waits for few tokens (8 tokens
// of 20 heads: 3.6 us of kernel, 5.0 one after the other), and one set of sums for dw.
//
// Measured (MI355X; a large copy moves 5.4 TB/s, two reads and a write 5.97; inputs past every cache), whole
// calls: B 8, L 4096, 16 + 16 heads of 64 bf16, columns of one projection: forward 55 us (4.9 TB/s), backward
// 85 (4.8), of it 5 the second kernel's; B 1, L 8192, 16 + 4 heads of 128 float32 backward 58 (4.3), of it 7;
// B 4, L 4096, 16 + 4 heads of 128 float32 forward 60 (5.6).  Short prompts are far from that: up to 8191
// tokens a workgroup has one (the rule at the end of this file), which leaves most of its rows' places empty
// where the heads are few: 4096 tokens of 16 + 4 heads of 64 bf16 17 us for 21 MB, 2002 of 12 + 12 float32
// in pairs 10 for 25 MB.  The second kernel reads each 128-byte line of the parts from eight workgroups.  Steps,
// with inputs partly in the last-level cache: a 64-bit division a row 54 / 103, walks without it and the
// tensors' numbers taken out of the loop 51.6 / 98 (an index into the call's arguments is a load a row),
// 8-byte vectors backward 89, the rest 50 / 85.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sc_internal.h"
#include "sc_rows.h"

namespace sc {

namespace {

constexpr int NT = 256;

// cos and sin of p f.  The product has up to 55 bits: a double and what that leaves.  The quarter turns are
// taken off it with 2 / pi in two parts, so for angles under 2^48 the rest is right to 2^-53 of a quarter
// turn (2 / pi is good to 2^-108; the number of turns is off by 2^-6 at most before it is rounded), and
// Taylor series (to x^9 and x^10, the next terms under 3e-9) then give float32 values.
__device__ __forceinline__ float2 turn_of(int p, float f)
{
    const double a = (double)p * (double)f, left = fma((double)p, (double)f, -a);
    const double n = rint(a * 0.63661977236758134308);
    double r = fma(a, 0.63661977236758134308, -n);
    r = fma(a, -3.9357353350364971764e-17, r);   // 2 / pi less its double
    r = fma(left, 0.63661977236758134308, r);
    const float x = (float)(r * 1.57079632679489661923);
    const int q = (int)(n - 4.0 * floor(n * 0.25));
    const float z = x * x;
    float s = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
    s = __builtin_fmaf(s, z, 1.0f / 120.0f);
    s = __builtin_fmaf(s, z, -1.0f / 6.0f);
    s = __builtin_fmaf(s * z, x, x);
    float c = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    c = __builtin_fmaf(c, z, -1.0f / 720.0f);
    c = __builtin_fmaf(c, z, 1.0f / 24.0f);
    c = __builtin_fmaf(c, z, -0.5f);
    c = __builtin_fmaf(c, z, 1.0f);
    const float cq = q & 1 ? s : c, sq = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -cq : cq, q >= 2 ? -sq : sq);
}

// V neighbouring values of a row: 8 or 16 bytes.
template <class IO, int V>
struct Vec {
    typedef uint32_t Raw __attribute__((ext_vector_type(V * IO::SIZE / 4)));
    __device__ __forceinline__ static Raw load(const typename IO::T* p) { return *(const Raw*)p; }
    __device__ __forceinline__ static float at(const Raw& r, int i)
    {
        if constexpr (IO::SIZE == 2) return __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
        else return __uint_as_float(r[i]);
    }
    __device__ __forceinline__ static void store(typename IO::T* p, const float (&x)[V])
    {
        Raw r;
#pragma unroll
        for (int i = 0; i < V * IO::SIZE / 4; ++i) {
            if constexpr (IO::SIZE == 2) r[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            else r[i] = __float_as_uint(x[i]);
        }
        *(Raw*)p = r;
    }
};

// One value at a time: rows that start anywhere.
template <class IO>
struct Vec<IO, 1> {
    typedef float Raw;
    __device__ __forceinline__ static Raw load(const typename IO::T* p) { return IO::load(p, 0); }
    __device__ __forceinline__ static float at(Raw r, int) { return r; }
    __device__ __forceinline__ static void store(typename IO::T* p, const float (&x)[1]) { IO::store(p, 0, x[0]); }
};

// Where lane l of a row's D / 2V finds its V pairs: the elements a + i and b + i, or, of a vector pair
// a, b = a + V, neighbours (PAIRS).  Pairs past R / 2 are the values that do not turn.
template <int V, bool PAIRS>
struct Cut {
    int a, b;
    bool lone;   // one value at a time: the last of an odd D has no second (b is it again)
    __device__ __forceinline__ Cut(int R, int D, int l)
    {
        const bool halves = !PAIRS && V * l < R / 2;
        a = halves ? V * l : 2 * V * l;
        b = halves ? R / 2 + a : a + V;
        lone = V == 1 && b >= D;
        if (lone) b = a;
    }
};

// 2 V values of a row as V pairs.
template <class IO, int V, bool PAIRS>
struct Row {
    using W = Vec<IO, V>;
    float a[V], b[V];
    __device__ __forceinline__ void from(const typename W::Raw& u, const typename W::Raw& v, const Cut<V, PAIRS>& c)
    {
        if constexpr (V == 1) {
            a[0] = W::at(u, 0);
            b[0] = c.lone ? 0.f : W::at(v, 0);
            return;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = !PAIRS ? W::at(u, i) : 2 * i < V ? W::at(u, 2 * i % V) : W::at(v, 2 * i % V);
            b[i] = !PAIRS ? W::at(v, i) : 2 * i < V ? W::at(u, (2 * i + 1) % V) : W::at(v, (2 * i + 1) % V);
        }
    }
    __device__ __forceinline__ void to(typename IO::T* p, const Cut<V, PAIRS>& c) const
    {
        if constexpr (V == 1) {
            W::store(p + c.a, a);
            if (!c.lone) W::store(p + c.b, b);
            return;
        }
        float x[V], y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = PAIRS ? (i & 1 ? b[i / 2] : a[i / 2]) : a[i];
            y[i] = PAIRS ? (i & 1 ? b[V / 2 + i / 2] : a[V / 2 + i / 2]) : b[i];
        }
        W::store(p + c.a, x);
        W::store(p + c.b, y);
    }
};

// Sum over the LPR neighbouring lanes of a row, in every one of them.  Up to 16 lanes the partner comes
// with the addition (data-parallel primitives: lane ^ 1, lane ^ 2, then the mirror of 8 and of 16 lanes,
// whose halves are equal by then).
template <int CTRL>
__device__ __forceinline__ float from_lane(float x)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
    if constexpr (LPR >= 2) x += from_lane<0xb1>(x);
    if constexpr (LPR >= 4) x += from_lane<0x4e>(x);
    if constexpr (LPR >= 8) x += from_lane<0x141>(x);
    if constexpr (LPR >= 16) x += from_lane<0x140>(x);
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
    if constexpr (LPR >= 64) x += __shfl_xor(x, 32);
    return x;
}

// Tokens of a workgroup's turn: t0 .. t0 + n - 1 of sequence b.
struct Span {
    int64_t b, t0;
    int n;
    __device__ __forceinline__ Span(const QkArgs& a, uint32_t turn)
    {
        const uint32_t seq = turn / (uint32_t)a.turns;   // uniform
        b = seq;
        t0 = (int64_t)(turn - seq * (uint32_t)a.turns) * a.tb;
        n = (int)std::min<int64_t>(a.tb, a.L - t0);
    }
};

// A slot's rows slot, slot + step, ... of H heads a token: token i, head h, without a division a row.
struct Walk {
    int i, h, di, dh, H;
    __device__ __forceinline__ Walk(int slot, int step, int H_) : i(slot / H_), h(slot - i * H_), di(step / H_), dh(step - di * H_), H(H_) {}
    // to the next row; true if that wrapped the head
    __device__ __forceinline__ bool next()
    {
        const bool wrap = h + dh >= H;
        i += di + (wrap ? 1 : 0);
        h += dh - (wrap ? H : 0);
        return wrap;
    }
};

// The place of a walk's row in a tensor (the tensor's numbers are taken once: an index into the call's
// arguments inside the loop would be a load for each row).
template <class E>
struct Path {
    E* p;
    int64_t inc, wrap;
    __device__ __forceinline__ Path(E* base, int64_t sb, int64_t st, int64_t sh, const Span& s, const Walk& w)
        : p(base + s.b * sb + (s.t0 + w.i) * st + w.h * sh), inc(w.di * st + w.dh * sh), wrap(st - w.H * sh)
    {
    }
    __device__ __forceinline__ void next(bool wrapped) { p += wrapped ? inc + wrap : inc; }
};

// The angles of the span's tokens into table[token][pair] (D / 2 pairs a token, odd D: one more; those past
// R / 2 stay where they are).
__device__ __forceinline__ void fill_angles(const QkArgs& a, float2* table, const Span& p)
{
    const int half = (a.D + 1) / 2;
    for (int i = threadIdx.x; i < p.n * half; i += NT) {
        const int t = i / half, k = i - t * half;
        const int64_t at = p.t0 + t;
        const int pos = a.pos ? a.pos[p.b * a.L + at] : (int)(a.len ? a.len[p.b] - a.L + at : at);
        table[i] = 2 * k < a.R ? turn_of(pos, a.freq[k]) : make_float2(1.f, 0.f);
    }
}

// (v + eps)^-1/2 to about 1 ulp; the reciprocal root takes no subnormal numbers.
__device__ __forceinline__ float rstd_of(float v)
{
    const bool low = v < 0x1p-96f;
    return __builtin_amdgcn_rsqf(low ? v * 0x1p64f : v) * (low ? 0x1p32f : 1.f);
}

// The first wgs[0] workgroups take q's rows, the others k's, each their tokens in turns.
struct Share {
    int s;
    uint32_t id, step;
    __device__ __forceinline__ Share(const QkArgs& a)
        : s(blockIdx.x >= a.wgs[0]), id(blockIdx.x - (s ? a.wgs[0] : 0u)), step(s ? a.wgs[1] : a.wgs[0])
    {
    }
    // where this workgroup's sums of dw go
    __device__ __forceinline__ float* part(const QkArgs& a) const { return a.part + (int64_t)blockIdx.x * a.D; }
};

// Rows of a workgroup's tokens in turn, a row's loads issued before the row before it is finished: LPR
// lanes a row, D / 2V of them with values.
template <class IO, int V, int LPR, bool PAIRS, bool BWD>
__global__ __launch_bounds__(NT) void qk_rows(QkArgs a)
{
    using E = typename IO::T;
    using W = Vec<IO, V>;
    constexpr int RPP = NT / LPR;   // rows at a time
    extern __shared__ float2 table[];
    __shared__ float sum[BWD ? 4 : 1][BWD ? 2 * V * LPR : 1];
    const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR, half = (a.D + 1) / 2;
    const bool on = 2 * V * l < a.D;
    const int lv = on ? l : 0;
    const Cut<V, PAIRS> cut(a.R, a.D, lv);
    using RowT = Row<IO, V, PAIRS>;
    const float inv = 1.0f / (float)a.D;
    struct Raw {
        typename W::Raw xa, xb, ga, gb;
    };

    const Share share(a);
    const int H = share.s ? a.H[1] : a.H[0];
    const auto pick = [&](const int64_t(&t)[2][3], int i) { return share.s ? t[1][i] : t[0][i]; };
    const E* wp = (const E*)(share.s ? a.w[1] : a.w[0]);
    RowT w;
    if (wp) {
        w.from(W::load(wp + cut.a), W::load(wp + cut.b), cut);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) w.a[i] = w.b[i] = 1.f;
    }
    float dw[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) dw[0][i] = dw[1][i] = 0.f;

    for (uint32_t turn = share.id; turn < a.all; turn += share.step) {
        const Span span(a, turn);
        const int rows = span.n * H;
        Walk walk(slot, RPP, H);
        Path<const E> x((const E*)(share.s ? a.x[1] : a.x[0]), pick(a.xs, 0), pick(a.xs, 1), pick(a.xs, 2), span, walk);
        Path<const E> g((const E*)(share.s ? a.dy[1] : a.dy[0]), pick(a.dys, 0), pick(a.dys, 1), pick(a.dys, 2), span, walk);
        Path<E> y((E*)(share.s ? a.y[1] : a.y[0]), pick(a.ys, 0), pick(a.ys, 1), pick(a.ys, 2), span, walk);
        Raw now;
        auto load = [&] {
            now.xa = W::load(x.p + cut.a);
            now.xb = W::load(x.p + cut.b);
            if constexpr (BWD) {
                now.ga = W::load(g.p + cut.a);
                now.gb = W::load(g.p + cut.b);
            }
        };
        if (slot < rows) load();
        __syncthreads();
        fill_angles(a, table, span);
        __syncthreads();
        for (int r = slot; r < rows; r += RPP) {
            const float2* cs = table + walk.i * half + lv * V;
            E* yp = y.p;
            RowT v, e;
            v.from(now.xa, now.xb, cut);
            if constexpr (BWD) e.from(now.ga, now.gb, cut);
            const bool wrap = walk.next();
            y.next(wrap);
            if (r + RPP < rows) {   // else the same row again, for nothing: no branch around the loads
                x.next(wrap);
                if constexpr (BWD) g.next(wrap);
            }
            load();
            float sq = 0.f, ex = 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) sq += v.a[k] * v.a[k] + v.b[k] * v.b[k];
            if constexpr (BWD) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float2 c = cs[k];
                    const float ea = e.a[k] * c.x + e.b[k] * c.y, eb = e.b[k] * c.x - e.a[k] * c.y;
                    e.a[k] = ea;
                    e.b[k] = eb;
                    ex += ea * w.a[k] * v.a[k] + eb * w.b[k] * v.b[k];
                }
                ex = row_sum<LPR>(on ? ex : 0.f);
            }
            sq = row_sum<LPR>(on ? sq : 0.f);
            const float rstd = rstd_of(sq * inv + a.eps);
            if constexpr (BWD) {
                const float m = ex * inv * rstd;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float na = v.a[k] * rstd, nb = v.b[k] * rstd;
                    dw[0][k] += e.a[k] * na;
                    dw[1][k] += e.b[k] * nb;
                    v.a[k] = (e.a[k] * w.a[k] - na * m) * rstd;
                    v.b[k] = (e.b[k] * w.b[k] - nb * m) * rstd;
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float2 c = cs[k];
                    const float na = v.a[k] * rstd * w.a[k], nb = v.b[k] * rstd * w.b[k];
                    v.a[k] = na * c.x - nb * c.y;
                    v.b[k] = nb * c.x + na * c.y;
                }
            }
            if (on) v.to(yp, cut);
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        // the rows of a wave, then the waves
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
            float x = dw[k / V][k % V];
#pragma unroll
            for (int m = LPR; m < 64; m <<= 1) x += __shfl_xor(x, m);
            if ((threadIdx.x & 63) < LPR) sum[threadIdx.x >> 6][k * LPR + l] = x;
        }
        __syncthreads();
        if (slot != 0 || !on) return;
        float* out = share.part(a);
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) {
            const int at = k * LPR + l, i = k % V;
            if (V == 1 && k == 1 && cut.lone) continue;
            out[PAIRS ? cut.a + 2 * i + k / V : (k < V ? cut.a : cut.b) + i] = (sum[0][at] + sum[1][at]) + (sum[2][at] + sum[3][at]);
        }
    }
}

// Any rows of more than 128 values: a wave a row, a lane the pairs lane, lane + 64, ...
constexpr int PAIRS = 4;   // D up to 512
template <class IO, bool BWD>
__global__ __launch_bounds__(NT) void qk_pairs(QkArgs a)
{
    using E = typename IO::T;
    extern __shared__ float2 table[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = (a.D + 1) / 2;
    const float inv = 1.0f / (float)a.D;
    int ia[PAIRS], ib[PAIRS];   // the elements, -1: none
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
        const int p = lane + 64 * k;
        const bool turned = 2 * p < a.R && !a.pairs;
        ia[k] = turned ? p : 2 * p;
        ib[k] = turned ? a.R / 2 + p : 2 * p + 1;
        if (ia[k] >= a.D) ia[k] = -1;
        if (ib[k] >= a.D) ib[k] = -1;
    }
    const Share share(a);
    const int s = share.s, H = s ? a.H[1] : a.H[0];
    const auto pick = [&](const int64_t(&t)[2][3], int i) { return s ? t[1][i] : t[0][i]; };
    const E *xp = (const E*)(s ? a.x[1] : a.x[0]), *gp = (const E*)(s ? a.dy[1] : a.dy[0]), *w = (const E*)(s ? a.w[1] : a.w[0]);
    E* yp = (E*)(s ? a.y[1] : a.y[0]);
    float dw[2][PAIRS];
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) dw[0][k] = dw[1][k] = 0.f;
    auto get = [](const E* p, int i) { return i < 0 ? 0.f : IO::load(p, i); };

    for (uint32_t turn = share.id; turn < a.all; turn += share.step) {
        const Span span(a, turn);
        __syncthreads();
        fill_angles(a, table, span);
        __syncthreads();
        {
            const int rows = span.n * H;
            Walk walk(wave, NT / 64, H);
            for (int r = wave; r < rows; r += NT / 64, walk.next()) {
                const int i = walk.i;
                const int64_t t = span.t0 + i;
                const E* x = xp + span.b * pick(a.xs, 0) + t * pick(a.xs, 1) + walk.h * pick(a.xs, 2);
                const E* g = BWD ? gp + span.b * pick(a.dys, 0) + t * pick(a.dys, 1) + walk.h * pick(a.dys, 2) : nullptr;
                E* y = yp + span.b * pick(a.ys, 0) + t * pick(a.ys, 1) + walk.h * pick(a.ys, 2);
                float va[PAIRS], vb[PAIRS], ea[PAIRS], eb[PAIRS], wa[PAIRS], wb[PAIRS], sq = 0.f, ex = 0.f;
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) {
                    va[k] = get(x, ia[k]);
                    vb[k] = get(x, ib[k]);
                    wa[k] = w ? get(w, ia[k]) : 1.f;
                    wb[k] = w ? get(w, ib[k]) : 1.f;
                    sq += va[k] * va[k] + vb[k] * vb[k];
                    if constexpr (BWD) {
                        const float2 c = ia[k] < 0 ? make_float2(1.f, 0.f) : table[i * half + lane + 64 * k];
                        const float ga = get(g, ia[k]), gb = get(g, ib[k]);
                        ea[k] = ga * c.x + gb * c.y;
                        eb[k] = gb * c.x - ga * c.y;
                        ex += ea[k] * wa[k] * va[k] + eb[k] * wb[k] * vb[k];
                    }
                }
                const float rstd = rstd_of(row_sum<64>(sq) * inv + a.eps);
                const float m = BWD ? row_sum<64>(ex) * inv * rstd : 0.f;
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) {
                    float oa, ob;
                    if constexpr (BWD) {
                        const float na = va[k] * rstd, nb = vb[k] * rstd;
                        dw[0][k] += ea[k] * na;
                        dw[1][k] += eb[k] * nb;
                        oa = (ea[k] * wa[k] - na * m) * rstd;
                        ob = (eb[k] * wb[k] - nb * m) * rstd;
                    } else {
                        const float2 c = ia[k] < 0 ? make_float2(1.f, 0.f) : table[i * half + lane + 64 * k];
                        const float na = va[k] * rstd * wa[k], nb = vb[k] * rstd * wb[k];
                        oa = na * c.x - nb * c.y;
                        ob = nb * c.x + na * c.y;
                    }
                    if (ia[k] >= 0) IO::store(y, ia[k], oa);
                    if (ib[k] >= 0) IO::store(y, ib[k], ob);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        __shared__ float sum[4][2][64 * PAIRS];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            sum[wave][0][64 * k + lane] = dw[0][k];
            sum[wave][1][64 * k + lane] = dw[1][k];
        }
        __syncthreads();
        float* out = share.part(a);
        if (wave < 2) {   // wave 0 the pairs' first values, wave 1 the second
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) {
                const int at = 64 * k + lane, i = wave ? ib[k] : ia[k];
                const float x = (sum[0][wave][at] + sum[1][wave][at]) + (sum[2][wave][at] + sum[3][wave][at]);
                if (i >= 0) out[i] = x;
            }
        }
    }
}

// dw = the workgroups' sums added: 4 columns a workgroup, 64 threads a column, whose loads are all in
// flight at once (up to 1024 parts: 16 a thread).  In 64 bits: a part adds a few rows, but there are up to
// 2048 parts, whose sum may be small beside them.
template <class IO>
__global__ __launch_bounds__(NT) void qk_sum(QkArgs a)
{
    __shared__ double sum[NT];
    const int at = blockIdx.x * 4 + threadIdx.x % 4, s = at >= a.D;
    double x = 0.0;
    if (at < 2 * a.D) {
        const float* p = a.part + (s ? (int64_t)a.wgs[0] * a.D : 0) + (at - s * a.D);
        const int parts = (int)a.wgs[s];
#pragma unroll 16
        for (int k = threadIdx.x / 4; k < parts; k += 64) x += p[(int64_t)k * a.D];
    }
    sum[threadIdx.x] = x;
    __syncthreads();
#pragma unroll
    for (int m = NT / 2; m >= 4; m >>= 1) {
        if ((int)threadIdx.x < m) sum[threadIdx.x] += sum[threadIdx.x + m];
        __syncthreads();
    }
    if (threadIdx.x >= 4 || at >= 2 * a.D) return;
    typename IO::T* out = (typename IO::T*)a.dw[at < a.D ? 0 : 1];
    if (out) IO::store(out, at % a.D, (float)sum[threadIdx.x]);
}

// Tokens of a turn (of one sequence): so many that the turns fill the GPU several times over, up to what
// 16 KB of angles hold (forward above in 1024 turns 60 us, 2048 57, 4096 55, 8192 58.5, 16384 82; backward,
// whose workgroups keep sums, 1024 87.5, 2048 84, 4096 88).
constexpr int64_t FILL = 4096, FILL_BWD = 2048, MOST = 1 << 20;   // MOST: what a launch holds; they walk the rest
constexpr int ANGLES = 2048;
struct Plan {
    int64_t tb, turns, all, wgs[2];   // turns of a sequence, of all of them; workgroups of q's rows, of k's
};
Plan plan(const QkArgs& a, bool bwd)
{
    const int64_t half = (a.D + 1) / 2, most = bwd ? FILL_BWD : MOST, heads = (int64_t)a.H[0] + a.H[1];
    Plan p;
    p.tb = std::max<int64_t>(1, std::min<int64_t>({a.tokens / (bwd ? FILL_BWD : FILL), ANGLES / half, a.L}));
    p.turns = (a.L + p.tb - 1) / p.tb;
    p.all = a.B * p.turns;
    for (int s = 0; s < 2; ++s)
        p.wgs[s] = a.H[s] == 0 ? 0 : std::max<int64_t>(1, std::min(p.all, most * a.H[s] / heads));
    return p;
}

template <class IO, bool BWD>
hipError_t go(QkArgs a, hipStream_t st)
{
    const Plan p = plan(a, BWD);
    a.tb = (int)p.tb;
    a.turns = (int)p.turns;
    if (p.all > INT32_MAX) return hipErrorInvalidValue;   // (the walk's 32 bits)
    a.all = (uint32_t)p.all;
    a.wgs[0] = (uint32_t)p.wgs[0];
    a.wgs[1] = (uint32_t)p.wgs[1];
    const dim3 grid(a.wgs[0] + a.wgs[1]), block(NT);
    const size_t lds = (size_t)a.tb * ((a.D + 1) / 2) * sizeof(float2);
    // V pairs a lane where the rows are whole lanes of them: 16-byte vectors forward, half of them backward
    // (half the registers: B 4, L 4096, 20 heads of 128 bf16 57 us, 68 with 16 bytes), half or a quarter
    // where the sizes ask for it, else single values
    auto fits = [&](int v) { return a.whole && a.D % (2 * v) == 0 && (a.pairs || a.R % (2 * v) == 0); };
    auto rows = [&](auto v, auto lpr) {
        constexpr int V = decltype(v)::value, LPR = decltype(lpr)::value;
        if (a.pairs) hipLaunchKernelGGL((qk_rows<IO, V, LPR, true, BWD>), grid, block, lds, st, a);
        else hipLaunchKernelGGL((qk_rows<IO, V, LPR, false, BWD>), grid, block, lds, st, a);
    };
    using std::integral_constant;
    auto lanes = [&](auto v) {
        const int n = (a.D + 2 * decltype(v)::value - 1) / (2 * decltype(v)::value);
        if (n <= 4) rows(v, integral_constant<int, 4>());
        else if (n <= 8) rows(v, integral_constant<int, 8>());
        else if (n <= 16) rows(v, integral_constant<int, 16>());
        else if (n <= 32) rows(v, integral_constant<int, 32>());
        else rows(v, integral_constant<int, 64>());
    };
    constexpr int W = vec_elems<IO>;
    if (!BWD && W == 8 && fits(8)) lanes(integral_constant<int, W>());
    else if (fits(4)) lanes(integral_constant<int, 4>());
    else if (fits(2) && a.D <= 256) lanes(integral_constant<int, 2>());
    else if (a.D <= 128) lanes(integral_constant<int, 1>());
    else hipLaunchKernelGGL((qk_pairs<IO, BWD>), grid, block, lds, st, a);
    return hipGetLastError();
}

template <class IO>
hipError_t bwd(QkArgs a, void* ws, hipStream_t st)
{
    a.part = a.dw[0] || a.dw[1] ? (float*)ws : nullptr;
    if (a.tokens > 0) {   // (else sums of no rows)
        const hipError_t e = go<IO, true>(a, st);
        if (e != hipSuccess || !a.part) return e;
        const Plan p = plan(a, true);
        a.wgs[0] = (uint32_t)p.wgs[0];
        a.wgs[1] = (uint32_t)p.wgs[1];
    }
    if (!a.dw[0] && !a.dw[1]) return hipSuccess;
    hipLaunchKernelGGL(qk_sum<IO>, dim3((2 * a.D + 3) / 4), dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk(Store s, const QkArgs& a, hipStream_t st)
{
    return s == Store::F32 ? go<f32_io, false>(a, st) : go<bf16_io, false>(a, st);
}

size_t qk_bwd_bytes(Store, const QkArgs& a)
{
    if (a.tokens == 0) return 0;
    const Plan p = plan(a, true);
    return (size_t)(p.wgs[0] + p.wgs[1]) * a.D * sizeof(float);
}

hipError_t launch_qk_bwd(Store s, const QkArgs& a, void* ws, hipStream_t st)
{
    return s == Store::F32 ? bwd<f32_io>(a, ws, st) : bwd<bf16_io>(a, ws, st);
}

}  // namespace sc
