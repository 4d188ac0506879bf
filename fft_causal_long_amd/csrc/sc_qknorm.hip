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
// Bound by memory: two elements a value move forward, three backward.  A lane holds the pairs it
// turns: the 16-byte vectors at l V and R/2 + l V of a row, or two neighbouring vectors where
// neighbours are pairs, so a row is read once and turned without an exchange, and its sums are a
// few shuffles.  Rows that are not such vectors go pair by pair, a wave a row.  The angles of a
// token are the same for all its heads: a workgroup makes those of its tokens once, one a thread,
// in LDS, while its first rows are on their way.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_internal.h"
#include "sc_rows.h"

namespace sc {

namespace {

constexpr int NT = 256;

// cos and sin of p f.  The product is exact in 64 bits for |p| < 2^29; the quarter turns are taken
// off it with 2 / pi in two parts, so the rest is right to 2^-53 of a quarter turn whatever p, and
// Taylor series (to x^9 and x^10, the next terms under 2e-9) then give float32 values.
__device__ __forceinline__ float2 turn_of(int p, float f)
{
    const double a = (double)p * (double)f;
    const double n = rint(a * 0.63661977236758134308);
    double r = fma(a, 0.63661977236758134308, -n);
    r = fma(a, -3.9357353350364971764e-17, r);   // 2 / pi less its double
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

// Where the pairs of a row lie.  WHOLE: lane l of a row's D / 2V holds V pairs, the elements a + i and
// b + i (or a + 2 i and a + 2 i + 1).  Pairs past R / 2 are the values that do not turn.
template <class IO>
struct Cut {
    static constexpr int V = vec_elems<IO>;
    int a, b;
    __device__ __forceinline__ Cut(const QkArgs& q, int l)
    {
        if (q.pairs) {
            a = 2 * V * l;
            b = a + V;
        } else if (V * l < q.R / 2) {
            a = V * l;
            b = q.R / 2 + a;
        } else {
            a = 2 * V * l;
            b = a + V;
        }
    }
};

// 2 V values of a row as V pairs.
template <class IO>
struct Row {
    static constexpr int V = vec_elems<IO>;
    float a[V], b[V];
    __device__ __forceinline__ void from(const uint4& u, const uint4& v, bool pairs)
    {
        const Lanes<IO> x = widen<IO>(u), y = widen<IO>(v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = pairs ? (2 * i < V ? x.x[2 * i % V] : y.x[2 * i % V]) : x.x[i];
            b[i] = pairs ? (2 * i < V ? x.x[(2 * i + 1) % V] : y.x[(2 * i + 1) % V]) : y.x[i];
        }
    }
    __device__ __forceinline__ void to(typename IO::T* p, const Cut<IO>& c, bool pairs) const
    {
        Lanes<IO> x, y;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x.x[i] = pairs ? (i & 1 ? b[i / 2] : a[i / 2]) : a[i];
            y.x[i] = pairs ? (i & 1 ? b[V / 2 + i / 2] : a[V / 2 + i / 2]) : b[i];
        }
        *(uint4*)(p + c.a) = narrow<IO>(x);
        *(uint4*)(p + c.b) = narrow<IO>(y);
    }
};

// sum over the LPR neighbouring lanes of a row
template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

__device__ __forceinline__ int position(const QkArgs& a, int64_t token)
{
    if (a.pos) return a.pos[token];
    const int64_t b = token / a.L, t = token - b * a.L;
    return (int)(a.len ? a.len[b] - a.L + t : t);
}

// The angles of tokens t0 .. t0 + n - 1 into table[token][pair] (D / 2 pairs a token, odd D: one more;
// those past R / 2 stay where they are).
__device__ __forceinline__ void fill_angles(const QkArgs& a, float2* table, int64_t t0, int n)
{
    const int half = (a.D + 1) / 2;
    for (int i = threadIdx.x; i < n * half; i += NT) {
        const int t = i / half, p = i - t * half;
        table[i] = 2 * p < a.R ? turn_of(position(a, t0 + t), a.freq[p]) : make_float2(1.f, 0.f);
    }
}

template <class IO>
__device__ __forceinline__ int64_t row_at(const int64_t (&s)[3], int64_t b, int64_t t, int h)
{
    return b * s[0] + t * s[1] + h * s[2];
}

// Rows of a workgroup's tokens in turn, q's first: LPR lanes a row, D / 2V of them with values.
template <class IO, int LPR, bool BWD>
__global__ __launch_bounds__(NT) void qk_rows(QkArgs a)
{
    using E = typename IO::T;
    constexpr int V = vec_elems<IO>, RPP = NT / LPR;   // rows at a time
    extern __shared__ float2 table[];
    const int l = threadIdx.x % LPR, slot = threadIdx.x / LPR, half = (a.D + 1) / 2;
    const bool on = 2 * V * l < a.D;
    const Cut<IO> cut(a, on ? l : 0);
    const float inv = 1.0f / (float)a.D;
    float dw[BWD ? 2 : 1][2][V];
    if constexpr (BWD)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) dw[s][0][i] = dw[s][1][i] = 0.f;

    for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.tb) {
        const int n = (int)std::min<int64_t>(a.tb, a.tokens - t0);
        __syncthreads();
        fill_angles(a, table, t0, n);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int H = a.H[s], rows = n * H;
            Row<IO> w;
            if (a.w[s]) {
                w.from(*(const uint4*)((const E*)a.w[s] + cut.a), *(const uint4*)((const E*)a.w[s] + cut.b), a.pairs);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) w.a[i] = w.b[i] = 1.f;
            }
            for (int r = slot; r < rows; r += RPP) {
                const int i = r / H, h = r - i * H;
                const int64_t b = (t0 + i) / a.L, t = t0 + i - b * a.L;
                const E* x = (const E*)a.x[s] + row_at<IO>(a.xs[s], b, t, h);
                Row<IO> v, e;
                const uint4 xa = *(const uint4*)(x + cut.a), xb = *(const uint4*)(x + cut.b);
                v.from(xa, xb, a.pairs);
                if constexpr (BWD) {
                    const E* g = (const E*)a.dy[s] + row_at<IO>(a.dys[s], b, t, h);
                    e.from(*(const uint4*)(g + cut.a), *(const uint4*)(g + cut.b), a.pairs);
                }
                const float2* turn = table + i * half + (on ? l : 0) * V;
                float sq = 0.f, ex = 0.f;
#pragma unroll
                for (int k = 0; k < V; ++k) sq += v.a[k] * v.a[k] + v.b[k] * v.b[k];
                if constexpr (BWD) {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float2 c = turn[k];
                        const float ea = e.a[k] * c.x + e.b[k] * c.y, eb = e.b[k] * c.x - e.a[k] * c.y;
                        e.a[k] = ea;
                        e.b[k] = eb;
                        ex += ea * w.a[k] * v.a[k] + eb * w.b[k] * v.b[k];
                    }
                    ex = row_sum<LPR>(on ? ex : 0.f);
                }
                sq = row_sum<LPR>(on ? sq : 0.f);
                const float rstd = 1.0f / sqrtf(sq * inv + a.eps);
                if constexpr (BWD) {
                    const float m = ex * inv * rstd;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float na = v.a[k] * rstd, nb = v.b[k] * rstd;
                        dw[s][0][k] += e.a[k] * na;
                        dw[s][1][k] += e.b[k] * nb;
                        v.a[k] = (e.a[k] * w.a[k] - na * m) * rstd;
                        v.b[k] = (e.b[k] * w.b[k] - nb * m) * rstd;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float2 c = turn[k];
                        const float na = v.a[k] * rstd * w.a[k], nb = v.b[k] * rstd * w.b[k];
                        v.a[k] = na * c.x - nb * c.y;
                        v.b[k] = nb * c.x + na * c.y;
                    }
                }
                if (on) v.to((E*)a.y[s] + row_at<IO>(a.ys[s], b, t, h), cut, a.pairs);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        // the rows of a wave, then the waves
        __shared__ float sum[4][2][2 * V * LPR];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) {
                float x = dw[s][k / V][k % V];
#pragma unroll
                for (int m = LPR; m < 64; m <<= 1) x += __shfl_xor(x, m);
                if ((threadIdx.x & 63) < LPR) sum[wave][s][k * LPR + l] = x;
            }
        __syncthreads();
        float* out = a.part + (int64_t)blockIdx.x * 2 * a.D;
        if (slot < 2 && on) {
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) {
                const int at = k * LPR + l;
                const float x = (sum[0][slot][at] + sum[1][slot][at]) + (sum[2][slot][at] + sum[3][slot][at]);
                const int i = k % V;
                out[slot * a.D + (a.pairs ? cut.a + 2 * i + k / V : (k < V ? cut.a : cut.b) + i)] = x;
            }
        }
    }
}

// Any rows: a wave a row, a lane the pairs lane, lane + 64, ...
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
    float dw[BWD ? 2 : 1][2][PAIRS];
    if constexpr (BWD)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) dw[s][0][k] = dw[s][1][k] = 0.f;
    auto get = [](const E* p, int i) { return i < 0 ? 0.f : IO::load(p, i); };

    for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.tb) {
        const int n = (int)std::min<int64_t>(a.tb, a.tokens - t0);
        __syncthreads();
        fill_angles(a, table, t0, n);
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int H = a.H[s], rows = n * H;
            const E* w = (const E*)a.w[s];
            for (int r = wave; r < rows; r += NT / 64) {
                const int i = r / H, h = r - i * H;
                const int64_t b = (t0 + i) / a.L, t = t0 + i - b * a.L;
                const E* x = (const E*)a.x[s] + row_at<IO>(a.xs[s], b, t, h);
                const E* g = BWD ? (const E*)a.dy[s] + row_at<IO>(a.dys[s], b, t, h) : nullptr;
                E* y = (E*)a.y[s] + row_at<IO>(a.ys[s], b, t, h);
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
                const float rstd = 1.0f / sqrtf(row_sum<64>(sq) * inv + a.eps);
                const float m = BWD ? row_sum<64>(ex) * inv * rstd : 0.f;
#pragma unroll
                for (int k = 0; k < PAIRS; ++k) {
                    float oa, ob;
                    if constexpr (BWD) {
                        const float na = va[k] * rstd, nb = vb[k] * rstd;
                        dw[s][0][k] += ea[k] * na;
                        dw[s][1][k] += eb[k] * nb;
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
        __shared__ float sum[4][2][2][64 * PAIRS];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) {
                sum[wave][s][0][64 * k + lane] = dw[s][0][k];
                sum[wave][s][1][64 * k + lane] = dw[s][1][k];
            }
        __syncthreads();
        float* out = a.part + (int64_t)blockIdx.x * 2 * a.D;
        if (wave < 2) {
#pragma unroll
            for (int k = 0; k < PAIRS; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = 64 * k + lane, i = j ? ib[k] : ia[k];
                    const float x = (sum[0][wave][j][at] + sum[1][wave][j][at]) + (sum[2][wave][j][at] + sum[3][wave][j][at]);
                    if (i >= 0) out[wave * a.D + i] = x;
                }
        }
    }
}

// dw = the workgroups' sums added: 8 columns a workgroup, 32 threads a column.
template <class IO>
__global__ __launch_bounds__(NT) void qk_sum(QkArgs a, int parts)
{
    __shared__ float sum[NT];
    const int at = blockIdx.x * 8 + threadIdx.x % 8;
    float x = 0.f;
    if (at < 2 * a.D) {
#pragma unroll 8
        for (int p = threadIdx.x / 8; p < parts; p += 32) x += a.part[(int64_t)p * 2 * a.D + at];
    }
    sum[threadIdx.x] = x;
    __syncthreads();
#pragma unroll
    for (int m = NT / 2; m >= 8; m >>= 1) {
        if ((int)threadIdx.x < m) sum[threadIdx.x] += sum[threadIdx.x + m];
        __syncthreads();
    }
    if (threadIdx.x >= 8 || at >= 2 * a.D) return;
    typename IO::T* out = (typename IO::T*)a.dw[at < a.D ? 0 : 1];
    if (out) IO::store(out, at % a.D, sum[threadIdx.x]);
}

struct Plan {
    int tb;
    int64_t wgs;
};

// Tokens of a workgroup: as many as give every thread an angle, fewer while the workgroups do not
// fill the GPU.
constexpr int64_t FILL = 1024, MOST = 1 << 20;   // MOST: what a launch holds; they walk the rest
Plan plan(const QkArgs& a, bool bwd)
{
    const int half = (a.D + 1) / 2;
    Plan p;
    p.tb = (int)std::max<int64_t>(1, std::min<int64_t>(std::max(1, NT / half), a.tokens / FILL));
    p.wgs = (a.tokens + p.tb - 1) / p.tb;
    p.wgs = std::min(p.wgs, bwd ? FILL : MOST);
    return p;
}

template <class IO, bool BWD>
hipError_t go(QkArgs a, hipStream_t st)
{
    constexpr int V = vec_elems<IO>;
    const Plan p = plan(a, BWD);
    a.tb = p.tb;
    if (!grid_ok(p.wgs, NT)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)p.wgs), block(NT);
    const size_t lds = (size_t)p.tb * ((a.D + 1) / 2) * sizeof(float2);
    const int lanes = a.D / (2 * V);
    const bool whole = a.whole && a.D % (2 * V) == 0 && (a.pairs || a.R % (2 * V) == 0);
    if (!whole) hipLaunchKernelGGL((qk_pairs<IO, BWD>), grid, block, lds, st, a);
    else if (lanes <= 4) hipLaunchKernelGGL((qk_rows<IO, 4, BWD>), grid, block, lds, st, a);
    else if (lanes <= 8) hipLaunchKernelGGL((qk_rows<IO, 8, BWD>), grid, block, lds, st, a);
    else if (lanes <= 16) hipLaunchKernelGGL((qk_rows<IO, 16, BWD>), grid, block, lds, st, a);
    else hipLaunchKernelGGL((qk_rows<IO, 64, BWD>), grid, block, lds, st, a);
    return hipGetLastError();
}

template <class IO>
hipError_t bwd(QkArgs a, void* ws, hipStream_t st)
{
    a.part = a.dw[0] || a.dw[1] ? (float*)ws : nullptr;
    if (a.tokens > 0) {
        const hipError_t e = go<IO, true>(a, st);
        if (e != hipSuccess || !a.part) return e;
    }
    if (!a.dw[0] && !a.dw[1]) return hipSuccess;
    const int parts = a.tokens > 0 ? (int)plan(a, true).wgs : 0;   // none: sums of no rows
    hipLaunchKernelGGL(qk_sum<IO>, dim3((2 * a.D + 7) / 8), dim3(NT), 0, st, a, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk(Store s, const QkArgs& a, hipStream_t st)
{
    return s == Store::F32 ? go<f32_io, false>(a, st) : go<bf16_io, false>(a, st);
}

size_t qk_bwd_bytes(Store, const QkArgs& a)
{
    return a.tokens > 0 ? (size_t)plan(a, true).wgs * 2 * a.D * sizeof(float) : 0;
}

hipError_t launch_qk_bwd(Store s, const QkArgs& a, void* ws, hipStream_t st)
{
    return s == Store::F32 ? bwd<f32_io>(a, ws, st) : bwd<bf16_io>(a, ws, st);
}

}  // namespace sc
