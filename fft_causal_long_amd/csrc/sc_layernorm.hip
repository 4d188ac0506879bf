// Layer norm, forward and backward (gfx950).
//
// Row x of C values (the normalisation before a mixing layer, "Caracal: Causal Architecture
// via Spectral Mixing", key design 1):
//
//     mean = sum x / C,  rstd = (sum (x - mean)^2 / C + eps)^-1/2,  y = (x - mean) rstd w + b
//
// and for the output gradient dy, with xh = (x - mean) rstd and e = dy w:
//
//     dx = rstd (e - mean(e) - xh mean(e xh)),   dw = sum_rows dy xh,   db = sum_rows dy
//
// Both directions are bound by memory: 2 elements a value forward, 3 backward.  A row is read
// once and kept in registers by TPR threads (16, 64 or 256, NV vectors of 16 bytes each), so
// the variance is the two-pass sum about the mean, exact to float32 rounding, at no second
// read.  Backward, a workgroup walks rows and keeps its share of dw and db in registers; the
// shares go to a workspace and a second kernel adds them in a fixed order: no atomics, the
// same bits every run.
// Rows longer than 8192 values do not fit the registers: they are read again from cache
// (lnl_* kernels), and dw, db come from a kernel that walks the rows column by column.
//
// Measured (MI355X; a large copy moves 5.4 TB/s): forward, 8192 x 768 float32, 10.8 us (4.7 TB/s),
// 32768 x 2048 bfloat16 57 us (4.7); 8 x 768 bfloat16, one decoding step, 3.5 us, less than a
// launch costs.  Backward, 32768 x 1024 bfloat16, 39 us with the sums of dw and db (5.2).  Rows of
// 16384 float32, read twice: forward 2048 of them 90 us (3.0), backward 160 us (2.5).  Rows that are
// not whole vectors go element by element: 16384 of 767 float32 forward 19 us (5.3) and backward 36
// (4.2); 32768 of 1023 bfloat16, two bytes a load, 57 (2.3) and 48 (4.2).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sc_internal.h"
#include "sc_rows.h"

namespace sc {

namespace {

constexpr int NT = 256;          // threads
constexpr int LNL_STRIPS = 64;   // row strips of the column kernel (long rows)

// Sum of v over the TPR threads of a row, in every one of them.  TPR = 256 goes through
// `red` (4 floats, one buffer per call so that one barrier is enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red)
{
#pragma unroll
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) v += __shfl_xor(v, m);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (red[0] + red[1]) + (red[2] + red[3]);
    }
    return v;
}

// A thread's columns of its row's vector i: V neighbours, or (rows that are not whole vectors, read
// element by element) V that lie TPR apart, so that each load of the TPR threads takes TPR neighbours:
// 16384 rows of 767 float32 take 20 us forward, 48 with neighbours a thread.
template <int TPR, int V, bool WHOLE>
struct Columns {
    static constexpr int STEP = WHOLE ? 1 : TPR;
    __device__ __forceinline__ static int first(int i, int lt) { return WHOLE ? (i * TPR + lt) * V : i * TPR * V + lt; }
};

template <class IO, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NT) void ln_fwd(const typename IO::T* __restrict__ x,
                                             const typename IO::T* __restrict__ w,
                                             const typename IO::T* __restrict__ b,
                                             typename IO::T* __restrict__ y,
                                             float* __restrict__ mean, float* __restrict__ rstd,
                                             int64_t rows, int C, int64_t xs, int64_t ys,
                                             float eps)
{
    constexpr int V = vec_elems<IO>, RPB = NT / TPR;
    using R = Columns<TPR, V, WHOLE>;
    __shared__ float red[2][2][4];   // double-buffered over the row loop
    const int lt = threadIdx.x % TPR;
    const float n = (float)C;
    uint4 wr[NV], br[NV];   // read before the first row's sums, not after them
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = R::first(i, lt), cc = c < C ? c : 0;
        if (w) wr[i] = load_raw<IO, WHOLE, R::STEP>(w, cc, C);
        if (b) br[i] = load_raw<IO, WHOLE, R::STEP>(b, cc, C);
    }
    int buf = 0;
    // every thread of a workgroup makes the same number of turns (the barriers of TPR = 256)
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = r0 + threadIdx.x / TPR;
        const bool on = row < rows;
        const typename IO::T* xr = x + (on ? row : 0) * xs;
        Lanes<IO> v[NV];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            const uint4 raw = load_raw<IO, WHOLE, R::STEP>(xr, c < C ? c : 0, C);
            v[i] = widen<IO>(c < C ? raw : make_uint4(0, 0, 0, 0));
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[i].x[e];
        }
        const float mu = row_sum<TPR>(s, red[buf][0]) / n;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i].x[e] -= mu;
                q += c + e * R::STEP < C ? v[i].x[e] * v[i].x[e] : 0.f;
            }
        }
        const float var = row_sum<TPR>(q, red[buf][1]) / n;
        const float rs = 1.0f / sqrtf(var + eps);
        buf ^= 1;
        if (!on) continue;
        if (lt == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            if (c >= C) continue;
            Lanes<IO> o;
            Lanes<IO> wv, bv;
            if (w) wv = widen<IO>(wr[i]);
            if (b) bv = widen<IO>(br[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float t = v[i].x[e] * rs;
                if (w) t *= wv.x[e];
                o.x[e] = b ? t + bv.x[e] : t;
            }
            store_raw<IO, WHOLE, R::STEP>(y + row * ys, c, C, o);
        }
    }
}

template <class IO, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NT) void ln_bwd(const typename IO::T* __restrict__ dy,
                                             const typename IO::T* __restrict__ x,
                                             const typename IO::T* __restrict__ w,
                                             const float* __restrict__ mean,
                                             const float* __restrict__ rstd,
                                             typename IO::T* __restrict__ dx,
                                             float* __restrict__ part, int64_t rows, int C,
                                             int64_t dys, int64_t xs, int64_t dxs)
{
    constexpr int V = vec_elems<IO>, RPB = NT / TPR;
    using R = Columns<TPR, V, WHOLE>;
    __shared__ float red[2][2][4];
    __shared__ float acc[RPB > 1 ? TPR * NV * V * 2 : 1];
    const int lt = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float n = (float)C;
    Lanes<IO> wv[NV], aw[NV], ab[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = R::first(i, lt);
        if (w) wv[i] = widen<IO>(load_raw<IO, WHOLE, R::STEP>(w, c < C ? c : 0, C));
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (!w) wv[i].x[e] = 1.f;
            aw[i].x[e] = ab[i].x[e] = 0.f;
        }
    }
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * RPB;
    uint4 nx[NV], ny[NV];   // the next row, in flight while this one is reduced
    float nmu = 0.f, nrs = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t r = row < rows ? row : rows - 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            // past the row or the last row: some valid address, zeroed where dy is used
            const int cc = c < C ? c : 0;
            nx[i] = load_raw<IO, WHOLE, R::STEP>(x + r * xs, cc, C);
            ny[i] = load_raw<IO, WHOLE, R::STEP>(dy + r * dys, cc, C);
        }
        nmu = mean[r];
        nrs = rstd[r];
    };
    fetch((int64_t)blockIdx.x * RPB + grp);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += step) {
        const int64_t row = r0 + grp;
        Lanes<IO> xh[NV], g[NV];
        const float mu = nmu, rs = nrs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            xh[i] = widen<IO>(nx[i]);
            g[i] = widen<IO>(row < rows && c < C ? ny[i] : make_uint4(0, 0, 0, 0));
        }
        fetch(row + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            if (c < C && row < rows) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    // past the row's end dy reads 0, so nothing below counts there
                    xh[i].x[e] = (xh[i].x[e] - mu) * rs;
                    ab[i].x[e] += g[i].x[e];
                    aw[i].x[e] = __builtin_fmaf(g[i].x[e], xh[i].x[e], aw[i].x[e]);
                    g[i].x[e] *= wv[i].x[e];
                    s1 += g[i].x[e];
                    s2 = __builtin_fmaf(g[i].x[e], xh[i].x[e], s2);
                }
            }
        }
        const float m1 = row_sum<TPR>(s1, red[buf][0]) / n;
        const float m2 = row_sum<TPR>(s2, red[buf][1]) / n;
        buf ^= 1;
        if (row >= rows) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = R::first(i, lt);
            if (c >= C) continue;
            Lanes<IO> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.x[e] = rs * (g[i].x[e] - m1 - xh[i].x[e] * m2);
            store_raw<IO, WHOLE, R::STEP>(dx + row * dxs, c, C, o);
        }
    }
    if (!part) return;
    float* mine = part + (int64_t)blockIdx.x * 2 * C;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = R::first(i, lt) + e * R::STEP;
                if (c < C) {
                    mine[c] = aw[i].x[e];
                    mine[C + c] = ab[i].x[e];
                }
            }
    } else {
        // the row groups' shares, added in order
        constexpr int W = TPR * NV * V;
        for (int k = 0; k < RPB; ++k) {
            __syncthreads();
            if (grp == k) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const int c = R::first(i, lt) + e * R::STEP;
                        acc[c] = k ? acc[c] + aw[i].x[e] : aw[i].x[e];
                        acc[W + c] = k ? acc[W + c] + ab[i].x[e] : ab[i].x[e];
                    }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += NT) {
            mine[c] = acc[c];
            mine[C + c] = acc[W + c];
        }
    }
}

// dw, db from n shares of 2 C sums each: PCOL columns and 1024 / PCOL share lanes per workgroup,
// eight loads in flight a thread (512 shares of C = 1024: 4 us; 11 us for twice the shares with one
// load at a time).  16 and 8 columns give more workgroups and are 2-4% slower over the whole call.
constexpr int PCOL = 32;
constexpr int64_t PARAM_BLOCKS = 1 << 20;   // a launch holds fewer than 2^32 threads

template <class IO>
__global__ __launch_bounds__(1024) void ln_params(const float* __restrict__ part, int n, int C,
                                                  typename IO::T* __restrict__ dw,
                                                  typename IO::T* __restrict__ db)
{
    constexpr int PL = 1024 / PCOL;
    __shared__ float s[16][PCOL];
    const int cl = threadIdx.x % PCOL, pl = threadIdx.x / PCOL, wave = threadIdx.x >> 6;
    const int64_t cols = 2 * (int64_t)C;
    // more than one turn only past PARAM_BLOCKS workgroups
    for (int64_t c0 = (int64_t)blockIdx.x * PCOL; c0 < cols; c0 += (int64_t)gridDim.x * PCOL) {
        const int64_t col = c0 + cl;
        const bool in = col < cols;
        float v = 0.f;
#pragma unroll 8
        for (int p = pl; p < n; p += PL) v += part[(int64_t)p * cols + (in ? col : 0)];
#pragma unroll
        for (int m = PCOL; m < 64; m <<= 1) v += __shfl_xor(v, m);
        if ((threadIdx.x & 63) < PCOL) s[wave][cl] = v;
        __syncthreads();
        if (threadIdx.x < PCOL && in) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < 16; ++w) t += s[w][cl];
            if (col < C) {
                if (dw) IO::store(dw, col, t);
            } else if (db) {
                IO::store(db, col - C, t);
            }
        }
        __syncthreads();
    }
}

// ---- rows longer than the registers hold: one workgroup per row, the row re-read from cache

template <class IO, bool WHOLE>
__global__ __launch_bounds__(NT) void lnl_fwd(const typename IO::T* __restrict__ x,
                                              const typename IO::T* __restrict__ w,
                                              const typename IO::T* __restrict__ b,
                                              typename IO::T* __restrict__ y,
                                              float* __restrict__ mean, float* __restrict__ rstd,
                                              int64_t rows, int C, int64_t xs, int64_t ys,
                                              float eps)
{
    constexpr int V = vec_elems<IO>;
    using R = Columns<NT, V, WHOLE>;
    __shared__ float red[2][2][4];
    int buf = 0;
    const float n = (float)C;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const typename IO::T* xr = x + row * xs;
        float s = 0.f;
        for (int64_t c = R::first(0, threadIdx.x); c < C; c += NT * V) {
            const Lanes<IO> v = widen<IO>(load_raw<IO, WHOLE, R::STEP>(xr, (int)c, C));
#pragma unroll
            for (int e = 0; e < V; ++e) s += v.x[e];
        }
        const float mu = row_sum<NT>(s, red[buf][0]) / n;
        float q = 0.f;
        for (int64_t c = R::first(0, threadIdx.x); c < C; c += NT * V) {
            const Lanes<IO> v = widen<IO>(load_raw<IO, WHOLE, R::STEP>(xr, (int)c, C));
#pragma unroll
            for (int e = 0; e < V; ++e) q += c + e * R::STEP < C ? (v.x[e] - mu) * (v.x[e] - mu) : 0.f;
        }
        const float rs = 1.0f / sqrtf(row_sum<NT>(q, red[buf][1]) / n + eps);
        buf ^= 1;
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
        for (int64_t c = R::first(0, threadIdx.x); c < C; c += NT * V) {
            Lanes<IO> v = widen<IO>(load_raw<IO, WHOLE, R::STEP>(xr, (int)c, C));
            Lanes<IO> wv, bv;
            if (w) wv = widen<IO>(load_raw<IO, WHOLE, R::STEP>(w, (int)c, C));
            if (b) bv = widen<IO>(load_raw<IO, WHOLE, R::STEP>(b, (int)c, C));
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float t = (v.x[e] - mu) * rs;
                if (w) t *= wv.x[e];
                v.x[e] = b ? t + bv.x[e] : t;
            }
            store_raw<IO, WHOLE, R::STEP>(y + row * ys, (int)c, C, v);
        }
    }
}

template <class IO, bool WHOLE>
__global__ __launch_bounds__(NT) void lnl_bwd(const typename IO::T* __restrict__ dy,
                                              const typename IO::T* __restrict__ x,
                                              const typename IO::T* __restrict__ w,
                                              const float* __restrict__ mean,
                                              const float* __restrict__ rstd,
                                              typename IO::T* __restrict__ dx, int64_t rows, int C,
                                              int64_t dys, int64_t xs, int64_t dxs)
{
    constexpr int V = vec_elems<IO>;
    using R = Columns<NT, V, WHOLE>;
    __shared__ float red[2][2][4];
    int buf = 0;
    const float n = (float)C;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mu = mean[row], rs = rstd[row];
        auto terms = [&](int c, Lanes<IO>& e, Lanes<IO>& xh) {
            e = widen<IO>(load_raw<IO, WHOLE, R::STEP>(dy + row * dys, c, C));
            xh = widen<IO>(load_raw<IO, WHOLE, R::STEP>(x + row * xs, c, C));
            Lanes<IO> wv;
            if (w) wv = widen<IO>(load_raw<IO, WHOLE, R::STEP>(w, c, C));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh.x[i] = (xh.x[i] - mu) * rs;
                if (w) e.x[i] *= wv.x[i];
            }
        };
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = R::first(0, threadIdx.x); c < C; c += NT * V) {
            Lanes<IO> e, xh;
            terms((int)c, e, xh);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s1 += e.x[i];
                s2 = __builtin_fmaf(e.x[i], xh.x[i], s2);
            }
        }
        const float m1 = row_sum<NT>(s1, red[buf][0]) / n;
        const float m2 = row_sum<NT>(s2, red[buf][1]) / n;
        buf ^= 1;
        for (int64_t c = R::first(0, threadIdx.x); c < C; c += NT * V) {
            Lanes<IO> e, xh;
            terms((int)c, e, xh);
#pragma unroll
            for (int i = 0; i < V; ++i) e.x[i] = rs * (e.x[i] - m1 - xh.x[i] * m2);
            store_raw<IO, WHOLE, R::STEP>(dx + row * dxs, (int)c, C, e);
        }
    }
}

// shares of dw, db: workgroup (strip, column block) walks the rows of its strip
template <class IO>
__global__ __launch_bounds__(NT) void lnl_params(const typename IO::T* __restrict__ dy,
                                                 const typename IO::T* __restrict__ x,
                                                 const float* __restrict__ mean,
                                                 const float* __restrict__ rstd,
                                                 float* __restrict__ part, int64_t rows, int C,
                                                 int64_t dys, int64_t xs)
{
    const int c = blockIdx.x * NT + threadIdx.x, strip = blockIdx.y;
    if (c >= C) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t row = strip; row < rows; row += LNL_STRIPS) {
        const float g = IO::load(dy, row * dys + c);
        ab += g;
        aw = __builtin_fmaf(g, (IO::load(x, row * xs + c) - mean[row]) * rstd[row], aw);
    }
    float* mine = part + (int64_t)strip * 2 * C;
    mine[c] = aw;
    mine[C + c] = ab;
}

// (a null pointer counts as aligned: nothing is read there)
bool aligned_rows(const void* p, int64_t stride, size_t es)
{
    return (uintptr_t)p % 16 == 0 && stride * (int64_t)es % 16 == 0;
}

// Threads per row and vectors per thread for rows of C values: the fewest threads whose
// registers hold the row (16 or 64 threads need no barrier: rows of 768 float32 take 10.8 us for
// 8192 of them on 64 threads and 13.7 on 256; only backward rows of 2048 bfloat16 are 4% faster on
// 256).
struct RowPlan {
    int tpr, nv;   // nv 0: the row does not fit
};

RowPlan row_plan(int C, int V)
{
    const int vecs = (C + V - 1) / V;
    if (vecs <= 16) return {16, 1};
    if (vecs <= 64) return {64, 1};
    if (vecs <= 128) return {64, 2};
    if (vecs <= 256) return {64, 4};
    if (vecs <= 512) return {256, 2};
    if (vecs <= 1024) return {256, 4};
    if (vecs <= 2048 && V == 4) return {256, 8};
    return {256, 0};
}

// calls f(std::integral_constant<TPR>, std::integral_constant<NV>) for the plan
template <class F>
hipError_t with_plan(const RowPlan& p, F&& f)
{
    using std::integral_constant;
    if (p.tpr == 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (p.tpr == 64 && p.nv == 1) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (p.tpr == 64 && p.nv == 2) return f(integral_constant<int, 64>(), integral_constant<int, 2>());
    if (p.tpr == 64) return f(integral_constant<int, 64>(), integral_constant<int, 4>());
    if (p.nv == 2) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (p.nv == 4) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    return f(integral_constant<int, 256>(), integral_constant<int, 8>());
}

// Workgroups of the backward kernel: each writes 2 C sums, so no more than it takes to keep enough
// loads in flight.  bfloat16, 32768 x 1024: 256 workgroups 44.9 us, 512 39.8, 1024 42.1; float32,
// 8192 x 768: 19.1, 19.4, 22.9; bfloat16, 16384 x 2048: 44.2, 44.7, 52.5.
constexpr int64_t BWD_BLOCKS = 512;

int64_t bwd_blocks(int64_t rows, const RowPlan& p)
{
    const int64_t rpb = NT / p.tpr;
    return std::min<int64_t>(BWD_BLOCKS, (rows + rpb - 1) / rpb);
}

template <class IO, bool WHOLE>
hipError_t fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
               int64_t rows, int C, int64_t xs, int64_t ys, float eps, hipStream_t st)
{
    using E = typename IO::T;
    const RowPlan p = row_plan(C, vec_elems<IO>);
    // the row loop covers what a grid of this many workgroups leaves; element by element w and b cost
    // as many loads as a row, so a workgroup then keeps them for several rows (32768 of 1023 bfloat16
    // 57 us, 70 with a workgroup for each four rows, 66 with 1024 workgroups and 61 with 4096)
    const int64_t rpb = NT / p.tpr, blocks = std::min<int64_t>((rows + rpb - 1) / rpb, WHOLE ? 1 << 20 : 2048);
    if (p.nv == 0) {
        hipLaunchKernelGGL((lnl_fwd<IO, WHOLE>), dim3((unsigned)blocks), dim3(NT), 0, st, (const E*)x,
                           (const E*)w, (const E*)b, (E*)y, mean, rstd, rows, C, xs, ys, eps);
        return hipGetLastError();
    }
    return with_plan(p, [&](auto tpr, auto nv) {
        if constexpr (decltype(nv)::value == 8 && IO::SIZE == 2) return hipErrorInvalidValue;
        else {
            hipLaunchKernelGGL((ln_fwd<IO, decltype(tpr)::value, decltype(nv)::value, WHOLE>),
                               dim3((unsigned)blocks), dim3(NT), 0, st, (const E*)x, (const E*)w,
                               (const E*)b, (E*)y, mean, rstd, rows, C, xs, ys, eps);
            return hipGetLastError();
        }
    });
}

template <class IO, bool WHOLE>
hipError_t bwd(const void* dy, const void* x, const void* w, const float* mean, const float* rstd,
               void* dx, void* dw, void* db, int64_t rows, int C, int64_t dys, int64_t xs,
               int64_t dxs, float* part, hipStream_t st)
{
    using E = typename IO::T;
    const RowPlan p = row_plan(C, vec_elems<IO>);
    const bool params = dw || db;
    int64_t shares = 0;
    hipError_t e = hipSuccess;
    if (p.nv == 0) {
        const int64_t blocks = std::min<int64_t>(rows, 1 << 20);
        if (blocks > 0) {
            hipLaunchKernelGGL((lnl_bwd<IO, WHOLE>), dim3((unsigned)blocks), dim3(NT), 0, st,
                               (const E*)dy, (const E*)x, (const E*)w, mean, rstd, (E*)dx, rows, C,
                               dys, xs, dxs);
            e = hipGetLastError();
        }
        if (e == hipSuccess && params && rows > 0) {
            shares = LNL_STRIPS;
            hipLaunchKernelGGL((lnl_params<IO>), dim3((unsigned)((C + NT - 1) / NT), LNL_STRIPS),
                               dim3(NT), 0, st, (const E*)dy, (const E*)x, mean, rstd, part, rows,
                               C, dys, xs);
            e = hipGetLastError();
        }
    } else if (rows > 0) {
        shares = bwd_blocks(rows, p);
        e = with_plan(p, [&](auto tpr, auto nv) {
            if constexpr (decltype(nv)::value == 8 && IO::SIZE == 2) return hipErrorInvalidValue;
            else {
                hipLaunchKernelGGL((ln_bwd<IO, decltype(tpr)::value, decltype(nv)::value, WHOLE>),
                                   dim3((unsigned)shares), dim3(NT), 0, st, (const E*)dy,
                                   (const E*)x, (const E*)w, mean, rstd, (E*)dx,
                                   params ? part : nullptr, rows, C, dys, xs, dxs);
                return hipGetLastError();
            }
        });
    }
    if (e != hipSuccess || !params) return e;
    const int64_t blocks = std::min<int64_t>((2 * (int64_t)C + PCOL - 1) / PCOL, PARAM_BLOCKS);
    hipLaunchKernelGGL((ln_params<IO>), dim3((unsigned)blocks), dim3(1024), 0, st, part, (int)shares, C, (E*)dw,
                       (E*)db);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm(Store s, const void* x, const void* w, const void* b, void* y,
                            float* mean, float* rstd, int64_t rows, int C, int64_t xs, int64_t ys,
                            float eps, hipStream_t st)
{
    const size_t es = s == Store::F32 ? 4 : 2;
    const bool whole = C % (16 / es) == 0 && aligned_rows(x, xs, es) && aligned_rows(y, ys, es) &&
                       aligned_rows(w, 0, es) && aligned_rows(b, 0, es);
    auto f = s == Store::F32 ? (whole ? fwd<f32_io, true> : fwd<f32_io, false>)
                             : (whole ? fwd<bf16_io, true> : fwd<bf16_io, false>);
    return f(x, w, b, y, mean, rstd, rows, C, xs, ys, eps, st);
}

size_t layernorm_bwd_bytes(Store s, int64_t rows, int C)
{
    const RowPlan p = row_plan(C, s == Store::F32 ? 4 : 8);
    const int64_t shares = p.nv == 0 ? (rows > 0 ? LNL_STRIPS : 0) : bwd_blocks(rows, p);
    return (size_t)shares * 2 * (size_t)C * sizeof(float);
}

hipError_t launch_layernorm_bwd(Store s, const void* dy, const void* x, const void* w,
                                const float* mean, const float* rstd, void* dx, void* dw, void* db,
                                int64_t rows, int C, int64_t dys, int64_t xs, int64_t dxs,
                                void* ws, hipStream_t st)
{
    const size_t es = s == Store::F32 ? 4 : 2;
    const bool whole = C % (16 / es) == 0 && aligned_rows(dy, dys, es) && aligned_rows(x, xs, es) &&
                       aligned_rows(dx, dxs, es) && aligned_rows(w, 0, es);
    auto f = s == Store::F32 ? (whole ? bwd<f32_io, true> : bwd<f32_io, false>)
                             : (whole ? bwd<bf16_io, true> : bwd<bf16_io, false>);
    return f(dy, x, w, mean, rstd, dx, dw, db, rows, C, dys, xs, dxs, (float*)ws, st);
}

}  // namespace sc
