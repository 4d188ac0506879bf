// Gated linear recurrence along the tokens of (B, L, C) activations (gfx950).
//
//     f_t = sigmoid(z_t),   h_t = f_t h_{t-1} + (1 - f_t) u_t          (each channel its own)
//
// and, for the output gradient dh (and dhT, that of the last state),
//
//     g_t = dh_t + c_t,  c_{t-1} = f_t g_t  (c_{L-1} = dhT),
//     du_t = (1 - f_t) g_t,   dz_t = g_t (h_{t-1} - u_t) f_t (1 - f_t),   dh0 = c_{-1}.
//
// Both are first-order recurrences s <- a s + b, forward over t with (a, b) = (f, (1-f) u),
// backward over descending t with (f, f dh), and pairs compose as (a2, b2) o (a1, b1) =
// (a2 a1, a2 b1 + b2).  Bound by memory: 3 elements a value forward, 6 backward, so the data
// passes once: a workgroup owns 32 channels of one batch row and walks the tokens in tiles.
// Lane (tl, cl) holds R consecutive tokens of one 16-byte channel vector; it folds them into
// one pair, the pairs are scanned over the token lanes by wave shuffles and over the four waves
// through LDS, and h_t = (local h_t) + (product of f up to t) * (state before the lane).  The
// next tile's loads are issued before this tile is folded.
// With few channels (B C / 32 workgroups do not fill the GPU) the tokens are cut into
// segments: a first pass folds each segment into its pair (reads only), a small kernel chains
// the pairs, and the same walk runs on every segment with its state.  The order of all
// compositions depends on the shape alone, so results repeat bit for bit.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_internal.h"
#include "sc_rows.h"

namespace sc {

namespace {

constexpr int NT = 256;    // threads
constexpr int NW = NT / 64;
constexpr int CG = 32;     // channels of a workgroup

// e = exp(-|z|) keeps both gates exact where the other saturates: f = 1/(1+e) or e/(1+e)
__device__ __forceinline__ void gates(float z, float& f, float& k)
{
    const float e = __expf(-fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;   // about 1 ulp
    f = z >= 0.f ? r : s;
    k = z >= 0.f ? s : r;
}

struct Args {
    const void *z, *u, *h, *dh;   // forward reads z, u; backward z, u, h, dh
    void *o0, *o1;                // forward h; backward dz, du
    const float* s0;              // state before the first token of the walk (h0 or dhT), or null
    float* s1;                    // state after the last (hT or dh0), or null
    const float* hinit;           // backward: h0, the h before token 0, or null
    float* seg;                   // segment pairs [B][nseg][2][C] (fold) / states (walk)
    int64_t L, zs, us, hs, dhs, os0, os1;   // token strides
    int C, ngroups, nseg;
    int64_t slen;                 // tokens of a segment
    int whole;                    // every row of every array starts 16-byte aligned
};

// FOLD: only the segment's pair is wanted (nothing written but seg)
template <class IO, bool BWD, bool FOLD, int R>
__global__ __launch_bounds__(NT) void recur_tiles(Args a)
{
    using E = typename IO::T;
    constexpr int V = vec_elems<IO>, LPT = CG / V, TL = 64 / LPT;
    constexpr int T = NW * TL * R;   // tokens of a tile
    constexpr bool LOAD_U = !BWD || !FOLD;
    __shared__ float tot[2][NW][2][CG];   // the waves' pairs, double-buffered over tiles

    uint32_t id = blockIdx.x;
    const int grp = (int)(id % (uint32_t)a.ngroups);
    id /= (uint32_t)a.ngroups;
    const int sg = (int)(id % (uint32_t)a.nseg);
    const int64_t b = id / (uint32_t)a.nseg;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cl = lane % LPT, tl = lane / LPT;
    const int c0 = grp * CG + cl * V, C = a.C;
    const bool con = c0 < C;
    const int64_t L = a.L;
    const int64_t lo = (int64_t)sg * a.slen, hi = std::min<int64_t>(L, lo + a.slen);
    const E* zp = (const E*)a.z + b * L * a.zs;
    const E* up = (const E*)a.u + b * L * a.us;
    const E* hp = BWD ? (const E*)a.h + b * L * a.hs : nullptr;
    const E* dp = BWD ? (const E*)a.dh + b * L * a.dhs : nullptr;

    float carry[V];
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = 0.f;
    float cprod[FOLD ? V : 1];   // FOLD: the product of a over the segment so far
    if constexpr (FOLD) {
#pragma unroll
        for (int e = 0; e < V; ++e) cprod[e] = 1.f;
    } else if (con) {
        const float* s = a.nseg > 1 ? a.seg + (b * a.nseg + sg) * 2 * C : a.s0 ? a.s0 + b * C : nullptr;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (s && c0 + e < C) carry[e] = s[c0 + e];
    }

    // token r of this lane in the tile that starts `n` tokens into the segment (in walk order)
    auto token = [&](int64_t n, int r) -> int64_t {
        const int64_t k = n + (wave * TL + tl) * R + r;
        return BWD ? hi - 1 - k : lo + k;
    };
    auto valid = [&](int64_t t) { return con && t >= lo && t < hi; };

    uint4 rz[R], ru[LOAD_U ? R : 1], rd[BWD ? R : 1], rh[BWD && !FOLD ? R : 1];
    auto fetch = [&](int64_t n) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = token(n, r);
            const bool on = valid(t);
            const uint4 zero = make_uint4(0, 0, 0, 0);
            rz[r] = on ? load_raw<IO>(zp + t * a.zs, c0, C, a.whole) : zero;
            if constexpr (LOAD_U) ru[r] = on ? load_raw<IO>(up + t * a.us, c0, C, a.whole) : zero;
            if constexpr (BWD) rd[r] = on ? load_raw<IO>(dp + t * a.dhs, c0, C, a.whole) : zero;
            if constexpr (BWD && !FOLD)
                rh[r] = on && t > 0 ? load_raw<IO>(hp + (t - 1) * a.hs, c0, C, a.whole) : zero;
        }
    };
    fetch(0);
    int buf = 0;
    for (int64_t n = 0; n < hi - lo; n += T, buf ^= 1) {
        // fold the lane's tokens: after token r, P[r] = product of a up to and with r,
        // S[r] = the state there for a zero state before the lane
        Lanes<IO> P[R], S[R];
        Lanes<IO> du[BWD && !FOLD ? R : 1], dz[BWD && !FOLD ? R : 1];   // factors of g
        float pa[V], ps[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            pa[e] = 1.f;
            ps[e] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = token(n, r);
            const bool on = valid(t);
            const Lanes<IO> z = widen<IO>(rz[r]);
            Lanes<IO> u, d, h;
            if constexpr (LOAD_U) u = widen<IO>(ru[r]);
            if constexpr (BWD) d = widen<IO>(rd[r]);
            if constexpr (BWD && !FOLD) {
                h = widen<IO>(rh[r]);
                if (on && t == 0 && a.hinit) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c0 + e < C) h.x[e] = a.hinit[b * C + c0 + e];
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float f, k;
                gates(z.x[e], f, k);
                if constexpr (!BWD) {
                    ps[e] = on ? __builtin_fmaf(f, ps[e], k * u.x[e]) : ps[e];
                    pa[e] = on ? f * pa[e] : pa[e];
                    P[r].x[e] = pa[e];
                    S[r].x[e] = ps[e];
                } else {
                    // g_t = (dh_t + local c) + (product before t) * (state before the lane)
                    const float g = d.x[e] + ps[e];
                    S[r].x[e] = g;
                    P[r].x[e] = pa[e];
                    ps[e] = on ? f * g : ps[e];
                    pa[e] = on ? f * pa[e] : pa[e];
                    if constexpr (!FOLD) {
                        du[r].x[e] = k;
                        dz[r].x[e] = (h.x[e] - u.x[e]) * (f * k);
                    }
                }
            }
        }
        if (n + T < hi - lo) fetch(n + T);
        // inclusive scan of the lanes' pairs over the wave's token lanes
        float xa[V], xs[V];   // then: the pair before this lane (exclusive)
#pragma unroll
        for (int m = 1; m < TL; m <<= 1) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float qa = __shfl_up(pa[e], m * LPT), qs = __shfl_up(ps[e], m * LPT);
                if (tl >= m) {
                    ps[e] = __builtin_fmaf(pa[e], qs, ps[e]);
                    pa[e] *= qa;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float qa = __shfl_up(pa[e], LPT), qs = __shfl_up(ps[e], LPT);
            xa[e] = tl ? qa : 1.f;
            xs[e] = tl ? qs : 0.f;
        }
        if (tl == TL - 1) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                tot[buf][wave][0][cl * V + e] = pa[e];
                tot[buf][wave][1][cl * V + e] = ps[e];
            }
        }
        __syncthreads();
        // the state before this wave, and the one after the tile
        float st[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float s = carry[e];
            st[e] = s;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float wa = tot[buf][w][0][cl * V + e];
                if (w == wave) st[e] = s;
                s = __builtin_fmaf(wa, s, tot[buf][w][1][cl * V + e]);
                if constexpr (FOLD) cprod[e] *= wa;
            }
            carry[e] = s;
        }
        if constexpr (!FOLD) {
#pragma unroll
            for (int e = 0; e < V; ++e) st[e] = __builtin_fmaf(xa[e], st[e], xs[e]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t t = token(n, r);
                if (!valid(t)) continue;
                Lanes<IO> o, o2;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float v = __builtin_fmaf(P[r].x[e], st[e], S[r].x[e]);
                    if constexpr (BWD) {
                        o.x[e] = dz[r].x[e] * v;
                        o2.x[e] = du[r].x[e] * v;
                    } else {
                        o.x[e] = v;
                    }
                }
                store_raw<IO>((E*)a.o0 + (b * L + t) * a.os0, c0, C, a.whole, o);
                if constexpr (BWD) store_raw<IO>((E*)a.o1 + (b * L + t) * a.os1, c0, C, a.whole, o2);
            }
        }
    }
    __syncthreads();   // every lane has used its initial state: s1 may be s0's memory
    if (!con || wave != 0 || tl != 0) return;
    if constexpr (FOLD) {
        float* s = a.seg + (b * a.nseg + sg) * 2 * C;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c0 + e < C) {
                s[c0 + e] = cprod[e];
                s[C + c0 + e] = carry[e];
            }
    } else if (a.nseg == 1 && a.s1) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c0 + e < C) a.s1[b * C + c0 + e] = carry[e];
    }
}

// The segments' pairs chained in walk order (segment nseg-1 first for the backward pass): each
// pair's first half becomes the state before its segment; the last state goes to s1.
__global__ __launch_bounds__(NT) void recur_chain(float* seg, const float* s0, float* s1,
                                                  int64_t n, int C, int nseg, int down)
{
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= n) return;
    const int64_t b = i / C, c = i % C;
    float s = s0 ? s0[i] : 0.f;
    for (int k = 0; k < nseg; ++k) {
        float* p = seg + (b * nseg + (down ? nseg - 1 - k : k)) * 2 * C + c;
        const float fa = p[0], fb = p[C];
        p[0] = s;
        s = __builtin_fmaf(fa, s, fb);
    }
    if (s1) s1[i] = s;
}

// Few tokens: one thread per batch row and channel vector walks them.
template <class IO, bool BWD>
__global__ __launch_bounds__(64) void recur_walk(Args a, int64_t n, int nvec)
{
    using E = typename IO::T;
    constexpr int V = vec_elems<IO>;
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (i >= n) return;
    const int64_t b = i / nvec;
    const int c0 = (int)(i % nvec) * V, C = a.C;
    float s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = a.s0 && c0 + e < C ? a.s0[b * C + c0 + e] : 0.f;
    for (int64_t k = 0; k < a.L; ++k) {
        const int64_t t = b * a.L + (BWD ? a.L - 1 - k : k);
        const Lanes<IO> z = widen<IO>(load_raw<IO>((const E*)a.z + t * a.zs, c0, C, a.whole));
        const Lanes<IO> u = widen<IO>(load_raw<IO>((const E*)a.u + t * a.us, c0, C, a.whole));
        Lanes<IO> o, o2;
        if constexpr (BWD) {
            const Lanes<IO> d = widen<IO>(load_raw<IO>((const E*)a.dh + t * a.dhs, c0, C, a.whole));
            Lanes<IO> h;
            if (k + 1 < a.L) h = widen<IO>(load_raw<IO>((const E*)a.h + (t - 1) * a.hs, c0, C, a.whole));
            else
#pragma unroll
                for (int e = 0; e < V; ++e) h.x[e] = a.hinit && c0 + e < C ? a.hinit[b * C + c0 + e] : 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float f, q;
                gates(z.x[e], f, q);
                const float g = d.x[e] + s[e];
                o.x[e] = (h.x[e] - u.x[e]) * (f * q) * g;
                o2.x[e] = q * g;
                s[e] = f * g;
            }
            store_raw<IO>((E*)a.o1 + t * a.os1, c0, C, a.whole, o2);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float f, q;
                gates(z.x[e], f, q);
                s[e] = __builtin_fmaf(f, s[e], q * u.x[e]);
                o.x[e] = s[e];
            }
        }
        store_raw<IO>((E*)a.o0 + t * a.os0, c0, C, a.whole, o);
    }
    if (!a.s1) return;
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (c0 + e < C) a.s1[b * C + c0 + e] = s[e];
}

// Lengths up to this are walked by single threads.
constexpr int64_t WALK_MAX_L = 16;
// Workgroups below which the tokens are cut into segments, and the shortest segment.
constexpr int64_t FILL = 512;
constexpr int64_t SEG_MIN = 1024;

struct Plan {
    int64_t nseg, slen, ngroups;
};

Plan plan(int64_t B, int64_t L, int C)
{
    Plan p{1, L, (C + CG - 1) / CG};
    const int64_t wgs = B * p.ngroups;
    if (L <= WALK_MAX_L || wgs <= 0 || 2 * wgs > FILL) return p;
    const int64_t want = std::min<int64_t>((FILL + wgs - 1) / wgs, L / SEG_MIN);
    if (want < 2) return p;
    // whole tiles (256 tokens) per segment
    p.slen = ((L + want - 1) / want + 255) / 256 * 256;
    p.nseg = (L + p.slen - 1) / p.slen;
    return p;
}

template <class IO, bool BWD>
hipError_t go(Args a, int64_t B, hipStream_t st)
{
    constexpr int V = vec_elems<IO>;
    if (a.L <= WALK_MAX_L) {
        const int nvec = (a.C + V - 1) / V;
        const int64_t n = B * nvec, blocks = (n + 63) / 64;
        if (!grid_ok(blocks, 64)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((recur_walk<IO, BWD>), dim3((unsigned)blocks), dim3(64), 0, st, a, n, nvec);
        return hipGetLastError();
    }
    constexpr int R = BWD ? (V == 8 ? 2 : 4) : (V == 8 ? 4 : 8);
    const Plan p = plan(B, a.L, a.C);
    a.ngroups = (int)p.ngroups;
    a.nseg = (int)p.nseg;
    a.slen = p.slen;
    const int64_t blocks = B * p.ngroups * p.nseg;
    if (!grid_ok(blocks, NT)) return hipErrorInvalidValue;
    if (p.nseg > 1) {
        hipLaunchKernelGGL((recur_tiles<IO, BWD, true, R>), dim3((unsigned)blocks), dim3(NT), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t n = B * a.C;
        hipLaunchKernelGGL(recur_chain, dim3((unsigned)((n + NT - 1) / NT)), dim3(NT), 0, st, a.seg, a.s0,
                           a.s1, n, a.C, a.nseg, BWD ? 1 : 0);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((recur_tiles<IO, BWD, false, R>), dim3((unsigned)blocks), dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

size_t recur_bytes(int64_t B, int64_t L, int C)
{
    const Plan p = plan(B, L, C);
    return p.nseg > 1 ? (size_t)B * p.nseg * 2 * C * sizeof(float) : 0;
}

hipError_t launch_recur(Store s, const RecurFwd& r, int64_t B, int64_t L, int C, void* ws,
                        hipStream_t st)
{
    Args a{};
    a.z = r.z; a.u = r.u; a.o0 = r.h; a.s0 = r.h0; a.s1 = r.hT; a.seg = (float*)ws;
    a.L = L; a.C = C; a.zs = r.zs; a.us = r.us; a.os0 = r.hs; a.whole = r.whole;
    return s == Store::F32 ? go<f32_io, false>(a, B, st) : go<bf16_io, false>(a, B, st);
}

hipError_t launch_recur_bwd(Store s, const RecurBwd& r, int64_t B, int64_t L, int C, void* ws,
                            hipStream_t st)
{
    Args a{};
    a.z = r.z; a.u = r.u; a.h = r.h; a.dh = r.dh; a.o0 = r.dz; a.o1 = r.du; a.s0 = r.dhT;
    a.s1 = r.dh0; a.hinit = r.h0; a.seg = (float*)ws;
    a.L = L; a.C = C; a.zs = r.zs; a.us = r.us; a.hs = r.hs; a.dhs = r.dhs; a.os0 = r.dzs;
    a.os1 = r.dus; a.whole = r.whole;
    return s == Store::F32 ? go<f32_io, true>(a, B, st) : go<bf16_io, true>(a, B, st);
}

}  // namespace sc
