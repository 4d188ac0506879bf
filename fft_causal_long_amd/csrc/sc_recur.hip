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
// A lane holds R consecutive tokens of NC channels, folds them into one pair per channel, the
// pairs are scanned over the wave's token lanes by shuffles and over the waves through LDS, and
// h_t = (local h_t) + (product of f up to t) * (state before the lane).  The next tile's loads
// are issued as soon as this tile is folded, in a loop without branches.
// With few channels (B C / 32 workgroups do not fill the GPU) the tokens are cut into
// segments: a first pass folds each segment into its pair (reads only), a small kernel chains
// the pairs, and the same walk runs on every segment with its state.  The order of all
// compositions depends on the shape alone, so results repeat bit for bit.
//
// Measured (MI355X): B 8, L 4096, C 1024 bfloat16 forward 50.6 us (4.0 TB/s of the bytes it
// cannot do without; a large copy reaches 5.4), backward 111 us (3.6); B 8, L 1024, C 768
// float32 backward 34 us (4.4); B 1, L 65536, C 1536 float32 forward 428 us, where the fold
// reads z and u a second time (2.0 GB in all, 4.7 TB/s); its three kernels take 184, 5 and 240 us.
// NC, R and the waves were chosen there: for bfloat16 forward, 2 channels and 8 tokens a lane took
// 50.6 us, 4 x 8 54.2, 8 x 4 55.2 (more shuffles a value); 4 waves a workgroup 61, and loads two tiles
// ahead 60; for float32 4 x 4 and 2 x 8 are within 2%.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sc_internal.h"
#include "sc_rows.h"

namespace sc {

namespace {

constexpr int NT = 256;    // threads of the small kernels
constexpr int CG = 32;     // channels of a workgroup

// f = 1 / (1 + e), 1 - f = e f with e = exp(-z): neither loses its relative precision where the other
// saturates.  The rounding of the exponent moves e, and the smaller gate with it, by about |z| units
// of 2^-24 (31 at |z| = 40); beside it a few ulp.  The exponent stops at 2^125, below which the
// reciprocal is a normal number (past 2^126 it is flushed to 0, and e f with it), so f stays at 2^-125
// for z below -86.6; a comparison, not a minimum, so a NaN in z stays.
__device__ __forceinline__ void gates(float z, float& f, float& k)
{
    const float t = z * -1.44269504088896340736f;
    const float e = __builtin_amdgcn_exp2f(t > 125.0f ? 125.0f : t);
    f = __builtin_amdgcn_rcpf(1.0f + e);   // about 1 ulp
    k = e * f;
}

// NC neighbouring channels of a row as stored (4, 8 or 16 bytes).
template <class IO, int NC>
struct Pack {
    static constexpr int NWORD = NC * IO::SIZE / 4;
    typedef uint32_t Word __attribute__((ext_vector_type(NWORD < 2 ? 2 : NWORD)));
    typedef typename std::conditional<NWORD == 1, uint32_t, Word>::type Raw;

    // WHOLE: the vector is aligned and all its channels exist
    template <bool WHOLE>
    __device__ __forceinline__ static Raw load(const typename IO::T* p, int c, int C)
    {
        if constexpr (WHOLE) {
            return *(const Raw*)(p + c);
        } else {
            uint32_t w[NWORD] = {};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int at = c + i < C ? c + i : C - 1;   // a channel past the last repeats it
                if constexpr (IO::SIZE == 2) w[i / 2] |= (uint32_t)p[at] << (16 * (i & 1));
                else w[i] = __float_as_uint(p[at]);
            }
            Raw r;
            if constexpr (NWORD == 1) r = w[0];
            else
#pragma unroll
                for (int i = 0; i < NWORD; ++i) r[i] = w[i];
            return r;
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ static void store(typename IO::T* p, int c, int C, const float (&v)[NC])
    {
        if constexpr (WHOLE) {
            Raw r;
            if constexpr (NWORD == 1) r = pack_bf16x2(v[0], v[1]);
            else
#pragma unroll
                for (int i = 0; i < NWORD; ++i) {
                    if constexpr (IO::SIZE == 2) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    else r[i] = __float_as_uint(v[i]);
                }
            *(Raw*)(p + c) = r;
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (c + i < C) IO::store(p, c + i, v[i]);
        }
    }
    __device__ __forceinline__ static float at(const Raw& r, int e)
    {
        uint32_t w;
        if constexpr (NWORD == 1) w = r;
        else w = r[e * IO::SIZE / 4];
        if constexpr (IO::SIZE == 2) return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
        else return __uint_as_float(w);
    }
    __device__ __forceinline__ static Raw fill(uint32_t w)
    {
        if constexpr (NWORD == 1) return w;
        else return (Raw)w;
    }
};

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
};

// FOLD: only the segment's pair is wanted (nothing written but seg)
template <class IO, bool BWD, bool FOLD, int MODE, int NC, int R, int NW>
__global__ __launch_bounds__(64 * NW) void recur_tiles(Args a)
{
    using E = typename IO::T;
    using PK = Pack<IO, NC>;
    typedef typename PK::Raw Word;
    constexpr int LPT = CG / NC, TL = 64 / LPT;
    constexpr int T = NW * TL * R;   // tokens of a tile
    constexpr bool LOAD_U = !BWD || !FOLD, LOAD_H = BWD && !FOLD, WHOLE = MODE > 0;
    __shared__ float tot[2][NW][2][CG];   // the waves' pairs, double-buffered over tiles

    uint32_t id = die_order(blockIdx.x, gridDim.x);
    const int grp = (int)(id % (uint32_t)a.ngroups);
    id /= (uint32_t)a.ngroups;
    const int sg = (int)(id % (uint32_t)a.nseg);
    const int64_t b = id / (uint32_t)a.nseg;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cl = lane % LPT, tl = lane / LPT;
    const int c0 = grp * CG + cl * NC, C = a.C;
    const bool con = MODE == 2 || c0 < C;
    const int cc = con ? c0 : 0;   // a lane past the channels reads some valid address
    const int64_t L = a.L;
    const int64_t lo = (int64_t)sg * a.slen, hi = std::min<int64_t>(L, lo + a.slen), len = hi - lo;
    const int64_t k0 = (wave * TL + tl) * R;   // the lane's first token within a tile
    // token k of the segment in walk order
    auto token = [&](int64_t k) -> int64_t { return BWD ? hi - 1 - k : lo + k; };
    const E* zp = (const E*)a.z + b * L * a.zs;
    const E* up = (const E*)a.u + b * L * a.us;
    const E* hp = BWD ? (const E*)a.h + b * L * a.hs : nullptr;
    const E* dp = BWD ? (const E*)a.dh + b * L * a.dhs : nullptr;

    float carry[NC], cprod[NC], hfirst[NC];   // cprod (FOLD): product of a so far; the h before token 0
#pragma unroll
    for (int e = 0; e < NC; ++e) {
        carry[e] = hfirst[e] = 0.f;
        cprod[e] = 1.f;
    }
    if constexpr (!FOLD) {
        const float* s = a.nseg > 1 ? a.seg + (b * a.nseg + sg) * 2 * C : a.s0 ? a.s0 + b * C : nullptr;
#pragma unroll
        for (int e = 0; e < NC; ++e)
            if (s && c0 + e < C) carry[e] = s[c0 + e];
    }
    if constexpr (LOAD_H) {
#pragma unroll
        for (int e = 0; e < NC; ++e)
            if (a.hinit && c0 + e < C) hfirst[e] = a.hinit[b * C + c0 + e];
    }
    constexpr uint32_t INF = IO::SIZE == 2 ? 0x7f807f80u : 0x7f800000u;

    struct Raw {
        Word z[R], u[LOAD_U ? R : 1], d[BWD ? R : 1], h[LOAD_H ? R : 1];
    };
    // a tile of which every token exists (and, for h, the one before it)
    auto fetch = [&](int64_t n, Raw& raw) {
        const int64_t t = token(n + k0);
        const E *z = zp + t * a.zs, *u = up + t * a.us, *d = dp + t * a.dhs, *h = hp + (t - 1) * a.hs;
        const int64_t sz = BWD ? -a.zs : a.zs, su = BWD ? -a.us : a.us;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            raw.z[r] = PK::template load<WHOLE>(z + r * sz, cc, C);
            if constexpr (LOAD_U) raw.u[r] = PK::template load<WHOLE>(u + r * su, cc, C);
            if constexpr (BWD) raw.d[r] = PK::template load<WHOLE>(d - r * a.dhs, cc, C);
            if constexpr (LOAD_H) raw.h[r] = PK::template load<WHOLE>(h - r * a.hs, cc, C);
        }
    };
    // any tile
    auto fetch_end = [&](int64_t n, Raw& raw) {
        // past the segment's end: a valid address, and z = inf, the rest 0 in its place (the gate
        // 1 leaves the state as it is)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t k = n + k0 + r;
            const bool on = k < len;
            const int64_t t = token(on ? k : len - 1);
            const Word z = PK::template load<WHOLE>(zp + t * a.zs, cc, C);
            raw.z[r] = on ? z : PK::fill(INF);
            if constexpr (LOAD_U) {
                const Word u = PK::template load<WHOLE>(up + t * a.us, cc, C);
                raw.u[r] = on ? u : PK::fill(0);
            }
            if constexpr (BWD) {
                const Word d = PK::template load<WHOLE>(dp + t * a.dhs, cc, C);
                raw.d[r] = on ? d : PK::fill(0);
            }
            if constexpr (LOAD_H) raw.h[r] = PK::template load<WHOLE>(hp + (t > 0 ? t - 1 : 0) * a.hs, cc, C);
        }
    };
    // one tile: fold what `raw` holds, refill it with the next tile, finish.  `steady`: both
    // tiles are whole, so loads and stores are issued without branches and the wait for the next
    // tile's loads does not include this tile's stores (a wait behind a branch waits for all).
    auto tile = [&](int64_t n, int buf, Raw& raw, auto steady) {
        constexpr bool STEADY = decltype(steady)::value;
        const int64_t t0 = token(n + k0);
        // fold the lane's tokens: after token r, P[r] = product of a up to and with r, S[r] = the
        // state there for a zero state before the lane (backward: up to but without r, and g)
        float P[R][NC], S[R][NC], du[LOAD_H ? R : 1][NC], dz[LOAD_H ? R : 1][NC];   // du, dz: factors of g
        float pa[NC], ps[NC];
#pragma unroll
        for (int e = 0; e < NC; ++e) {
            pa[e] = 1.f;
            ps[e] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                float f, k;
                gates(PK::at(raw.z[r], e), f, k);
                if constexpr (!BWD) {
                    ps[e] = __builtin_fmaf(f, ps[e], k * PK::at(raw.u[r], e));
                    pa[e] *= f;
                    P[r][e] = pa[e];
                    S[r][e] = ps[e];
                } else {
                    // g_t = (dh_t + local c) + (product before t) * (state before the lane)
                    const float g = PK::at(raw.d[r], e) + ps[e];
                    S[r][e] = g;
                    P[r][e] = pa[e];
                    ps[e] = f * g;
                    pa[e] *= f;
                    if constexpr (LOAD_H) {
                        const float h = t0 - r == 0 ? hfirst[e] : PK::at(raw.h[r], e);
                        du[r][e] = k;
                        dz[r][e] = (h - PK::at(raw.u[r], e)) * (f * k);
                    }
                }
            }
        if constexpr (STEADY) fetch(n + T, raw);
        else if (n + T < len) fetch_end(n + T, raw);
        // inclusive scan of the lanes' pairs over the wave's token lanes, then exclusive
        float xa[NC], xs[NC];
#pragma unroll
        for (int e = 0; e < NC; ++e) {
#pragma unroll
            for (int m = 1; m < TL; m <<= 1) {
                const float qa = __shfl_up(pa[e], m * LPT), qs = __shfl_up(ps[e], m * LPT);
                ps[e] = tl >= m ? __builtin_fmaf(pa[e], qs, ps[e]) : ps[e];
                pa[e] = tl >= m ? pa[e] * qa : pa[e];
            }
            const float qa = __shfl_up(pa[e], LPT), qs = __shfl_up(ps[e], LPT);
            xa[e] = tl ? qa : 1.f;
            xs[e] = tl ? qs : 0.f;
        }
        if (tl == TL - 1) {
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                tot[buf][wave][0][cl * NC + e] = pa[e];
                tot[buf][wave][1][cl * NC + e] = ps[e];
            }
        }
        __syncthreads();
        // the state before this wave, and the one after the tile
        float st[NC];
#pragma unroll
        for (int e = 0; e < NC; ++e) st[e] = carry[e];
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                const float wa = tot[buf][w][0][cl * NC + e], ws = tot[buf][w][1][cl * NC + e];
                if (w == wave) st[e] = carry[e];
                carry[e] = __builtin_fmaf(wa, carry[e], ws);
                if constexpr (FOLD) cprod[e] *= wa;
            }
        if constexpr (!FOLD) {
#pragma unroll
            for (int e = 0; e < NC; ++e) st[e] = __builtin_fmaf(xa[e], st[e], xs[e]);
            E* o0 = (E*)a.o0 + (b * L + t0) * a.os0;
            E* o1 = BWD ? (E*)a.o1 + (b * L + t0) * a.os1 : nullptr;
            const int64_t q0 = BWD ? -a.os0 : a.os0;
            auto put = [&](int r) {
                float v[NC], w[NC];
#pragma unroll
                for (int e = 0; e < NC; ++e) {
                    v[e] = __builtin_fmaf(P[r][e], st[e], S[r][e]);
                    if constexpr (BWD) {
                        w[e] = du[r][e] * v[e];
                        v[e] *= dz[r][e];
                    }
                }
                PK::template store<WHOLE>(o0 + r * q0, c0, C, v);
                if constexpr (BWD) PK::template store<WHOLE>(o1 - r * a.os1, c0, C, w);
            };
            if constexpr (STEADY) {
                if (con) {
#pragma unroll
                    for (int r = 0; r < R; ++r) put(r);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (con && n + k0 + r < len) put(r);
            }
        }
    };
    Raw raw;
    int64_t n = 0;
    int buf = 0;
    if (T + (LOAD_H ? 1 : 0) <= len) fetch(0, raw);
    else fetch_end(0, raw);
    for (; n + 2 * T + (LOAD_H ? 1 : 0) <= len; n += T, buf ^= 1) tile(n, buf, raw, std::true_type());
    for (; n < len; n += T, buf ^= 1) tile(n, buf, raw, std::false_type());
    __syncthreads();   // every lane has used its initial state: s1 may be s0's memory
    if (!con || wave != 0 || tl != 0) return;
    if constexpr (FOLD) {
        float* s = a.seg + (b * a.nseg + sg) * 2 * C;
#pragma unroll
        for (int e = 0; e < NC; ++e)
            if (c0 + e < C) {
                s[c0 + e] = cprod[e];
                s[C + c0 + e] = carry[e];
            }
    } else if (a.nseg == 1 && a.s1) {
#pragma unroll
        for (int e = 0; e < NC; ++e)
            if (c0 + e < C) a.s1[b * C + c0 + e] = carry[e];
    }
}

// The segments' pairs chained in walk order (segment nseg-1 first for the backward pass): each
// pair's first half becomes the state before its segment; the last state goes to s1.  Eight pairs
// are read at a time, so that their loads overlap.
__global__ __launch_bounds__(NT) void recur_chain(float* seg, const float* s0, float* s1,
                                                  int64_t n, int C, int nseg, int down)
{
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= n) return;
    const int64_t b = i / C, c = i % C;
    float s = s0 ? s0[i] : 0.f;
    for (int k0 = 0; k0 < nseg; k0 += 8) {
        float *p[8], fa[8], fb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = min(k0 + e, nseg - 1);
            p[e] = seg + (b * nseg + (down ? nseg - 1 - k : k)) * 2 * C + c;
            fa[e] = p[e][0];
            fb[e] = p[e][C];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k0 + e < nseg) {
                p[e][0] = s;
                s = __builtin_fmaf(fa[e], s, fb[e]);
            }
    }
    if (s1) s1[i] = s;
}

// Few tokens: one thread per batch row and channel vector walks them.
template <class IO, bool BWD, bool WHOLE>
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
        const Lanes<IO> z = widen<IO>(load_raw<IO, WHOLE>((const E*)a.z + t * a.zs, c0, C));
        const Lanes<IO> u = widen<IO>(load_raw<IO, WHOLE>((const E*)a.u + t * a.us, c0, C));
        Lanes<IO> o, o2;
        if constexpr (BWD) {
            const Lanes<IO> d = widen<IO>(load_raw<IO, WHOLE>((const E*)a.dh + t * a.dhs, c0, C));
            Lanes<IO> h;
            if (k + 1 < a.L) h = widen<IO>(load_raw<IO, WHOLE>((const E*)a.h + (t - 1) * a.hs, c0, C));
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
            store_raw<IO, WHOLE>((E*)a.o1 + t * a.os1, c0, C, o2);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float f, q;
                gates(z.x[e], f, q);
                s[e] = __builtin_fmaf(f, s[e], q * u.x[e]);
                o.x[e] = s[e];
            }
        }
        store_raw<IO, WHOLE>((E*)a.o0 + t * a.os0, c0, C, o);
    }
    if (!a.s1) return;
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (c0 + e < C) a.s1[b * C + c0 + e] = s[e];
}

// Lengths up to this are walked by single threads: one token of 8 sequences, C 1024, bfloat16, takes
// 4.4 us and 5.4 by tiles; 32 tokens 17 us and under 11.
constexpr int64_t WALK_MAX_L = 16;
// With fewer than ENOUGH workgroups (one per CU) the tokens are cut into segments of at least
// SEG_MIN tokens, FILL workgroups in all.  The long case above: 1024 workgroups 437 us (with a
// slower chain kernel), 512 469, 256 569, unsplit 719; the first case has 256 and takes 50.6 us whole,
// 97 in two segments.
constexpr int64_t ENOUGH = 256, FILL = 1024;
constexpr int64_t SEG_MIN = 1024;

struct Plan {
    int64_t nseg, slen, ngroups;
};

Plan plan(int64_t B, int64_t L, int C)
{
    Plan p{1, L, (C + CG - 1) / CG};
    const int64_t wgs = B * p.ngroups;
    if (L <= WALK_MAX_L || wgs <= 0 || wgs >= ENOUGH) return p;
    const int64_t want = std::min<int64_t>((FILL + wgs - 1) / wgs, L / SEG_MIN);
    if (want < 2) return p;
    // a multiple of every form's tile (128 or 256 tokens)
    p.slen = ((L + want - 1) / want + 255) / 256 * 256;
    p.nseg = (L + p.slen - 1) / p.slen;
    return p;
}

template <class IO, bool BWD, int MODE>
hipError_t go(Args a, int64_t B, hipStream_t st)
{
    constexpr int V = vec_elems<IO>;
    if (a.L <= WALK_MAX_L) {
        const int nvec = (a.C + V - 1) / V;
        const int64_t n = B * nvec, blocks = (n + 63) / 64;
        if (!grid_ok(blocks, 64)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((recur_walk<IO, BWD, (MODE > 0)>), dim3((unsigned)blocks), dim3(64), 0, st, a, n, nvec);
        return hipGetLastError();
    }
    constexpr int NC = V == 8 ? 2 : 4, R = (V == 8 ? 8 : 4) / (BWD ? 2 : 1), NW = 8, NTT = 64 * NW;
    const Plan p = plan(B, a.L, a.C);
    a.ngroups = (int)p.ngroups;
    a.nseg = (int)p.nseg;
    a.slen = p.slen;
    const int64_t blocks = B * p.ngroups * p.nseg;
    if (!grid_ok(blocks, NTT)) return hipErrorInvalidValue;
    if (p.nseg > 1) {
        hipLaunchKernelGGL((recur_tiles<IO, BWD, true, MODE, NC, R, NW>), dim3((unsigned)blocks), dim3(NTT), 0, st, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t n = B * a.C;
        hipLaunchKernelGGL(recur_chain, dim3((unsigned)((n + NT - 1) / NT)), dim3(NT), 0, st, a.seg, a.s0,
                           a.s1, n, a.C, a.nseg, BWD ? 1 : 0);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((recur_tiles<IO, BWD, false, MODE, NC, R, NW>), dim3((unsigned)blocks), dim3(NTT), 0, st, a);
    return hipGetLastError();
}

// 0: rows read element by element; 1: in vectors; 2: and every workgroup's channels all exist
template <class IO, bool BWD>
hipError_t pick(const Args& a, int64_t B, bool whole, hipStream_t st)
{
    if (!whole || a.C % vec_elems<IO>) return go<IO, BWD, 0>(a, B, st);
    return a.C % CG ? go<IO, BWD, 1>(a, B, st) : go<IO, BWD, 2>(a, B, st);
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
    a.L = L; a.C = C; a.zs = r.zs; a.us = r.us; a.os0 = r.hs;
    return s == Store::F32 ? pick<f32_io, false>(a, B, r.whole, st) : pick<bf16_io, false>(a, B, r.whole, st);
}

hipError_t launch_recur_bwd(Store s, const RecurBwd& r, int64_t B, int64_t L, int C, void* ws,
                            hipStream_t st)
{
    Args a{};
    a.z = r.z; a.u = r.u; a.h = r.h; a.dh = r.dh; a.o0 = r.dz; a.o1 = r.du; a.s0 = r.dhT;
    a.s1 = r.dh0; a.hinit = r.h0; a.seg = (float*)ws;
    a.L = L; a.C = C; a.zs = r.zs; a.us = r.us; a.hs = r.hs; a.dhs = r.dhs; a.os0 = r.dzs;
    a.os1 = r.dus;
    return s == Store::F32 ? pick<f32_io, true>(a, B, r.whole, st) : pick<bf16_io, true>(a, B, r.whole, st);
}

}  // namespace sc
