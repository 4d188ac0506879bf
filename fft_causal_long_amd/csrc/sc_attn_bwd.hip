// Causal attention, backward pass (gfx950).
//
// With P_ij = exp(s_ij - lse_i) recomputed from q, k and the forward's lse, and
// delta_i = do_i . o_i:
//
//     dv_j = sum_i P_ij do_i,   dP_ij = do_i . v_j,   dS_ij = P_ij (dP_ij - delta_i)
//     dx_ij = dS_ij (1 - tanh^2),   dq_i = scale sum_j dx_ij k_j,   dk_j = scale sum_i dx_ij q_i
//
// Two kernels, neither with atomics, so the sums have a fixed order:
//  * attn_bwd_q: a workgroup owns 128 packed rows (token r / G, head r % G of the group) and
//    walks key tiles; it makes delta on the way in and leaves (lse, delta) of each row and the
//    key range of each 32-row strip for the second kernel.
//  * attn_bwd_kv: a workgroup owns 128 keys of a key head and walks the strips of packed rows,
//    all heads of the group in turn, so the gradients of shared heads are plain sums.
// Both keep their own side's operands in registers (B operands), stage the other side through
// LDS, and feed the score-shaped products to the next product from registers (sc_attn.h).
// Seven products instead of the five of a single kernel that would add dq with atomics.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace attn;

constexpr int BN = 64;        // keys of a tile (attn_bwd_q)
constexpr int NQ = 2;         // 16-row blocks of a wave
constexpr int WM = 16 * NQ;   // rows of a wave and of a strip
constexpr int BM = 4 * WM;    // rows of a workgroup
constexpr int NK = 2;         // 16-key blocks of a wave (attn_bwd_kv)
constexpr int WK = 16 * NK;
constexpr int BK = 4 * WK;    // keys of a workgroup

// Score and the factor of dS that the cap adds; y = raw product q.k, dist = j - p.
template <class IO, bool CAP, bool BIAS>
__device__ __forceinline__ float score2(float y, float scale2, float cap2, float slope, float dist,
                                        float& dcap)
{
    float x;
    if constexpr (CAP) {
        const float t = tanh_of<IO>(y * scale2);
        dcap = 1.0f - t * t;
        x = cap2 * t;
        if constexpr (BIAS) x = __builtin_fmaf(slope, dist, x);
    } else if constexpr (BIAS) {
        x = __builtin_fmaf(y, scale2, slope * dist);
    } else {
        x = y * scale2;
    }
    return x;
}

template <class IO, int DP, bool CAP, bool BIAS>
__global__ __launch_bounds__(NT) void attn_bwd_q(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int P = pitch<IO, DP>, V = vec_elems<IO>, CH = DP / V, NCH = BN * CH / NT;
    constexpr int KK = DP / 32, ND = DP / 16;
    __shared__ __attribute__((aligned(16))) E Kt[BN * P];
    __shared__ __attribute__((aligned(16))) E Vt[BN * P];
    __shared__ int range[2][4];

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)a.nbh);
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;

    int row[NQ], pos[NQ], lo[NQ];
    bool empty[NQ];
    Frag<IO> q[NQ][KK], go[NQ][KK];
    float slope[NQ], lse2[NQ], delta[NQ];
    int wlo = BIG, whi = -1, mlo = 0, mpos = BIG;
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        row[m] = tile * BM + wave * WM + 16 * m + c;
        const bool in = row[m] < a.nrow;
        const int i = in ? row[m] / a.G : 0, h = hk * a.G + (in ? row[m] % a.G : 0);
        pos[m] = n - a.Lq + i;
        lo[m] = in ? first_key(a, b, pos[m], n) : BIG;
        empty[m] = lo[m] == BIG;
        if (!empty[m]) {
            wlo = min(wlo, lo[m]);
            whi = max(whi, pos[m]);
            mlo = max(mlo, lo[m]);
            mpos = min(mpos, pos[m]);
        } else {
            lo[m] = 0;
            pos[m] = BIG;
        }
        slope[m] = BIAS ? a.slopes[h] * LOG2E : 0.f;
        // an empty row's weights are 2^-inf = 0
        lse2[m] = empty[m] ? INFINITY : a.lse[((int64_t)b * a.H + h) * a.Lq + i] * LOG2E;
        const E* qp = (const E*)a.q + b * a.qs[0] + (int64_t)i * a.qs[1] + h * a.qs[2];
        const E* gp = (const E*)a.dout + b * a.dos[0] + (int64_t)i * a.dos[1] + h * a.dos[2];
        const E* op = (const E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
        float dl = 0.f;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const int d = 32 * k + 8 * g;
            const bool on = !empty[m] && d < a.D;
            q[m][k] = on ? frag_at<IO>(qp + d) : frag_zero<IO>();
            go[m][k] = on ? frag_at<IO>(gp + d) : frag_zero<IO>();
            const Frag<IO> of = on ? frag_at<IO>(op + d) : frag_zero<IO>();
            if constexpr (IO::SIZE == 2) {
                const Lanes<IO> x = widen<IO>(go[m][k].v), y = widen<IO>(of.v);
#pragma unroll
                for (int e = 0; e < V; ++e) dl = __builtin_fmaf(x.x[e], y.x[e], dl);
            } else {
                dl = __builtin_fmaf(go[m][k].a.x, of.a.x, dl);
                dl = __builtin_fmaf(go[m][k].a.y, of.a.y, dl);
                dl = __builtin_fmaf(go[m][k].a.z, of.a.z, dl);
                dl = __builtin_fmaf(go[m][k].a.w, of.a.w, dl);
                dl = __builtin_fmaf(go[m][k].b.x, of.b.x, dl);
                dl = __builtin_fmaf(go[m][k].b.y, of.b.y, dl);
                dl = __builtin_fmaf(go[m][k].b.z, of.b.z, dl);
                dl = __builtin_fmaf(go[m][k].b.w, of.b.w, dl);
            }
        }
        delta[m] = gsum(dl);
        if (g == 0 && in) a.rowstat[(int64_t)bh * a.nrow + row[m]] = make_float2(lse2[m], delta[m]);
    }
    wlo = wave_min(wlo);
    whi = wave_max(whi);
    mlo = wave_max(mlo);
    mpos = wave_min(mpos);
    if (lane == 0) {
        range[0][wave] = wlo;
        range[1][wave] = whi;
        // every key head's rows have the same ranges: the first one's workgroup records them
        if (hk == 0)
            a.strips[(int64_t)b * a.ntile * 4 + tile * 4 + wave] = make_int4(wlo, whi, mlo, mpos);
    }
    __syncthreads();
    const int klo = min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3]));
    const int khi = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3]));
    const int t0 = khi < 0 ? 0 : klo / BN, t1 = khi < 0 ? 0 : khi / BN + 1;

    const float scale2 = CAP ? a.scale / a.cap : a.scale * LOG2E, cap2 = a.cap * LOG2E;
    f32x4 acc[ND][NQ];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < NQ; ++m) acc[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    const E* kp = (const E*)a.k + b * a.ks[0] + hk * a.ks[2];
    const E* vp = (const E*)a.v + b * a.vs[0] + hk * a.vs[2];
    uint4 rk[NCH], rv[NCH];
    int rdoc = 0;
    auto fetch = [&](int j0) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int id_ = tid + NT * i, j = j0 + id_ / CH, d = (id_ % CH) * V;
            const bool on = d < a.D && key_live(a, b, j, n);
            rk[i] = on ? *(const uint4*)(kp + (int64_t)j * a.ks[1] + d) : make_uint4(0, 0, 0, 0);
            rv[i] = on ? *(const uint4*)(vp + (int64_t)j * a.vs[1] + d) : make_uint4(0, 0, 0, 0);
        }
        if (a.doc) rdoc = j0 + lane < n ? a.doc[(int64_t)b * a.Lk + j0 + lane] : BIG;
    };
    if (t0 < t1) fetch(t0 * BN);
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * BN;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int id_ = tid + NT * i, at = (id_ / CH) * P + (id_ % CH) * V;
            *(uint4*)(Kt + at) = rk[i];
            *(uint4*)(Vt + at) = rv[i];
        }
        const uint64_t live = a.doc ? __ballot(rdoc <= j0 + lane) : ~0ull;
        __syncthreads();
        if (t + 1 < t1) fetch(j0 + BN);
        if (j0 > whi || j0 + BN - 1 < wlo) continue;

        const bool edge = j0 < mlo || j0 + BN - 1 > mpos || live != ~0ull;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {   // 32 keys at a time
            f32x4 s[2][NQ], dp[2][NQ];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                for (int m = 0; m < NQ; ++m) s[kb][m] = dp[kb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    const int at = (32 * hf + 16 * kb + c) * P + 32 * k + 8 * g;
                    const Frag<IO> fk = frag_at<IO>(Kt + at), fv = frag_at<IO>(Vt + at);
#pragma unroll
                    for (int m = 0; m < NQ; ++m) {
                        s[kb][m] = mma(fk, q[m][k], s[kb][m]);
                        dp[kb][m] = mma(fv, go[m][k], dp[kb][m]);
                    }
                }
            }
            Frag<IO> w[NQ];
#pragma unroll
            for (int m = 0; m < NQ; ++m) {
                const float far = (float)(j0 + 4 * g - pos[m]);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int jj = 32 * hf + 16 * kb + 4 * g + r, j = j0 + jj;
                        float dcap = 1.f;
                        const float x = score2<IO, CAP, BIAS>(s[kb][m][r], scale2, cap2, slope[m],
                                                          far + (float)(32 * hf + 16 * kb + r), dcap);
                        float p = exp2_hw(x - lse2[m]);
                        if (edge && (j < lo[m] || j > pos[m] || !(live >> jj & 1))) p = 0.f;
                        float ds = p * (dp[kb][m][r] - delta[m]);
                        if constexpr (CAP) ds *= dcap;
                        s[kb][m][r] = ds;
                    }
                w[m] = frag_of<IO>(s[0][m], s[1][m]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<IO> f = frag_tr<IO, P>(Kt, 32 * hf, 16 * d, g, c);
#pragma unroll
                for (int m = 0; m < NQ; ++m) acc[d][m] = mma(f, w[m], acc[d][m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        if (row[m] >= a.nrow) continue;
        const int i = row[m] / a.G, h = hk * a.G + row[m] % a.G;
        E* p = (E*)a.dq + b * a.dqs[0] + (int64_t)i * a.dqs[1] + h * a.dqs[2];
        const float f = empty[m] ? 0.f : a.scale;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int d0 = 16 * d + 4 * g;
            if (d0 >= a.D) continue;
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = empty[m] ? 0.f : f * acc[d][m][r];
            if constexpr (IO::SIZE == 2)
                *(uint2*)(p + d0) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            else
                *(float4*)(p + d0) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

template <class IO, int DP, bool CAP, bool BIAS>
__global__ __launch_bounds__(NT) void attn_bwd_kv(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int P = pitch<IO, DP>, V = vec_elems<IO>, CH = DP / V;
    constexpr int NCH = (WM * CH + NT - 1) / NT;
    constexpr int KK = DP / 32, ND = DP / 16;
    static_assert(WM * CH % NT == 0, "whole rounds of loads");
    __shared__ __attribute__((aligned(16))) E Qt[WM * P];
    __shared__ __attribute__((aligned(16))) E Gt[WM * P];
    __shared__ __attribute__((aligned(16))) float Ls[WM], Dl[WM], Sl[WM];
    __shared__ __attribute__((aligned(16))) int Lo[WM], Ps[WM];

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    const int kt = (int)(id / (uint32_t)a.nbh);   // the first keys are seen by most rows: first
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
    const int jb = kt * BK, jw = jb + wave * WK;   // first key of the workgroup, of the wave

    Frag<IO> k[NK][KK], v[NK][KK];
    int key[NK];
    bool dead = false;
#pragma unroll
    for (int m = 0; m < NK; ++m) {
        const int j = jw + 16 * m + c;
        const bool live = key_live(a, b, j, n);
        key[m] = live ? j : -1;   // a dead key lies before every row's first
        dead |= !live;
        const E* kp = (const E*)a.k + b * a.ks[0] + (int64_t)j * a.ks[1] + hk * a.ks[2];
        const E* vp = (const E*)a.v + b * a.vs[0] + (int64_t)j * a.vs[1] + hk * a.vs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int d = 32 * kk + 8 * g;
            const bool on = live && d < a.D;
            k[m][kk] = on ? frag_at<IO>(kp + d) : frag_zero<IO>();
            v[m][kk] = on ? frag_at<IO>(vp + d) : frag_zero<IO>();
        }
    }
    dead = __any(dead);

    f32x4 dk[ND][NK], dv[ND][NK];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < NK; ++m) dk[d][m] = dv[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    const float scale2 = CAP ? a.scale / a.cap : a.scale * LOG2E, cap2 = a.cap * LOG2E;
    const int off = n - a.Lq;   // position of row 0
    // strips of packed rows at positions jb .. jb + BK - 1 + window - 1
    int s0 = 0, s1 = 0;
    {
        const int64_t plo = std::max<int64_t>(jb, off);
        const int64_t phi = std::min<int64_t>(n - 1, (int64_t)jb + BK - 1 + a.window - 1);
        if (plo <= phi) {
            s0 = (int)((plo - off) * a.G / WM);
            s1 = (int)(((phi - off + 1) * a.G - 1) / WM + 1);
        }
    }
    const int4* strips = a.strips + (int64_t)b * a.ntile * 4;
    // the next strip at or after s whose keys meet this workgroup's, 64 looked at together
    auto seek = [&](int s) {
        while (s < s1) {
            bool hit = false;
            if (s + lane < s1) {
                const int4 r = strips[s + lane];
                hit = r.x <= jb + BK - 1 && r.y >= jb;
            }
            const uint64_t m = __ballot(hit);
            if (m) return s + __builtin_ctzll(m);
            s += 64;
        }
        return s1;
    };

    uint4 rq[NCH], rg[NCH];
    float2 rs = make_float2(0.f, 0.f);
    int rlo = BIG, rpos = 0;
    float rsl = 0.f;
    auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int id_ = tid + NT * i, r = s * WM + id_ / CH, d = (id_ % CH) * V;
            const bool in = r < a.nrow;
            const int t = in ? r / a.G : 0, h = hk * a.G + (in ? r % a.G : 0);
            const bool on = in && d < a.D && first_key(a, b, off + t, n) != BIG;
            rq[i] = on ? *(const uint4*)((const E*)a.q + b * a.qs[0] + (int64_t)t * a.qs[1] + h * a.qs[2] + d)
                       : make_uint4(0, 0, 0, 0);
            rg[i] = on ? *(const uint4*)((const E*)a.dout + b * a.dos[0] + (int64_t)t * a.dos[1] + h * a.dos[2] + d)
                       : make_uint4(0, 0, 0, 0);
        }
        if (tid < WM) {
            const int r = s * WM + tid;
            const bool in = r < a.nrow;
            const int t = in ? r / a.G : 0;
            rpos = off + t;
            rlo = in ? first_key(a, b, rpos, n) : BIG;
            rs = in ? a.rowstat[(int64_t)bh * a.nrow + r] : make_float2(INFINITY, 0.f);
            rsl = BIAS && in ? a.slopes[hk * a.G + r % a.G] * LOG2E : 0.f;
        }
    };
    int s = seek(s0);
    if (s < s1) fetch(s);
    while (s < s1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int id_ = tid + NT * i, at = (id_ / CH) * P + (id_ % CH) * V;
            *(uint4*)(Qt + at) = rq[i];
            *(uint4*)(Gt + at) = rg[i];
        }
        if (tid < WM) {
            Ls[tid] = rs.x;
            Dl[tid] = rs.y;
            Sl[tid] = rsl;
            Lo[tid] = rlo;
            Ps[tid] = rpos;
        }
        __syncthreads();
        const int4 st = strips[s];   // lowest key, highest key, highest first key, lowest position
        s = seek(s + 1);
        if (s < s1) fetch(s);
        if (st.x > jw + WK - 1 || st.y < jw) continue;   // no row of the strip sees this wave's keys
        const bool edge = dead || st.z > jw || st.w < jw + WK - 1;

        // rows x keys
        f32x4 w[2][NK], dp[2][NK];
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
#pragma unroll
            for (int m = 0; m < NK; ++m) w[rb][m] = dp[rb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int at = (16 * rb + c) * P + 32 * kk + 8 * g;
                const Frag<IO> fq = frag_at<IO>(Qt + at), fg = frag_at<IO>(Gt + at);
#pragma unroll
                for (int m = 0; m < NK; ++m) {
                    w[rb][m] = mma(fq, k[m][kk], w[rb][m]);
                    dp[rb][m] = mma(fg, v[m][kk], dp[rb][m]);
                }
            }
        }
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            const f32x4 ls = *(const f32x4*)(Ls + 16 * rb + 4 * g), dl = *(const f32x4*)(Dl + 16 * rb + 4 * g);
            const int4 lo4 = *(const int4*)(Lo + 16 * rb + 4 * g), ps4 = *(const int4*)(Ps + 16 * rb + 4 * g);
            const int lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, ps[4] = {ps4.x, ps4.y, ps4.z, ps4.w};
            f32x4 sl = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (BIAS) sl = *(const f32x4*)(Sl + 16 * rb + 4 * g);
#pragma unroll
            for (int m = 0; m < NK; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float dcap = 1.f;
                    const float x = score2<IO, CAP, BIAS>(w[rb][m][r], scale2, cap2, sl[r],
                                                      (float)(key[m] - ps[r]), dcap);
                    float p = exp2_hw(x - ls[r]);
                    if (edge && (key[m] < lo[r] || key[m] > ps[r])) p = 0.f;
                    float ds = p * (dp[rb][m][r] - dl[r]);
                    if constexpr (CAP) ds *= dcap;
                    w[rb][m][r] = p;
                    dp[rb][m][r] = ds;
                }
        }
        Frag<IO> fp[NK], fs[NK];
#pragma unroll
        for (int m = 0; m < NK; ++m) {
            fp[m] = frag_of<IO>(w[0][m], w[1][m]);
            fs[m] = frag_of<IO>(dp[0][m], dp[1][m]);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const Frag<IO> fg = frag_tr<IO, P>(Gt, 0, 16 * d, g, c);
            const Frag<IO> fq = frag_tr<IO, P>(Qt, 0, 16 * d, g, c);
#pragma unroll
            for (int m = 0; m < NK; ++m) {
                dv[d][m] = mma(fg, fp[m], dv[d][m]);
                dk[d][m] = mma(fq, fs[m], dk[d][m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < NK; ++m) {
        const int j = jw + 16 * m + c;
        if (j >= a.Lk) continue;
        E* kp = (E*)a.dk + b * a.dks[0] + (int64_t)j * a.dks[1] + hk * a.dks[2];
        E* vp = (E*)a.dv + b * a.dvs[0] + (int64_t)j * a.dvs[1] + hk * a.dvs[2];
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int d0 = 16 * d + 4 * g;
            if (d0 >= a.D) continue;
            const f32x4 x = dk[d][m] * a.scale, y = dv[d][m];
            if constexpr (IO::SIZE == 2) {
                *(uint2*)(kp + d0) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                *(uint2*)(vp + d0) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            } else {
                *(float4*)(kp + d0) = make_float4(x[0], x[1], x[2], x[3]);
                *(float4*)(vp + d0) = make_float4(y[0], y[1], y[2], y[3]);
            }
        }
    }
}

template <class IO, int DP, bool CAP, bool BIAS>
hipError_t go(const AttnArgs& a, hipStream_t st)
{
    const int64_t qb = (int64_t)a.ntile * a.nbh, kb = (int64_t)((a.Lk + BK - 1) / BK) * a.nbh;
    if (!grid_ok(qb, NT) || !grid_ok(kb, NT)) return hipErrorInvalidValue;
    if (qb > 0) {
        hipLaunchKernelGGL((attn_bwd_q<IO, DP, CAP, BIAS>), dim3((unsigned)qb), dim3(NT), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (kb == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_bwd_kv<IO, DP, CAP, BIAS>), dim3((unsigned)kb), dim3(NT), 0, st, a);
    return hipGetLastError();
}

template <class IO, int DP>
hipError_t pick(const AttnArgs& a, hipStream_t st)
{
    if (a.cap > 0.f)
        return a.slopes ? go<IO, DP, true, true>(a, st) : go<IO, DP, true, false>(a, st);
    return a.slopes ? go<IO, DP, false, true>(a, st) : go<IO, DP, false, false>(a, st);
}

size_t stat_bytes(const AttnArgs& a) { return ((size_t)a.nbh * a.nrow * sizeof(float2) + 255) / 256 * 256; }

}  // namespace

size_t attn_bwd_bytes(const AttnArgs& a)
{
    return stat_bytes(a) + (size_t)a.B * ((a.nrow + BM - 1) / BM) * 4 * sizeof(int4);
}

hipError_t launch_attn_bwd(Store s, const AttnArgs& a, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.ntile = (a.nrow + BM - 1) / BM;
    x.rowstat = (float2*)ws;
    x.strips = (int4*)((char*)ws + stat_bytes(a));
    if (s == Store::F32) return a.D <= 64 ? pick<f32_io, 64>(x, st) : pick<f32_io, 128>(x, st);
    return a.D <= 64 ? pick<bf16_io, 64>(x, st) : pick<bf16_io, 128>(x, st);
}

}  // namespace sc
