// Causal attention, backward pass (gfx950).
//
// With P_ij = exp(s_ij - lse_i) recomputed from q, k and the forward's lse, and
// delta_i = do_i . o_i:
//
//     dv_j = sum_i P_ij do_i,   dP_ij = do_i . v_j,   dS_ij = P_ij (dP_ij - delta_i)
//     dx_ij = dS_ij (1 - tanh^2),   dq_i = scale sum_j dx_ij k_j,   dk_j = scale sum_i dx_ij q_i
//
// Two kernels, neither with atomics, so the sums have a fixed order:
//  * attn_bwd_q: a workgroup owns 128 tokens of one head and walks key tiles; it makes delta on
//    the way in and leaves (lse, delta) of each row for the second kernel, and with documents
//    the key range of each 32-token strip.
//  * attn_bwd_kv: a workgroup owns 128 keys of a key head and walks the tokens that see them, all
//    heads of the group in turn, so the gradients of shared heads are plain sums.
// Both keep their own side's operands in registers (B operands), stage the other side through
// LDS with the next stage's loads in flight, and feed the score-shaped products to the next
// product from registers (sc_attn.h).  Seven products instead of the five of a single kernel
// that would add dq with atomics.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace attn;

constexpr int BN = 64;        // keys of a tile (attn_bwd_q), tokens of a stage (attn_bwd_kv)
constexpr int NQ = 2;         // 16-row blocks of a wave
constexpr int WM = 16 * NQ;   // tokens of a wave and of a strip
constexpr int BM = 4 * WM;    // tokens of a workgroup

// 16-key blocks of a wave (attn_bwd_kv): float32 operands of 128 leave room for one
template <class IO, int DP>
constexpr int key_blocks = IO::SIZE == 4 && DP == 128 ? 1 : 2;

#ifndef BQV
#define BQV(DP, SZ) (SZ == 4 ? 1 : DP == 64 ? 3 : 2)
#endif
#ifndef BKV
#define BKV(DP, SZ) (SZ == 4 ? 1 : DP == 64 ? 2 : 1)
#endif

// The score in base 2 of the raw product y plus `add`; dcap: the factor of dS that the cap adds.
template <class IO, bool CAP>
__device__ __forceinline__ float score2(float y, float scale2, float cap2, float add, float& dcap)
{
    if constexpr (CAP) {
        const float t = tanh_of<IO>(y * scale2);
        dcap = 1.0f - t * t;
        return __builtin_fmaf(cap2, t, add);
    } else {
        return __builtin_fmaf(y, scale2, add);
    }
}

template <class IO, int DP, bool CAP, bool BIAS>
__global__ __launch_bounds__(NT, BQV(DP, IO::SIZE)) void attn_bwd_q(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int P = pitch<IO, DP>, V = vec_elems<IO>, KK = DP / 32, ND = DP / 16;
    __shared__ __attribute__((aligned(16))) E Kt[BN * P];
    __shared__ __attribute__((aligned(16))) E Vt[BN * P];
    __shared__ int range[2][4];

    const int nbh = a.B * a.H;
    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)nbh);
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)nbh);
    const int b = bh / a.H, h = bh % a.H, hk = h / a.G;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;

    int pos[NQ], lo[NQ];
    bool empty[NQ];
    Frag<IO> q[NQ][KK], go[NQ][KK];
    float lse2[NQ], delta[NQ];
    const int rw = tile * BM + wave * WM;
    const float slope = BIAS ? a.slopes[h] * LOG2E : 0.f;
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        const int t = rw + 16 * m + c;
        const bool in = t < a.Lq;
        const int i = in ? t : 0;
        pos[m] = n - a.Lq + i;
        lo[m] = in ? first_key(a, b, pos[m], n) : BIG;
        empty[m] = lo[m] == BIG;
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
        if (g == 0 && in) a.rowstat[(int64_t)bh * a.Lq + i] = make_float2(lse2[m], delta[m]);
    }
    const RowRange rr = a.doc ? lanes_range(lo, pos) : token_range(a, n, rw, WM);
    int klo, khi;
    if (a.doc) {
        if (lane == 0) {
            range[0][wave] = rr.lo;
            range[1][wave] = rr.hi;
            // every head's rows have the same ranges: the first one's workgroup records them
            if (h == 0) a.strips[((int64_t)b * a.ntile + tile) * 4 + wave] = make_int4(rr.lo, rr.hi, rr.last, rr.pos);
        }
        __syncthreads();
        klo = min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3]));
        khi = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3]));
    } else {
        const RowRange all = token_range(a, n, tile * BM, BM);
        klo = all.lo;
        khi = all.hi;
    }
    klo = __builtin_amdgcn_readfirstlane(klo);
    khi = __builtin_amdgcn_readfirstlane(khi);
#pragma unroll
    for (int m = 0; m < NQ; ++m)
        if (empty[m]) {
            lo[m] = 0;
            pos[m] = BIG;
        }
    const int t0 = khi < 0 ? 0 : klo / BN, t1 = khi < 0 ? 0 : khi / BN + 1;

    const float scale2 = CAP ? a.scale / a.cap : a.scale * LOG2E, cap2 = a.cap * LOG2E;
    f32x4 acc[ND][NQ];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < NQ; ++m) acc[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    KeyTiles<IO, DP> tiles(a, b, hk, n, tid);
    if (t0 < t1) tiles.fetch(t0 * BN);
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * BN;
        __syncthreads();
        const uint64_t live = tiles.put(Kt, Vt, j0);
        __syncthreads();
        if (t + 1 < t1) tiles.fetch(j0 + BN);
        if (j0 > rr.hi || j0 + BN - 1 < rr.lo) continue;

        const bool edge = j0 < rr.last || j0 + BN - 1 > rr.pos || live != ~0ull;
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
                const float shift = BIAS ? slope * (float)(j0 + 4 * g - pos[m]) - lse2[m] : -lse2[m];
                f32x4 cf[2];   // the cap's factors
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float add = BIAS ? __builtin_fmaf(slope, (float)(32 * hf + 16 * kb + r), shift) : shift;
                        float dcap = 1.f;
                        s[kb][m][r] = exp2_hw(score2<IO, CAP>(s[kb][m][r], scale2, cap2, add, dcap));
                        cf[kb][r] = dcap;
                    }
                if (edge) {
                    keep_branch();
                    const int first = lo[m] - j0 - 4 * g;
                    const uint32_t span = (uint32_t)(pos[m] - lo[m]);
                    const uint64_t mine = live >> (4 * g);
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int jj = 32 * hf + 16 * kb + r;
                            if ((uint32_t)(jj - first) > span || !(mine >> jj & 1)) s[kb][m][r] = 0.f;
                        }
                }
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[kb][m][r] *= dp[kb][m][r] - delta[m];
                        if constexpr (CAP) s[kb][m][r] *= cf[kb][r];
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
        const int t = rw + 16 * m + c;
        if (t >= a.Lq) continue;
        E* p = (E*)a.dq + b * a.dqs[0] + (int64_t)t * a.dqs[1] + h * a.dqs[2];
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int d0 = 16 * d + 4 * g;
            if (d0 < a.D) put4<IO>(p + d0, empty[m] ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[d][m] * a.scale);
        }
    }
}

template <class IO, int DP, bool CAP, bool BIAS>
__global__ __launch_bounds__(NT, BKV(DP, IO::SIZE)) void attn_bwd_kv(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int P = pitch<IO, DP>, V = vec_elems<IO>, CH = DP / V, NCH = BN * CH / NT;
    constexpr int KK = DP / 32, ND = DP / 16, NK = key_blocks<IO, DP>, WK = 16 * NK, BK = 4 * WK;
    __shared__ __attribute__((aligned(16))) E Qt[BN * P];
    __shared__ __attribute__((aligned(16))) E Gt[BN * P];
    __shared__ __attribute__((aligned(16))) float Rt[BN], Dl[BN];
    __shared__ __attribute__((aligned(16))) int Lo[BN];

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
    const int off = n - a.Lq;   // position of token 0
    // stages of tokens at positions jb .. jb + BK - 1 + window - 1
    int s0 = 0, s1 = 0;
    {
        const int64_t plo = std::max<int64_t>(jb, off);
        const int64_t phi = std::min<int64_t>(n - 1, (int64_t)jb + BK - 1 + a.window - 1);
        if (plo <= phi) {
            s0 = (int)((plo - off) / BN);
            s1 = (int)((phi - off) / BN + 1);
        }
    }
    const int4* strips = a.strips + (int64_t)b * a.ntile * 4;
    // the next stage at or after s whose tokens see this workgroup's keys, 64 looked at together
    auto seek = [&](int s) {
        if (!a.doc) return s;
        while (s < s1) {
            bool hit = false;
            if (s + lane < s1) {
                const int4 x = strips[2 * (s + lane)], y = strips[2 * (s + lane) + 1];
                hit = min(x.x, y.x) <= jb + BK - 1 && max(x.y, y.y) >= jb;
            }
            const uint64_t m = __ballot(hit);
            if (m) return __builtin_amdgcn_readfirstlane(s + (int)__builtin_ctzll(m));
            s += 64;
        }
        return s1;
    };

    const int r0 = tid / CH, d0 = tid % CH * V;
    const bool din = d0 < a.D;
    const int32_t* doc = a.doc ? a.doc + (int64_t)b * a.Lk : nullptr;
    for (int h = hk * a.G; h < (hk + 1) * a.G; ++h) {
        const E* qp = (const E*)a.q + b * a.qs[0] + h * a.qs[2] + (din ? d0 : 0);
        const E* gp = (const E*)a.dout + b * a.dos[0] + h * a.dos[2] + (din ? d0 : 0);
        const float2* stat = a.rowstat + ((int64_t)b * a.H + h) * a.Lq;
        const float slope = BIAS ? a.slopes[h] * LOG2E : 0.f;
        uint4 rq[NCH], rg[NCH];
        float2 rs = make_float2(INFINITY, 0.f);
        int rdoc = 0;
        // nothing here waits for a load
        auto fetch = [&](int s) {
            const int tb = s * BN;
            if (tb + BN <= a.Lq) {
                const E *q = qp + (int64_t)(tb + r0) * a.qs[1], *g_ = gp + (int64_t)(tb + r0) * a.dos[1];
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    rq[i] = *(const uint4*)(q + (int64_t)(NT / CH * i) * a.qs[1]);
                    rg[i] = *(const uint4*)(g_ + (int64_t)(NT / CH * i) * a.dos[1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int64_t t = min(tb + r0 + NT / CH * i, a.Lq - 1);
                    rq[i] = *(const uint4*)(qp + t * a.qs[1]);
                    rg[i] = *(const uint4*)(gp + t * a.dos[1]);
                }
            }
            const int t = min(tb + lane, a.Lq - 1);   // each wave: lane's row of the stage
            rs = stat[t];
            if (doc) rdoc = doc[min(max(off + t, 0), n - 1)];
        };
        int s = seek(s0);
        if (s < s1) fetch(s);
        while (s < s1) {
            __syncthreads();
            {
                const int tb = s * BN, p = off + tb + lane;
                int first = max(max(0, p - a.window + 1), doc ? rdoc : 0);
                if (tb + lane >= a.Lq || p < 0 || first > p) first = BIG;
                // empty rows read as 0, whatever the memory holds
                const uint64_t alive = __ballot(first != BIG);
                if (alive == ~0ull && DP == a.D) {
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const int at = (r0 + NT / CH * i) * P + d0;
                        *(uint4*)(Qt + at) = rq[i];
                        *(uint4*)(Gt + at) = rg[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const int r = r0 + NT / CH * i, at = r * P + d0;
                        const bool on = din && alive >> r & 1;
                        *(uint4*)(Qt + at) = on ? rq[i] : make_uint4(0, 0, 0, 0);
                        *(uint4*)(Gt + at) = on ? rg[i] : make_uint4(0, 0, 0, 0);
                    }
                }
                if (tid < BN) {
                    // the row's part of the exponent: - lse (infinite for an empty row), and - slope of
                    // its distance to the stage's first token
                    Rt[tid] = first == BIG ? -INFINITY : BIAS ? -rs.x - slope * (float)tid : -rs.x;
                    Dl[tid] = first == BIG ? 0.f : rs.y;
                    Lo[tid] = first;
                }
            }
            __syncthreads();
            const int tb = s * BN, pb = off + tb;
            s = seek(s + 1);
            if (s < s1) fetch(s);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {   // 32 tokens at a time
                const int tw = tb + 32 * hf;
                RowRange st;
                if (doc) {
                    const int4 x = strips[tw / WM];
                    st = {x.x, x.y, x.z, x.w};
                } else {
                    st = token_range(a, n, tw, WM);
                }
                if (st.lo > jw + WK - 1 || st.hi < jw) continue;   // no row of the strip sees this wave's keys
                const bool edge = dead || st.last > jw || st.pos < jw + WK - 1;
                // rows x keys
                f32x4 w[2][NK], dp[2][NK];
#pragma unroll
                for (int rb = 0; rb < 2; ++rb) {
#pragma unroll
                    for (int m = 0; m < NK; ++m) w[rb][m] = dp[rb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const int at = (32 * hf + 16 * rb + c) * P + 32 * kk + 8 * g;
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
                    const int rr = 32 * hf + 16 * rb + 4 * g;
                    const f32x4 rt = *(const f32x4*)(Rt + rr), dl = *(const f32x4*)(Dl + rr);
#pragma unroll
                    for (int m = 0; m < NK; ++m) {
                        const float kterm = BIAS ? slope * (float)(key[m] - pb) : 0.f;
                        f32x4 cf;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            float dcap = 1.f;
                            const float add = BIAS ? rt[r] + kterm : rt[r];
                            w[rb][m][r] = exp2_hw(score2<IO, CAP>(w[rb][m][r], scale2, cap2, add, dcap));
                            cf[r] = dcap;
                        }
                        if (edge) {
                            keep_branch();
                            const int4 lo4 = *(const int4*)(Lo + rr);
                            const int lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (key[m] < lo[r] || key[m] > pb + rr + r) w[rb][m][r] = 0.f;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            dp[rb][m][r] = w[rb][m][r] * (dp[rb][m][r] - dl[r]);
                            if constexpr (CAP) dp[rb][m][r] *= cf[r];
                        }
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
                    const Frag<IO> fg = frag_tr<IO, P>(Gt, 32 * hf, 16 * d, g, c);
                    const Frag<IO> fq = frag_tr<IO, P>(Qt, 32 * hf, 16 * d, g, c);
#pragma unroll
                    for (int m = 0; m < NK; ++m) {
                        dv[d][m] = mma(fg, fp[m], dv[d][m]);
                        dk[d][m] = mma(fq, fs[m], dk[d][m]);
                    }
                }
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
            const int x = 16 * d + 4 * g;
            if (x >= a.D) continue;
            put4<IO>(kp + x, dk[d][m] * a.scale);
            put4<IO>(vp + x, dv[d][m]);
        }
    }
}

template <class IO, int DP, bool CAP, bool BIAS>
hipError_t go(const AttnArgs& a, hipStream_t st)
{
    constexpr int BK = 64 * key_blocks<IO, DP>;
    const int64_t qb = (int64_t)a.ntile * a.B * a.H, kb = (int64_t)((a.Lk + BK - 1) / BK) * a.nbh;
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

size_t stat_bytes(const AttnArgs& a) { return ((size_t)a.B * a.H * a.Lq * sizeof(float2) + 255) / 256 * 256; }

}  // namespace

size_t attn_bwd_bytes(const AttnArgs& a)
{
    return stat_bytes(a) + (a.doc ? (size_t)a.B * ((a.Lq + BM - 1) / BM) * 4 * sizeof(int4) : 0);
}

hipError_t launch_attn_bwd(Store s, const AttnArgs& a, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.ntile = (a.Lq + BM - 1) / BM;
    x.rowstat = (float2*)ws;
    x.strips = (int4*)((char*)ws + stat_bytes(a));
    if (s == Store::F32) return a.D <= 64 ? pick<f32_io, 64>(x, st) : pick<f32_io, 128>(x, st);
    return a.D <= 64 ? pick<bf16_io, 64>(x, st) : pick<bf16_io, 128>(x, st);
}

}  // namespace sc
