// Causal attention, backward pass (gfx950).
//
// With P_ij = exp(s_ij - lse_i) recomputed from q, k and the forward's lse, and
// delta_i = do_i . o_i:
//
//     dv_j = sum_i P_ij do_i,   dP_ij = do_i . v_j,   dS_ij = P_ij (dP_ij - delta_i)
//     dx_ij = dS_ij (1 - tanh^2),   dq_i = scale sum_j dx_ij k_j,   dk_j = scale sum_i dx_ij q_i
//
// Two kernels, neither with atomics, so the sums have a fixed order:
//  * attn_bwd_q: a workgroup owns 64 or 128 tokens of one head and walks key tiles; it makes delta
//    on the way in and leaves (lse, delta) of each row for the second kernel, and with documents
//    the key range of each 32-token strip.
//  * attn_bwd_kv: a workgroup owns 64 or 128 keys of a key head and walks the tokens that see them,
//    all heads of the group in turn (or its part of them), so the gradients of shared heads are
//    plain sums.
// Both keep their own side's operands in registers (B operands), bring the other side into an LDS
// ring by asynchronous loads, and feed the score-shaped products to the next product from
// registers (sc_attn.h), P and dS rounded to the storage type on the way, as the forward pass rounds its
// weights.  Seven products instead of the five of a single kernel that would add dq
// with atomics.
//
// Measured (MI355X; a large copy moves 5.4 TB/s): bfloat16, B 8, L 4096, 16 heads of 64, window
// 256, bias, documents of about 700: 306 us, 130 of them attn_bwd_q and 179 attn_bwd_kv, where a
// copy of the tensors takes 102.  The loads and stores alone are 103 and 86 us.  Vector instructions
// keep a SIMD busy 46 and 34% of the time and the matrix products 14%: what is left are waits, for
// the first tiles of short walks (6 stages a workgroup) and for the waves that still have work.
// 16 tokens a wave and 8 waves: 146 us against 135, 32 x 8 187; keys: 16 x 8 180, as 32 x 4, at
// two waves a SIMD 243, 32 x 8 235; three waves a SIMD spill (552 us in all).
// float32, B 2, L 1001, 12 heads of 64, cap 30, bias, documents: 136 us (60 and 82).  384 workgroups
// of 64 rows are one and a half a CU: 0.7 waves a SIMD on average, each alone with its latencies
// (matrix products 19% of the time, vector instructions 10%).

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace attn;

constexpr int STRIP = 32;     // tokens of a strip (half a stage, or a stage)

// A workgroup's shape: N 16-row blocks a wave (tokens in attn_bwd_q, keys in attn_bwd_kv), NW waves.
template <int N_, int NW_>
struct Shape {
    static constexpr int N = N_, NW = NW_, W = 16 * N, ROWS = NW * W;   // rows of a wave, of a workgroup
};

// Waves a SIMD the kernels are compiled for: as many as their registers allow without spills but for
// three capped forms with a bias (of attn_bwd_kv, float32 heads over 64 in workgroups of 64 keys, and
// bfloat16 heads up to 64 with the tanh series in workgroups of 128: two registers; of attn_bwd_q, the
// latter's: five).
template <class IO, int DP>
constexpr int q_occupancy = IO::SIZE == 2 && DP == 64 ? 3 : 2;
template <class IO, int DP>
constexpr int kv_occupancy = IO::SIZE == 2 && DP == 128 ? 1 : 2;

// The score in base 2 of the raw product y plus `add`; dcap: the factor of dS that the cap adds.
template <class IO, Cap CAP>
__device__ __forceinline__ float score2(float y, float scale2, float cap2, float add, float& dcap)
{
    if constexpr (CAP != UNCAPPED) {
        const float t = tanh_of<IO, CAP>(y * scale2);
        dcap = 1.0f - t * t;
        return __builtin_fmaf(cap2, t, add);
    } else {
        return __builtin_fmaf(y, scale2, add);
    }
}

template <class IO, int DP, Cap CAP, bool BIAS, class S>
__global__ __launch_bounds__((64 * S::NW), (q_occupancy<IO, DP>)) void attn_bwd_q(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int NQ = S::N, NW = S::NW, WM = S::W, BM = S::ROWS;
    using R = Ring<IO, DP, 64 * NW>;
    constexpr int V = vec_elems<IO>, KK = DP / 32, ND = DP / 16, BN = stage_rows<IO, DP>;
    __shared__ __attribute__((aligned(1024))) typename R::Shared sh;
    __shared__ int4 range[NW];

    const int nbh = a.B * a.H;
    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)nbh);
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)nbh);
    const int b = bh / a.H, h = bh % a.H, hk = h / a.G;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform, so that branches on it are

    int pos[NQ], lo[NQ];
    bool empty[NQ];
    Frag<IO> q[NQ][KK], go[NQ][KK], of[NQ][KK];
    float lse2[NQ], delta[NQ];
    const int rw = tile * BM + wave * WM;
    const float slope = BIAS ? a.slopes[h] * LOG2E : 0.f;
    // everything the rows need is asked for at once: their place in the documents, and their data
    // whether or not they turn out to be empty
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        const int i = min(rw + 16 * m + c, a.Lq - 1);
        const E* qp = (const E*)a.q + b * a.qs[0] + (int64_t)i * a.qs[1] + h * a.qs[2];
        const E* gp = (const E*)a.dout + b * a.dos[0] + (int64_t)i * a.dos[1] + h * a.dos[2];
        const E* op = (const E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
        lse2[m] = a.lse[((int64_t)b * a.H + h) * a.Lq + i];
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            q[m][k] = frag_load<IO>(qp, 32 * k + 8 * g, a.D);
            go[m][k] = frag_load<IO>(gp, 32 * k + 8 * g, a.D);
            of[m][k] = frag_load<IO>(op, 32 * k + 8 * g, a.D);
        }
    }
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        const int t = rw + 16 * m + c;
        pos[m] = n - a.Lq + min(t, a.Lq - 1);
        lo[m] = t < a.Lq ? first_key(a, b, pos[m], n) : BIG;
        empty[m] = lo[m] == BIG;
    }
    const RowRange rr = a.doc ? lanes_range(lo, pos) : token_range(a, n, rw, WM);
    int klo, khi;
    if (a.doc) {
        join_ranges<NW>(range, rr, wave, lane, klo, khi);
        // every head's rows have the same ranges: the first one's workgroup records them
        if (h == 0 && tid < BM / STRIP) {
            constexpr int per = STRIP / WM;   // waves of a strip
            int4 x = range[tid * per];
            if (per > 1) {
                const int4 y = range[tid * per + per - 1];
                x = make_int4(min(x.x, y.x), max(x.y, y.y), max(x.z, y.z), min(x.w, y.w));
            }
            a.strips[(int64_t)b * a.nstrip + tile * (BM / STRIP) + tid] = x;
        }
    } else {
        const RowRange all = token_range(a, n, tile * BM, BM);
        klo = all.lo;
        khi = all.hi;
    }
    klo = __builtin_amdgcn_readfirstlane(klo);
    khi = __builtin_amdgcn_readfirstlane(khi);
    const int t0 = khi < 0 ? 0 : klo / BN, t1 = khi < 0 ? 0 : khi / BN + 1;

    const float scale2 = score_scale<CAP>(a), cap2 = a.cap * LOG2E;
    f32x4 acc[ND][NQ];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < NQ; ++m) acc[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    R ring(sh, n, a.D, a.ks[1], a.vs[1]);
    ring.from((const E*)a.k + b * a.ks[0] + hk * a.ks[2], (const E*)a.v + b * a.vs[0] + hk * a.vs[2]);
    if (a.doc) ring.wp[0] = (const uint32_t*)a.doc + (int64_t)b * a.Lk;
    ring.start(t0, t1);
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        float dl = 0.f;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const bool on = !empty[m] && 32 * k + 8 * g < a.D;
            frag_keep<IO>(q[m][k], on);
            frag_keep<IO>(go[m][k], on);
            frag_keep<IO>(of[m][k], on);
            if constexpr (IO::SIZE == 2) {
                const Lanes<IO> x = widen<IO>(go[m][k].v), y = widen<IO>(of[m][k].v);
#pragma unroll
                for (int e = 0; e < V; ++e) dl = __builtin_fmaf(x.x[e], y.x[e], dl);
            } else {
                const Frag<IO>&x = go[m][k], &y = of[m][k];
                dl = __builtin_fmaf(x.a.x, y.a.x, dl);
                dl = __builtin_fmaf(x.a.y, y.a.y, dl);
                dl = __builtin_fmaf(x.a.z, y.a.z, dl);
                dl = __builtin_fmaf(x.a.w, y.a.w, dl);
                dl = __builtin_fmaf(x.b.x, y.b.x, dl);
                dl = __builtin_fmaf(x.b.y, y.b.y, dl);
                dl = __builtin_fmaf(x.b.z, y.b.z, dl);
                dl = __builtin_fmaf(x.b.w, y.b.w, dl);
            }
        }
        delta[m] = gsum(dl);
        // an empty row's weights are 2^-inf = 0, with nothing masked
        lse2[m] = empty[m] ? INFINITY : lse2[m] * LOG2E;
        if (empty[m]) {
            lo[m] = 0;
            pos[m] = BIG;
        }
        const int t = rw + 16 * m + c;
        if (g == 0 && t < a.Lq) {
            const int64_t at = (int64_t)bh * a.Lq + t;
            a.rowstat[at] = lse2[m];
            a.rowstat[(int64_t)nbh * a.Lq + at] = delta[m];
        }
    }
    int place = 0;
    for (int t = t0; t < t1; ++t, place = R::after(place)) {
        const int j0 = t * BN;
        ring.step(t, t1, place);
        const E *Kt = sh.x[place], *Vt = sh.y[place];
        uint64_t live = ~0ull;   // keys that are not padding, bit j - j0
        if (a.doc || j0 + BN > n) {
            const int j = j0 + lane % BN;
            live = __ballot(j < n && (!a.doc || (int)sh.w[0][place][lane % BN] <= j));
            if (BN < 64) live |= ~0ull << (BN & 63);
            if (live != ~0ull) ring.blank(place, live);
        }
        if (j0 > rr.hi || j0 + BN - 1 < rr.lo) continue;

        const bool edge = j0 < rr.last || j0 + BN - 1 > rr.pos;
#pragma unroll
        for (int hf = 0; hf < BN / 32; ++hf) {   // 32 keys at a time
            f32x4 s[2][NQ], dp[2][NQ];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
                for (int m = 0; m < NQ; ++m) s[kb][m] = dp[kb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    const Frag<IO> fk = frag_row<IO, DP>(Kt, 32 * hf + 16 * kb, k, g, c);
                    const Frag<IO> fv = frag_row<IO, DP>(Vt, 32 * hf + 16 * kb, k, g, c);
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
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if ((uint32_t)(32 * hf + 16 * kb + r - first) > span) s[kb][m][r] = 0.f;
                }
                if (live != ~0ull) {
                    keep_branch();
                    const uint64_t mine = live >> (4 * g);
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (!(mine >> (32 * hf + 16 * kb + r) & 1)) s[kb][m][r] = 0.f;
                }
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[kb][m][r] *= dp[kb][m][r] - delta[m];
                        if constexpr (CAP != UNCAPPED) s[kb][m][r] *= cf[kb][r];
                    }
                w[m] = frag_of<IO>(s[0][m], s[1][m]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<IO> f = frag_tr<IO, DP>(Kt, 32 * hf, 16 * d, g, c);
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

template <class IO, int DP, Cap CAP, bool BIAS, class S>
__global__ __launch_bounds__((64 * S::NW), (kv_occupancy<IO, DP>)) void attn_bwd_kv(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int NW = S::NW, NK = S::N, WK = S::W, BK = S::ROWS;
    using R = Ring<IO, DP, 64 * NW>;
    constexpr int KK = DP / 32, ND = DP / 16, BN = stage_rows<IO, DP>, SP = BN / STRIP;   // tokens and strips of a stage
    __shared__ __attribute__((aligned(1024))) typename R::Shared sh;
    __shared__ __attribute__((aligned(16))) int first[NW][BN], span[NW][BN];   // each wave its own copy

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    id /= (uint32_t)a.nbh;
    const int part = (int)(id % (uint32_t)a.nparts), kt = (int)(id / (uint32_t)a.nparts);   // the first keys are
                                                                                      // seen by most rows: first
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform, so that branches on it are
    const int jb = kt * BK, jw = jb + wave * WK;   // first key of the workgroup, of the wave

    // this wave's keys, asked for whether or not they turn out to be padding; cleared below
    Frag<IO> k[NK][KK], v[NK][KK];
#pragma unroll
    for (int m = 0; m < NK; ++m) {
        const int64_t j = min(jw + 16 * m + c, a.Lk - 1);
        const E* kp = (const E*)a.k + b * a.ks[0] + j * a.ks[1] + hk * a.ks[2];
        const E* vp = (const E*)a.v + b * a.vs[0] + j * a.vs[1] + hk * a.vs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            k[m][kk] = frag_load<IO>(kp, 32 * kk + 8 * g, a.D);
            v[m][kk] = frag_load<IO>(vp, 32 * kk + 8 * g, a.D);
        }
    }

    f32x4 dk[ND][NK], dv[ND][NK];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < NK; ++m) dk[d][m] = dv[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    const float scale2 = score_scale<CAP>(a), cap2 = a.cap * LOG2E;
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
    const int4* strips = a.strips + (int64_t)b * a.nstrip;
    // With documents: which of 64 stages from sbase on see this workgroup's keys, and which of their
    // strips this wave's (hit) and every key of them (full), read together so that the walk itself
    // waits for no load of its own.
    int sbase = 0, sfilled = -1;
    uint64_t stage_hit = 0, hit[SP], full[SP];
    auto look = [&](int s) {
        sbase = s;
        sfilled = 1;
        bool any = false;
#pragma unroll
        for (int x = 0; x < SP; ++x) {
            bool h = false, f = false;
            if (s + lane < s1) {
                const int4 r = strips[SP * (s + lane) + x];
                any |= r.x <= jb + BK - 1 && r.y >= jb;
                h = r.x <= jw + WK - 1 && r.y >= jw;
                f = r.z <= jw && r.w >= jw + WK - 1;
            }
            hit[x] = __ballot(h);
            full[x] = __ballot(f);
        }
        stage_hit = __ballot(any);
    };
    // the next stage at or after s that sees this workgroup's keys
    auto seek = [&](int s) {
        if (!a.doc) return s;
        while (s < s1) {
            if (sfilled < 0 || s < sbase || s >= sbase + 64) look(s);
            const uint64_t m = stage_hit >> (s - sbase);
            if (m) return s + (int)__builtin_ctzll(m);
            s = sbase + 64;
        }
        return s1;
    };

    const int32_t* doc = a.doc ? a.doc + (int64_t)b * a.Lk : nullptr;
    R ring(sh, a.Lq, a.D, a.qs[1], a.dos[1]);
    int key[NK];
    bool dead = false;
    const int per = (a.G + a.nparts - 1) / a.nparts;   // heads of a part
    for (int h = hk * a.G + part * per; h < hk * a.G + min((part + 1) * per, a.G); ++h) {
        ring.from((const E*)a.q + b * a.qs[0] + h * a.qs[2], (const E*)a.dout + b * a.dos[0] + h * a.dos[2]);
        const float* stat = a.rowstat + ((int64_t)b * a.H + h) * a.Lq;
        ring.wp[0] = (const uint32_t*)stat;
        ring.wp[1] = (const uint32_t*)(stat + (int64_t)a.B * a.H * a.Lq);
        const float slope = BIAS ? a.slopes[h] * LOG2E : 0.f;
        __syncthreads();   // the places the last head used are free
        if (doc) {
            ring.wp[2] = (const uint32_t*)(doc + off);   // the rows' own documents
            ring.vfirst = max(0, -off);
        }
        // q0: the stage to use, q1 the one after, whose loads are in flight (NS = 3)
        int q0 = seek(s0), q1 = q0 < s1 ? seek(q0 + 1) : s1;
        if (R::NS > 1 && q0 < s1) ring.issue(q0, 0);
        if (R::NS > 1 && q1 < s1) ring.issue(q1, 1);
        if (h == hk * a.G + part * per) {
            // the keys that are padding read as 0 and lie before every row's first
#pragma unroll
            for (int m = 0; m < NK; ++m) {
                const int j = jw + 16 * m + c;
                const bool live = key_live(a, b, j, n);
                key[m] = live ? j : -1;
                dead |= !live;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    frag_keep<IO>(k[m][kk], live && 32 * kk + 8 * g < a.D);
                    frag_keep<IO>(v[m][kk], live && 32 * kk + 8 * g < a.D);
                }
            }
            dead = __any(dead);
        }
        int place = 0;
        for (; q0 < s1; place = R::after(place)) {
            const int tb = q0 * BN, pb = off + tb, here = q0;
            if constexpr (R::NS == 1) {
                __syncthreads();
                ring.issue(q0, 0);
                ring.ready(false);
            } else {
                ring.ready(q1 < s1);
            }
            // what look() said of this stage, before it may look further
            bool whit[SP], wfull[SP];
#pragma unroll
            for (int x = 0; x < SP; ++x) {
                if (doc) {
                    if (here < sbase || here >= sbase + 64) look(here);
                    whit[x] = hit[x] >> (here - sbase) & 1;
                    wfull[x] = full[x] >> (here - sbase) & 1;
                } else {
                    const RowRange st = token_range(a, n, tb + STRIP * x, STRIP);
                    whit[x] = st.lo <= jw + WK - 1 && st.hi >= jw;
                    wfull[x] = st.last <= jw && st.pos >= jw + WK - 1;
                }
            }
            q0 = q1;
            q1 = q1 < s1 ? seek(q1 + 1) : s1;
            if (R::NS > 1 && q1 < s1) ring.issue(q1, R::freed(place));
            const E *Qt = sh.x[place], *Gt = sh.y[place];
            const float *Ls = (const float*)sh.w[0][place], *Dl = (const float*)sh.w[1][place];
            const int* Doc = (const int*)sh.w[2][place];
            uint64_t alive = ~0ull;
            bool masked = dead;   // some strip needs its rows' bounds
#pragma unroll
            for (int x = 0; x < SP; ++x) masked |= whit[x] && !wfull[x];
            if (doc || pb < 0 || tb + BN > a.Lq || masked) {
                // lane's row of the stage: its first key, and how many it sees less one
                const int r = lane % BN, p = pb + r;
                int lo = max(0, p - a.window + 1);
                if (doc) lo = max(lo, Doc[r]);
                const bool some = tb + r < a.Lq && p >= 0 && lo <= p;
                first[wave][r] = some ? lo : BIG;
                span[wave][r] = some ? p - lo : -1;
                wave_lds_order();
                // rows that see nothing, or lie past the last: 0, whatever the memory holds
                alive = __ballot(some);
                if (BN < 64) alive |= ~0ull << (BN & 63);
                if (alive != ~0ull) ring.blank(place, alive);
            }
#pragma unroll
            for (int hf = 0; hf < SP; ++hf) {   // 32 tokens at a time
                if (!whit[hf]) continue;   // no row of the strip sees this wave's keys
                const bool edge = dead || !wfull[hf] || alive != ~0ull;
                // rows x keys
                f32x4 w[2][NK], dp[2][NK];
#pragma unroll
                for (int rb = 0; rb < 2; ++rb) {
#pragma unroll
                    for (int m = 0; m < NK; ++m) w[rb][m] = dp[rb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const Frag<IO> fq = frag_row<IO, DP>(Qt, 32 * hf + 16 * rb, kk, g, c);
                        const Frag<IO> fg = frag_row<IO, DP>(Gt, 32 * hf + 16 * rb, kk, g, c);
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
                    // the row's part of the exponent: - lse, and - slope of its distance to the
                    // stage's first token
                    const f32x4 ls = *(const f32x4*)(Ls + rr), dl = *(const f32x4*)(Dl + rr);
                    f32x4 rt;
#pragma unroll
                    for (int r = 0; r < 4; ++r) rt[r] = BIAS ? __builtin_fmaf(-slope, (float)(rr + r), -ls[r]) : -ls[r];
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
                            const int4 fi = *(const int4*)&first[wave][rr], sp = *(const int4*)&span[wave][rr];
                            const int f4[4] = {fi.x, fi.y, fi.z, fi.w}, s4[4] = {sp.x, sp.y, sp.z, sp.w};
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (key[m] - f4[r] < 0 || key[m] - f4[r] > s4[r]) w[rb][m][r] = 0.f;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            dp[rb][m][r] = w[rb][m][r] * (dp[rb][m][r] - dl[r]);
                            if constexpr (CAP != UNCAPPED) dp[rb][m][r] *= cf[r];
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
                    const Frag<IO> fg = frag_tr<IO, DP>(Gt, 32 * hf, 16 * d, g, c);
                    const Frag<IO> fq = frag_tr<IO, DP>(Qt, 32 * hf, 16 * d, g, c);
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
        if (a.nparts > 1) {
            float* p = a.part + (((int64_t)part * a.nbh + bh) * a.Lk + j) * 2 * a.D;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int x = 16 * d + 4 * g;
                if (x >= a.D) continue;
                *(f32x4*)(p + x) = dk[d][m] * a.scale;
                *(f32x4*)(p + a.D + x) = dv[d][m];
            }
            continue;
        }
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

// dk, dv of a key as the sum of its parts, in order; four values a thread.
template <class IO>
__global__ __launch_bounds__(256) void attn_bwd_join(AttnArgs a, int64_t n)
{
    using E = typename IO::T;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int per = 2 * a.D / 4;   // threads of a key
    const int64_t row = i / per;
    const int x = (int)(i % per) * 4;
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < a.nparts; ++p)
        sum += *(const f32x4*)(a.part + (((int64_t)p * a.nbh * a.Lk) + row) * 2 * a.D + x);
    const int bh = (int)(row / a.Lk), j = (int)(row % a.Lk), b = bh / a.Hkv, hk = bh % a.Hkv;
    E* o = x < a.D ? (E*)a.dk + b * a.dks[0] + (int64_t)j * a.dks[1] + hk * a.dks[2] + x
                   : (E*)a.dv + b * a.dvs[0] + (int64_t)j * a.dvs[1] + hk * a.dvs[2] + x - a.D;
    put4<IO>(o, sum);
}

template <class IO, int DP, Cap CAP, bool BIAS, class S>
hipError_t go_q(AttnArgs a, hipStream_t st)
{
    a.ntile = (a.Lq + S::ROWS - 1) / S::ROWS;
    const int64_t blocks = (int64_t)a.ntile * a.B * a.H;
    if (!grid_ok(blocks, 64 * S::NW)) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_bwd_q<IO, DP, CAP, BIAS, S>), dim3((unsigned)blocks), dim3(64 * S::NW), 0, st, a);
    return hipGetLastError();
}

template <class IO, int DP, Cap CAP, bool BIAS, class S>
hipError_t go_kv(const AttnArgs& a, hipStream_t st)
{
    const int64_t blocks = (int64_t)((a.Lk + S::ROWS - 1) / S::ROWS) * a.nbh * a.nparts;
    if (!grid_ok(blocks, 64 * S::NW)) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((attn_bwd_kv<IO, DP, CAP, BIAS, S>), dim3((unsigned)blocks), dim3(64 * S::NW), 0, st, a);
    return hipGetLastError();
}

// Workgroups of 128 rows or keys below which they take 64 (12 heads of 64, L 1024, bfloat16: 384
// workgroups 69 us, 768 of half the size 55; 768 83, 1536 84; 4096 and 8192 305 and 307 us); and
// workgroups below which the heads that share a key head are dealt out to several, whose parts a
// third kernel adds (B 2, L 1500, 8 heads of 128 on 2: 138 us, 343 in one part; L 2048, 16 heads of
// 64 on one: 105 and 848; 512 and 2048 instead of 1024 are 4% and more slower).
constexpr int64_t ENOUGH = 512, PARTS_FILL = 1024;

bool few(int64_t L, int64_t heads) { return (L + 127) / 128 * heads < ENOUGH; }

int parts(const AttnArgs& a)
{
    const int64_t bk = few(a.Lk, a.nbh) ? 64 : 128, wgs = (a.Lk + bk - 1) / bk * a.nbh;
    if (a.G <= 1 || wgs == 0 || wgs >= PARTS_FILL || a.Lq == 0) return 1;
    const int64_t want = std::min<int64_t>(a.G, (PARTS_FILL + wgs - 1) / wgs);
    const int64_t per = (a.G + want - 1) / want;   // heads of a part
    return (int)((a.G + per - 1) / per);
}

template <class IO, int DP, Cap CAP, bool BIAS>
hipError_t go(const AttnArgs& a, hipStream_t st)
{
    // float32: one block a wave (operands and results take twice the registers)
    constexpr int N = IO::SIZE == 4 ? 1 : 2;
    hipError_t e = few(a.Lq, (int64_t)a.B * a.H) ? go_q<IO, DP, CAP, BIAS, Shape<1, 4>>(a, st)
                                                 : go_q<IO, DP, CAP, BIAS, Shape<N, 8 / N>>(a, st);
    if (e != hipSuccess) return e;
    e = few(a.Lk, a.nbh) ? go_kv<IO, DP, CAP, BIAS, Shape<1, 4>>(a, st) : go_kv<IO, DP, CAP, BIAS, Shape<N, 8 / N>>(a, st);
    if (e != hipSuccess || a.nparts == 1) return e;
    const int64_t n = (int64_t)a.nbh * a.Lk * (2 * a.D / 4), blocks = (n + 255) / 256;
    if (!grid_ok(blocks, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_bwd_join<IO>), dim3((unsigned)blocks), dim3(256), 0, st, a, n);
    return hipGetLastError();
}

template <class IO, int DP>
hipError_t pick(const AttnArgs& a, hipStream_t st)
{
    return with_options<IO, true>(a, [&](auto cap, auto bias) {
        return go<IO, DP, decltype(cap)::value, decltype(bias)::value>(a, st);
    });
}

// strips of a batch row, whole tiles of 128 tokens and whole stages
int64_t strip_count(const AttnArgs& a) { return (a.Lq + 127) / 128 * (int64_t)(128 / STRIP); }
size_t stat_bytes(const AttnArgs& a) { return ((size_t)a.B * a.H * a.Lq * 2 * sizeof(float) + 255) / 256 * 256; }

size_t strip_bytes(const AttnArgs& a)
{
    return a.doc ? ((size_t)(a.B * strip_count(a)) * sizeof(int4) + 255) / 256 * 256 : 0;
}

}  // namespace

size_t attn_bwd_bytes(const AttnArgs& a)
{
    const int np = parts(a);
    return stat_bytes(a) + strip_bytes(a) + (np > 1 ? (size_t)np * a.nbh * a.Lk * 2 * a.D * sizeof(float) : 0);
}

hipError_t launch_attn_bwd(Store s, const AttnArgs& a, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.nstrip = (int)strip_count(a);
    x.nparts = parts(a);
    x.rowstat = (float*)ws;
    x.strips = (int4*)((char*)ws + stat_bytes(a));
    x.part = (float*)((char*)ws + stat_bytes(a) + strip_bytes(a));
    if (s == Store::F32) return a.D <= 64 ? pick<f32_io, 64>(x, st) : pick<f32_io, 128>(x, st);
    return a.D <= 64 ? pick<bf16_io, 64>(x, st) : pick<bf16_io, 128>(x, st);
}

}  // namespace sc
