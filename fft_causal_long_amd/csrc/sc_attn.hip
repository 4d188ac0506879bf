// Causal attention with a window, a distance bias, a tanh cap and documents: forward (gfx950).
//
// The hybrid stack of "Caracal: Causal Architecture via Spectral Mixing" (key design 3) puts a
// sliding-window attention layer after every two Fourier layers.  Query row i of batch row b
// sits at position p = n_b - Lq + i; it sees the keys lo_p <= j <= p:
//
//     x = scale q.k,  s = cap tanh(x / cap)  (cap > 0),  s -= slope_h (p - j)
//     o = sum_j softmax(s)_j v_j,   lse = log sum_j exp(s_j)
//
// One pass over the keys with a running maximum and sum, in base 2.  The heads that share a key
// head are packed into one row axis (row r = token r / G, head r % G), so a key tile is read
// once for all of them.  A workgroup takes 128 rows, 32 per wave, and walks tiles of 64 keys
// staged through LDS with the next tile's loads in flight.  Scores are made transposed
// (keys x rows): a lane then holds 16 keys of one row per 16-row block, the row's statistics
// are the lane's own but for two shuffles, and the weights are the B operand of the second
// product as they stand (sc_attn.h).  A wave skips tiles none of its rows sees and masks only
// tiles that an edge crosses.
// What bounds it: with a window of 256 the bytes of q, k, v, o; without one the vector
// instructions per score (scale, max, exponential, sum, rounding), not the matrix products.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace attn;

constexpr int BN = 64;            // keys of a tile
constexpr int NQ = 2;             // 16-row blocks of a wave
constexpr int WM = 16 * NQ;       // rows of a wave
constexpr int BM = 4 * WM;        // rows of a workgroup

template <class IO, int DP, bool CAP, bool BIAS>
__global__ __launch_bounds__(NT) void attn_fwd(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int P = pitch<IO, DP>, V = vec_elems<IO>, CH = DP / V, NCH = BN * CH / NT;
    constexpr int KK = DP / 32, ND = DP / 16;
    __shared__ __attribute__((aligned(16))) E Kt[BN * P];
    __shared__ __attribute__((aligned(16))) E Vt[BN * P];
    __shared__ int range[2][4];

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    id /= (uint32_t)a.nbh;
    const int split = (int)(id % (uint32_t)a.nsplit);
    // the last rows see most keys: first
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)a.nsplit);
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;

    // this lane's rows
    int row[NQ], pos[NQ], lo[NQ];
    bool empty[NQ];
    Frag<IO> q[NQ][KK];
    float slope[NQ];
    int wlo = BIG, whi = -1, mlo = 0, mpos = BIG;   // lowest key, highest key; to skip masking
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
            // an empty row takes part with q = 0 and nothing masked; its result is dropped
            lo[m] = 0;
            pos[m] = BIG;
        }
        slope[m] = BIAS ? a.slopes[h] * LOG2E : 0.f;
        const E* qp = (const E*)a.q + b * a.qs[0] + (int64_t)i * a.qs[1] + h * a.qs[2];
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            const int d = 32 * k + 8 * g;
            q[m][k] = !empty[m] && d < a.D ? frag_at<IO>(qp + d) : frag_zero<IO>();
        }
    }
    wlo = wave_min(wlo);
    whi = wave_max(whi);
    mlo = wave_max(mlo);
    mpos = wave_min(mpos);
    if (lane == 0) {
        range[0][wave] = wlo;
        range[1][wave] = whi;
    }
    __syncthreads();
    const int klo = min(min(range[0][0], range[0][1]), min(range[0][2], range[0][3]));
    const int khi = max(max(range[1][0], range[1][1]), max(range[1][2], range[1][3]));
    int t0 = khi < 0 ? 0 : klo / BN, t1 = khi < 0 ? 0 : khi / BN + 1;
    if (a.nsplit > 1) {
        const int per = (t1 - t0 + a.nsplit - 1) / a.nsplit;
        t0 = min(t1, t0 + split * per);
        t1 = min(t1, t0 + per);
    }

    const float scale2 = CAP ? a.scale / a.cap : a.scale * LOG2E, cap2 = a.cap * LOG2E;
    f32x4 o[ND][NQ];
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        mx[m] = -INFINITY;
        sum[m] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const E* kp = (const E*)a.k + b * a.ks[0] + hk * a.ks[2];
    const E* vp = (const E*)a.v + b * a.vs[0] + hk * a.vs[2];
    uint4 rk[NCH], rv[NCH];
    int rdoc = 0;
    // keys past the sequence and padding read as 0, whatever the memory holds
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
        if (j0 > whi || j0 + BN - 1 < wlo) continue;   // no row of this wave sees it

        // scores, keys x rows
        f32x4 s[4][NQ];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
            for (int m = 0; m < NQ; ++m) s[kb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                const Frag<IO> f = frag_at<IO>(Kt + (16 * kb + c) * P + 32 * k + 8 * g);
#pragma unroll
                for (int m = 0; m < NQ; ++m) s[kb][m] = mma(f, q[m][k], s[kb][m]);
            }
        }
        const bool edge = j0 < mlo || j0 + BN - 1 > mpos || live != ~0ull;
        Frag<IO> w[2][NQ];
#pragma unroll
        for (int m = 0; m < NQ; ++m) {
            // CAP and BIAS: s becomes the score in base 2; otherwise it stays the raw product
            // and the scale goes into the exponential's multiply-add
            const float far = (float)(j0 + 4 * g - pos[m]);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float x = s[kb][m][r];
                    if constexpr (CAP) x = cap2 * tanh_of<IO>(x * scale2);
                    if constexpr (BIAS) {
                        const float bias = slope[m] * (far + (float)(16 * kb + r));
                        x = CAP ? x + bias : __builtin_fmaf(x, scale2, bias);
                    }
                    s[kb][m][r] = x;
                }
            if (edge) {
#pragma unroll
                for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int jj = 16 * kb + 4 * g + r, j = j0 + jj;
                        if (j < lo[m] || j > pos[m] || !(live >> jj & 1)) s[kb][m][r] = -INFINITY;
                    }
            }
            float top = s[0][m][0];
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, s[kb][m][r]);
            top = gmax(top);
            if constexpr (!CAP && !BIAS) top *= scale2;
            const float now = fmaxf(mx[m], top);
            const float base = now == -INFINITY ? 0.f : now;   // nothing seen yet: weights are 0
            if (__any(now > mx[m])) {
                const float f = exp2_hw(mx[m] - base);
                sum[m] *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[d][m] *= f;
                mx[m] = now;
            }
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = exp2_hw(CAP || BIAS ? s[kb][m][r] - base
                                                        : __builtin_fmaf(s[kb][m][r], scale2, -base));
                    s[kb][m][r] = e;
                    sum[m] += e;
                }
            w[0][m] = frag_of<IO>(s[0][m], s[1][m]);
            w[1][m] = frag_of<IO>(s[2][m], s[3][m]);
        }
        // o^T += v^T w
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const Frag<IO> f = frag_tr<IO, P>(Vt, 32 * hf, 16 * d, g, c);
#pragma unroll
                for (int m = 0; m < NQ; ++m) o[d][m] = mma(f, w[hf][m], o[d][m]);
            }
    }

#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        const float l = gsum(sum[m]);
        if (row[m] >= a.nrow) continue;
        // a split that the row sees nothing of: weight 0 in the join
        const bool none = empty[m] || l == 0.f;
        const float inv = none ? 0.f : 1.0f / l;
        const float ls = none ? -INFINITY : mx[m] + __builtin_amdgcn_logf(l);
        const int i = row[m] / a.G, h = hk * a.G + row[m] % a.G;
        if (a.nsplit > 1) {
            const int64_t at = ((int64_t)split * a.nbh + bh) * a.nrow + row[m];
            float* op = a.part + at * a.D;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int d0 = 16 * d + 4 * g;
                if (d0 < a.D)
                    *(float4*)(op + d0) = make_float4(none ? 0.f : o[d][m][0] * inv, none ? 0.f : o[d][m][1] * inv,
                                                      none ? 0.f : o[d][m][2] * inv, none ? 0.f : o[d][m][3] * inv);
            }
            if (g == 0) a.part_lse[at] = ls;
            continue;
        }
        E* op = (E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int d0 = 16 * d + 4 * g;
            if (d0 >= a.D) continue;
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = none ? 0.f : o[d][m][r] * inv;
            if constexpr (IO::SIZE == 2)
                *(uint2*)(op + d0) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            else
                *(float4*)(op + d0) = make_float4(x[0], x[1], x[2], x[3]);
        }
        if (a.lse && g == 0) a.lse[((int64_t)b * a.H + h) * a.Lq + i] = ls * LN2;
    }
}

// Joins the splits of a row: o = sum_s 2^(lse_s - lse) o_s.  One wave per row, 64 columns a turn.
template <class IO>
__global__ __launch_bounds__(NT) void attn_join(AttnArgs a)
{
    using E = typename IO::T;
    const int64_t total = (int64_t)a.nbh * a.nrow;
    const int64_t at = (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= total) return;
    float mx = -INFINITY;
    for (int s = lane; s < a.nsplit; s += 64) mx = fmaxf(mx, a.part_lse[s * total + at]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    for (int s = lane; s < a.nsplit; s += 64) sum += exp2_hw(a.part_lse[s * total + at] - base);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    const int bh = (int)(at / a.nrow), r = (int)(at % a.nrow);
    const int b = bh / a.Hkv, i = r / a.G, h = bh % a.Hkv * a.G + r % a.G;
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
    E* op = (E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
    for (int d = lane; d < a.D; d += 64) {
        float x = 0.f;
        for (int s = 0; s < a.nsplit; ++s) {
            const float w = exp2_hw(a.part_lse[s * total + at] - base) * inv;
            x = __builtin_fmaf(w, a.part[(s * total + at) * a.D + d], x);
        }
        IO::store(op, d, x);
    }
    if (a.lse && lane == 0)
        a.lse[((int64_t)b * a.H + h) * a.Lq + i] = sum > 0.f ? (mx + __builtin_amdgcn_logf(sum)) * LN2 : -INFINITY;
}

// Key splits: as many as fill the GPU when the rows alone do not, each of at least 256 keys.
constexpr int64_t FILL = 512;
constexpr int64_t SPLIT_MIN = 256;
constexpr int64_t SPLIT_MAX = 64;

int splits(int64_t wgs, int64_t Lk, int window, int64_t Lq)
{
    const int64_t keys = std::min<int64_t>(Lk, (int64_t)window + std::min<int64_t>(Lq, BM));
    if (wgs <= 0 || 2 * wgs > FILL) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(FILL + wgs - 1) / wgs, keys / SPLIT_MIN, SPLIT_MAX}));
}

template <class IO, int DP, bool CAP, bool BIAS>
hipError_t go(const AttnArgs& a, int64_t blocks, hipStream_t st)
{
    hipLaunchKernelGGL((attn_fwd<IO, DP, CAP, BIAS>), dim3((unsigned)blocks), dim3(NT), 0, st, a);
    return hipGetLastError();
}

template <class IO, int DP>
hipError_t pick(const AttnArgs& a, int64_t blocks, hipStream_t st)
{
    if (a.cap > 0.f)
        return a.slopes ? go<IO, DP, true, true>(a, blocks, st) : go<IO, DP, true, false>(a, blocks, st);
    return a.slopes ? go<IO, DP, false, true>(a, blocks, st) : go<IO, DP, false, false>(a, blocks, st);
}

template <class IO>
hipError_t run(AttnArgs a, hipStream_t st)
{
    a.ntile = (a.nrow + BM - 1) / BM;
    const int64_t wgs = (int64_t)a.ntile * a.nbh;
    a.nsplit = splits(wgs, a.Lk, a.window, a.Lq);
    const int64_t blocks = wgs * a.nsplit;
    if (!grid_ok(blocks, NT)) return hipErrorInvalidValue;
    a.part_lse = a.part + (int64_t)a.nsplit * a.nbh * a.nrow * a.D;
    const hipError_t e = a.D <= 64 ? pick<IO, 64>(a, blocks, st) : pick<IO, 128>(a, blocks, st);
    if (e != hipSuccess || a.nsplit == 1) return e;
    const int64_t jb = ((int64_t)a.nbh * a.nrow + NT / 64 - 1) / (NT / 64);
    hipLaunchKernelGGL((attn_join<IO>), dim3((unsigned)jb), dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

size_t attn_fwd_bytes(const AttnArgs& a)
{
    const int64_t rows = (int64_t)a.nbh * a.nrow;
    const int ns = splits((a.nrow + BM - 1) / BM * (int64_t)a.nbh, a.Lk, a.window, a.Lq);
    return ns > 1 ? (size_t)ns * rows * (a.D + 1) * sizeof(float) : 0;
}

hipError_t launch_attn(Store s, const AttnArgs& a, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.part = (float*)ws;
    return s == Store::F32 ? run<f32_io>(x, st) : run<bf16_io>(x, st);
}

}  // namespace sc
