// Causal attention over a cache of 8-bit codes (layout in sc_cache.h), with a window, first tokens that
// stay visible (sinks), a distance bias and a tanh cap (gfx950).
//
// Query row i of batch row b stands at p = len_b - Lq + i and sees j <= p with j > p - window or
// j < sinks.  With codes K, V and block scales ks, vs:
//
//     x = scale ks q.K,  s = cap tanh(x / cap)  (cap > 0),  s -= slope_h (p - j)
//     o = sum_j softmax(s)_j vs V_j,   lse = log sum_j exp(s_j)
//
// One pass with a running base and sum, in base 2.  Codes are exact in half precision, so both products
// run on the half-precision matrix instruction: a query row is multiplied by the power of two that
// brings its largest value to 2^14 .. 2^15 (bfloat16 values then are exact down to 2^-29 of it; float32
// ones are the sum of two halves, 2^-22 of each).  A weight is two halves in float32 calls and in those
// of few rows.  In bfloat16 calls of more rows it is one, 11 bits: off by 2^-12 of itself at most, a
// sixteenth of the result's own rounding, while the second half and its product took a quarter to a third
// of the call (2048 tokens after 6144, 16 heads of 128 on 4: 214 us for 172; B 8, 1024 tokens over 4096, 16
// heads of 64: 236 for 173; but one token over the caches of the first call below: 45.3 for 43.8).  A
// block's vs goes into the weights' exponent, w = 2^(s + log2 vs - base), so that every weight is
// relative to the row's largest contribution to o, whatever the scales, and off by 2^-32 of that at most
// besides (half precision ends at 2^-24, the base stands for 2^HEAD); the sum takes w / vs.
// The heads that share a key head are packed into one row axis, scores are made transposed (keys x
// rows) and the blocks' byte order is that of the operands (sc_cache.h), so a score block, rounded, is
// the operand of the second product and codes go from memory to the products without an exchange.
//
// Few rows (decoding): the four waves of a workgroup share 16 rows and take blocks in turn, each with
// its next block on its way in registers, and join their results through LDS; keys are split over
// workgroups to fill the GPU.  More rows: a wave has rows of its own; a block's codes are turned into
// half precision once, a quarter by each wave, and shared through two LDS places.
//
// Measured (MI355X; a large copy moves 5.4 TB/s, reads alone up to 6.3, a half-precision product of 8192^3
// reaches 1200 TFLOP/s), whole calls:
//  * 8 sequences over ragged caches of up to 65536, one token, 16 heads of 64 on 4, int8: 45 us, of it 40 the
//    kernel (5.3 TB/s of the codes) and 4.6 the join: bound by the codes' bytes.  Loads past the caches took
//    the call from 50 to 44 (and the weights' second half to 45).  float32 45; the same in bfloat16 caches: 91.
//  * 64 sequences of 2048 to 4096, one token, 16 heads of 128 on 4, e4m3: 43 us for 202 MB (4.7 TB/s): 256
//    workgroups that each walk one row's blocks, one wave a SIMD.
//  * 32 sequences, window 256 and 4 sinks, 16 heads of 64, e4m3 in a pool: 10 us of kernel, five blocks a
//    workgroup: the chain length, table, codes, scores.
//  * 4 sequences of up to 10007, 5 tokens, 12 heads of 64, float32, capped: 18 us and 4 of join for 50 MB:
//    the same chain before the bytes, three blocks a wave.
//  * 5 and 16 tokens over the first call's caches (20 and 64 packed rows): 74 and 78 us, one block of codes
//    ahead a workgroup where one row has one a wave, and at 20 rows two waves of four without rows.
//  * 2048 tokens over 8192, 16 heads of 128 on 4, int8: 172 us, 700 TFLOP/s of the products that the mask
//    leaves (sc_causal_attn on bfloat16: 222 to 228); e4m3 178; float32, of two halves each, 237.  Three
//    things take turns: vector instructions (176 for 16 x 64 scores, of them 64 the conversion, 16
//    exponentials), 47% of the cycles; matrix instructions, 27%; and LDS, of which a wave of 16 rows reads an
//    operand of 1 KB for each product, 32 a block, and writes 8: 29 and 7 MB a CU, 95 and 24 us of the 172
//    at 128 bytes a clock.  At 1.7 waves a SIMD they do not overlap fully.  Four waves a SIMD (the keys of a
//    block in two halves) changed nothing, the next block's conversion placed beside the first product made
//    it 198, each wave converting for itself 257.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_cache.h"

namespace sc {

namespace {

using namespace attn;
using namespace cache;

constexpr float SLACK = 8.f;   // a row's base may lag its maximum by this (base 2)
constexpr float HEAD = 7.f;    // weights are 2^HEAD at the base: up to 2^15 in half precision

// q times this brings a row's largest magnitude to 2^14 .. 2^15.
constexpr int Q_TOP = 14;

// A workgroup's shape: NQ 16-row blocks a wave, NW waves; KEYS: the waves share the rows and take the
// blocks in turn.
template <int NQ_, int NW_, bool KEYS_>
struct Shape {
    static constexpr int NQ = NQ_, NW = NW_, WM = 16 * NQ, BM = KEYS_ ? WM : NW * WM;
    static constexpr bool KEYS = KEYS_;
};

__device__ __forceinline__ f32x4 mma(const half8_t& a, const half8_t& b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Eight float32 values as halves, and what that left of them.
__device__ __forceinline__ half8_t halves_of(const float (&x)[8])
{
    half8_t h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[e];
    return h;
}
__device__ __forceinline__ half8_t rest_of(const float (&x)[8], const half8_t& h)
{
    half8_t r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (_Float16)(x[e] - (float)h[e]);
    return r;
}

// The 64-token blocks a strip of rows sees, [0, sink) and [t0, t1), newest first: with a distance bias
// the first base is then near the last one.  (A base that rises by x leaves the scores it rose for with
// the roundings of x: from the first tokens on, 4096 keys of slope 1 / sqrt 2 cost lse 5e-6.)
struct Blocks {
    int sink, t0, t1;
    __device__ __forceinline__ int count() const { return sink + t1 - t0; }
    __device__ __forceinline__ int at(int u) const { return u < t1 - t0 ? t1 - 1 - u : sink - 1 - (u - (t1 - t0)); }
};

// Positions p0 .. p1 of the tokens t .. t + count - 1 that exist (p0 > p1: none).
__device__ __forceinline__ void positions(const AttnArgs& a, int64_t off, int t, int count, int& p0, int& p1)
{
    p0 = (int)std::min<int64_t>(std::max<int64_t>(off + t, 0), INT_MAX);
    p1 = (int)std::max<int64_t>(std::min<int64_t>(off + t + count - 1, a.Lk - 1), -1);
}

// Read once: past the caches' own keeping.
__device__ __forceinline__ uint4 stream16(const uint8_t* p)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 x = __builtin_nontemporal_load((const u32x4*)p);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// A block of a row and head: where it lies in the pool (-1: none) and its scales, loaded with its codes.
struct Place {
    int p;
    float ks, vs;
    __device__ __forceinline__ Place(const CacheArgs& c, int b, int hk, int blk) : p(block_of(c, b, blk))
    {
        const int64_t at = (int64_t)std::max(p, 0) * c.Hkv + hk;
        ks = c.ks[at];
        vs = c.vs[at];
    }
    __device__ __forceinline__ Place() : p(-1), ks(0.f), vs(0.f) {}
    __device__ __forceinline__ int64_t bytes(const CacheArgs& c, int hk) const
    {
        return ((int64_t)std::max(p, 0) * c.Hkv + hk) * (T * c.D);
    }
};

// One block's bytes of a wave: the operands of lane (g, c), 16 bytes each.
template <int J>
struct Bytes;
template <>
struct Bytes<0> {};
template <int J>
struct Bytes {
    uint4 k[4][J], v[4 * J];
    // `chunk` 16-value chunks of D; a lane past them reads the first (its query values are 0)
    __device__ __forceinline__ void from(const uint8_t* kp, const uint8_t* vp, int chunks, int g, int lane)
    {
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int ch = 4 * j + g < chunks ? 4 * j + g : 0;
                k[kb][j] = stream16(kp + ((kb * chunks + ch) * 16 + (lane & 15)) * 16);
            }
#pragma unroll
        for (int d = 0; d < 4 * J; ++d) v[d] = stream16(vp + ((d < chunks ? d : 0) * 64 + lane) * 16);
    }
};

template <class IO, Code CODE, int J, Cap CAP, bool BIAS, class S>
__global__ __launch_bounds__((64 * S::NW), 2) void cached_attn(AttnArgs a, CacheArgs cc, int sinks)
{
    using E = typename IO::T;
    constexpr int NQ = S::NQ, NW = S::NW, WM = S::WM, BM = S::BM, ND = 4 * J, P = IO::SIZE == 4 ? 2 : 1;
    constexpr int PW = S::KEYS ? 2 : P;   // halves of q, of a weight
    constexpr int DP = 64 * J, STAGE = 2 * T * DP * 2;
    // what the waves join, or two blocks in half precision
    constexpr int LDS = S::KEYS ? NW * WM * (DP + 2) * 4 : 2 * STAGE;
    __shared__ __attribute__((aligned(1024))) uint8_t sh[LDS];

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    id /= (uint32_t)a.nbh;
    const int split = (int)(id % (uint32_t)a.nsplit);
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)a.nsplit);   // the last rows see most keys: first
    const int b = bh / a.Hkv, hk = bh % a.Hkv, chunks = a.D / 16;
    const int64_t off = (int64_t)a.kv_len[b] - a.Lq;   // position of token 0
    const int n = (int)std::min<int64_t>(std::max<int64_t>(off + a.Lq, 0), a.Lk);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // what the wave's rows and the workgroup's see
    const int rw = tile * BM + (S::KEYS ? 0 : wave * WM);   // the wave's first row
    int p0, p1, w0, w1;
    {
        const int t = token_of(a, min(tile * BM, a.nrow - 1));
        positions(a, off, t, token_of(a, min(tile * BM + BM, a.nrow) - 1) - t + 1, p0, p1);
        const int tw = token_of(a, min(rw, a.nrow - 1));
        positions(a, off, tw, rw < a.nrow ? token_of(a, min(rw + WM, a.nrow) - 1) - tw + 1 : 0, w0, w1);
    }
    const int wlo = max(0, w0 - a.window + 1), wlast = max(0, w1 - a.window + 1);   // first keys of the wave's rows
    Blocks bl = {0, 0, 0};
    if (p0 <= p1) {
        const int klo = max(0, p0 - a.window + 1);
        bl.t0 = klo / T;
        bl.t1 = p1 / T + 1;
        bl.sink = min((min(sinks, klo) + T - 1) / T, bl.t0);
    }
    int u0 = 0, u1 = bl.count();
    if (a.nsplit > 1) {
        const int per = (u1 + a.nsplit - 1) / a.nsplit;
        u0 = min(u1, split * per);
        u1 = min(u1, u0 + per);
    }

    // KEYS: this wave's blocks are u0 + wave, + NW, ...; the first is on its way before the queries are
    Bytes<S::KEYS ? J : 0> now, next;
    auto bring = [&](int u, auto& to) {
        const Place p(cc, b, hk, bl.at(u));
        const int64_t at = p.bytes(cc, hk);
        to.from((const uint8_t*)cc.k + at, (const uint8_t*)cc.v + at, chunks, g, lane);
        return p;
    };
    Place here;
    if constexpr (S::KEYS)
        if (u0 + wave < u1) here = bring(u0 + wave, now);

    // this lane's rows
    int row[NQ], pos[NQ], lo[NQ];
    bool empty[NQ];
    half8_t q[NQ][J][2][P];
    float slope[NQ];
    int back[NQ];   // the exponent that undoes the row's power of two
    const float scale2 = score_scale<CAP>(a), cap2 = a.cap * LOG2E;
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        row[m] = rw + 16 * m + c;
        const bool in = row[m] < a.nrow;
        const int i = in ? token_of(a, row[m]) : 0, h = in ? hk * a.G + row[m] - i * a.G : hk * a.G;
        const int64_t p = off + i;
        empty[m] = !in || p < 0 || p >= a.Lk;
        // an empty row takes part with q = 0 and nothing masked; its result is dropped
        pos[m] = empty[m] ? BIG : (int)p;
        lo[m] = empty[m] ? 0 : max(0, (int)p - a.window + 1);
        slope[m] = BIAS ? a.slopes[h] * LOG2E : 0.f;
        const E* qp = (const E*)a.q + b * a.qs[0] + (int64_t)i * a.qs[1] + h * a.qs[2];
        float x[J][2][8], top = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = 16 * (4 * j + g) + 8 * k;
                const bool on = !empty[m] && d < a.D;
                const Frag<IO> f = frag_at<IO>(qp + (d < a.D ? d : 0));
                if constexpr (IO::SIZE == 2) {
                    const uint32_t w[4] = {f.v.x, f.v.y, f.v.z, f.v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[j][k][e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
                } else {
                    const float w[8] = {f.a.x, f.a.y, f.a.z, f.a.w, f.b.x, f.b.y, f.b.z, f.b.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[j][k][e] = w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[j][k][e] = on ? x[j][k][e] : 0.f;
                    top = fmaxf(top, fabsf(x[j][k][e]));
                }
            }
        top = gmax(top);
        const int ex = min((int)(__float_as_uint(top) >> 23), 254) - 127;
        back[m] = ex - Q_TOP;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][k][e] = __builtin_amdgcn_ldexpf(x[j][k][e], Q_TOP - ex);
                q[m][j][k][0] = halves_of(x[j][k]);
                if constexpr (P == 2) q[m][j][k][1] = rest_of(x[j][k], q[m][j][k][0]);
            }
    }
    f32x4 o[ND][NQ];
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        mx[m] = -INFINITY;
        sum[m] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // one block, its operands given by kf(kb, j, half of the 16 values) and vf(d, half of the 16 keys)
    auto block = [&](int j0, const Place& at, auto&& kf, auto&& vf) {
        const int ke = exponent_of_scale(at.ks);
        const int ve = exponent_of_scale(at.vs);
        f32x4 s[4][NQ];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
            for (int m = 0; m < NQ; ++m) s[kb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const half8_t f = kf(kb, j, k);
#pragma unroll
                    for (int m = 0; m < NQ; ++m)
#pragma unroll
                        for (int p = 0; p < P; ++p) s[kb][m] = mma(f, q[m][j][k][p], s[kb][m]);
                }
            }
        }
        const bool edge = j0 + T - 1 > w0 || (j0 < wlast && j0 + T > sinks);
        const float vexp = (float)ve, vback = power(-ve);
        half8_t w[NQ][2][PW];
#pragma unroll
        for (int m = 0; m < NQ; ++m) {
            // Scores in base 2 with the block's vs, less the row's base: the running maximum as it was
            // when a score last passed it by SLACK.
            const float base = mx[m] == -INFINITY ? 0.f : mx[m];
            // (all powers of two at once, and no more than float32 holds: a product of 0 stays 0)
            const float by = fminf(__builtin_amdgcn_ldexpf(scale2, back[m] + ke), 3.402823466e38f);
            const float shift = (BIAS ? slope[m] * (float)(j0 + 16 * g - pos[m]) : 0.f) + (vexp + HEAD - base);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float add = BIAS ? __builtin_fmaf(slope[m], (float)(4 * kb + r), shift) : shift;
                    if constexpr (CAP != UNCAPPED) s[kb][m][r] = __builtin_fmaf(cap2, tanh_of<IO, CAP>(s[kb][m][r] * by), add);
                    else s[kb][m][r] = __builtin_fmaf(s[kb][m][r], by, add);
                }
            if (edge) {
                keep_branch();
                const int j = j0 + 16 * g;
#pragma unroll
                for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = j + 4 * kb + r;   // (no short circuits: selects, not branches)
                        const bool hidden = (key > pos[m]) | ((key < lo[m]) & (key >= sinks));
                        s[kb][m][r] = hidden ? -INFINITY : s[kb][m][r];
                    }
            }
            float top = s[0][m][0];
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, s[kb][m][r]);
            const float limit = mx[m] == -INFINITY ? -INFINITY : HEAD + SLACK;
            if (__any(top > limit)) {
                top = gmax(top);
                if (top > limit) {
                    const float now = base + (top - HEAD), f = exp2_hw(mx[m] - now);
                    sum[m] *= f;
#pragma unroll
                    for (int d = 0; d < ND; ++d) o[d][m] *= f;
                    mx[m] = now;
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[kb][m][r] -= top - HEAD;
                }
            }
            float part = 0.f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = exp2_hw(s[kb][m][r]);
                    s[kb][m][r] = e;
                    part += e;
                }
            sum[m] = __builtin_fmaf(part, vback, sum[m]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float x[8] = {s[2 * k][m][0], s[2 * k][m][1], s[2 * k][m][2], s[2 * k][m][3],
                                    s[2 * k + 1][m][0], s[2 * k + 1][m][1], s[2 * k + 1][m][2], s[2 * k + 1][m][3]};
                w[m][k][0] = halves_of(x);
                if constexpr (PW == 2) w[m][k][1] = rest_of(x, w[m][k][0]);
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {   // (values past D repeat the first: a branch would wait for each)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const half8_t f = vf(d, k);
#pragma unroll
                for (int m = 0; m < NQ; ++m)
#pragma unroll
                    for (int p = 0; p < PW; ++p) o[d][m] = mma(f, w[m][k][p], o[d][m]);
            }
        }
    };
    // e4m3 bytes of v behind the sequence's last token may stand for NaN: weight 0 does not hide it
    auto clear = [&](int j0, uint4& u) {
        if (CODE != Code::E4M3 || j0 + T <= n) return;
        keep_branch();
        uint32_t* x = (uint32_t*)&u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int keep = n - j0 - 16 * g - 4 * k;
            x[k] &= keep >= 4 ? ~0u : keep <= 0 ? 0u : (1u << (8 * keep)) - 1;
        }
    };
    auto half = [](const uint4& u, int k) { return k ? halves8<CODE>(u.z, u.w) : halves8<CODE>(u.x, u.y); };

    if constexpr (S::KEYS) {
        for (int u = u0 + wave; u < u1; u += NW) {
            Place then;
            if (u + NW < u1) then = bring(u + NW, next);
            if (here.p >= 0) {
                const int j0 = bl.at(u) * T;
#pragma unroll
                for (int d = 0; d < ND; ++d) clear(j0, now.v[d]);
                block(j0, here, [&](int kb, int j, int k) { return half(now.k[kb][j], k); },
                      [&](int d, int k) { return half(now.v[d], k); });
            }
            now = next;
            here = then;
        }
        // join the waves: their rows' base, sum and o
        float* st = (float*)sh;                  // [wave][2][16]
        float* ow = st + NW * 2 * 16;            // [wave][16 rows][DP]
        const float l = gsum(sum[0]);
        if (g == 0) {
            st[(wave * 2) * 16 + c] = mx[0];
            st[(wave * 2 + 1) * 16 + c] = l;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) *(float4*)(ow + (wave * 16 + c) * DP + 16 * d + 4 * g) = make_float4(o[d][0][0], o[d][0][1], o[d][0][2], o[d][0][3]);
        __syncthreads();
        // wave w writes a quarter of each row's values
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, st[(w * 2) * 16 + c]);
        float f[NW], all = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float x = st[(w * 2) * 16 + c];
            f[w] = x == -INFINITY ? 0.f : exp2_hw(x - top);
            all = __builtin_fmaf(f[w], st[(w * 2 + 1) * 16 + c], all);
        }
        const bool none = empty[0] || all == 0.f;
        const float inv = none ? 0.f : 1.0f / all;
        const float ls = none ? -INFINITY : top - HEAD + __builtin_amdgcn_logf(all);
        if (row[0] >= a.nrow) return;
        const int i = token_of(a, row[0]), h = hk * a.G + row[0] - i * a.G;
        const int64_t at = ((int64_t)split * a.nbh + bh) * a.nrow + row[0];
#pragma unroll
        for (int d = 0; d < DP; d += 16 * NW) {
            const int d0 = d + 16 * wave + 4 * g;
            if (d0 >= a.D) continue;
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 y = *(const float4*)(ow + (w * 16 + c) * DP + d0);
                x += f32x4{y.x, y.y, y.z, y.w} * f[w];
            }
            x = none ? f32x4{0.f, 0.f, 0.f, 0.f} : x * inv;
            if (a.nsplit > 1) *(float4*)(a.part + at * a.D + d0) = make_float4(x[0], x[1], x[2], x[3]);
            else put4<IO>((E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2] + d0, x);
        }
        if (wave == 0 && g == 0) {
            if (a.nsplit > 1) a.part_lse[at] = ls;
            else if (a.lse) a.lse[((int64_t)b * a.H + h) * a.Lq + i] = ls * LN2;
        }
    } else {
        // the block's 8 J runs of 1024 bytes (k: kb J + j, then v: d), dealt to the waves; they lie in LDS in
        // half precision, two runs each, in the order of the operands
        constexpr int RUNS = 8 * J / NW;
        static_assert(8 * J % NW == 0, "whole runs");
        uint4 raw[RUNS];
        auto fetch = [&](int u) {
            const Place p(cc, b, hk, bl.at(u));
            const int64_t at = p.bytes(cc, hk);
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const int f = i * NW + wave, kb = f / J, d = f - 4 * J;
                const int ch = 4 * (f % J) + g;   // values past D read the first
                const uint8_t* src = f < 4 * J ? (const uint8_t*)cc.k + at + (kb * chunks + (ch < chunks ? ch : 0)) * 256
                                               : (const uint8_t*)cc.v + at + ((d < chunks ? d : 0) * 4 + g) * 256;
                raw[i] = *(const uint4*)(src + c * 16);
            }
            return p;
        };
        auto put = [&](int u, uint8_t* to) {
            const int j0 = bl.at(u) * T;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                const int f = i * NW + wave;
                if (f >= 4 * J) clear(j0, raw[i]);
#pragma unroll
                for (int k = 0; k < 2; ++k) *(half8_t*)(to + ((f * 2 + k) * 64 + lane) * 16) = half(raw[i], k);
            }
        };
        Place then;
        if (u0 < u1) {
            here = fetch(u0);
            put(u0, sh);
            if (u0 + 1 < u1) then = fetch(u0 + 1);
        }
        for (int u = u0; u < u1; ++u) {
            const uint8_t* at = sh + ((u - u0) & 1) * STAGE;
            stage_barrier();   // this block is in LDS, and the place of the one before is free
            const int j0 = bl.at(u) * T;
            const Place pl = here;
            if (u + 1 < u1) {
                put(u + 1, sh + ((u - u0 + 1) & 1) * STAGE);
                here = then;
                if (u + 2 < u1) then = fetch(u + 2);
            }
            if (pl.p < 0 || w0 > w1 || j0 > w1 || (j0 + T - 1 < wlo && j0 >= sinks)) continue;
            block(j0, pl,
                  [&](int kb, int j, int k) { return *(const half8_t*)(at + (((kb * J + j) * 2 + k) * 64 + lane) * 16); },
                  [&](int d, int k) { return *(const half8_t*)(at + (((4 * J + d) * 2 + k) * 64 + lane) * 16); });
        }
#pragma unroll
        for (int m = 0; m < NQ; ++m) {
            const float l = gsum(sum[m]);
            if (row[m] >= a.nrow) continue;
            const bool none = empty[m] || l == 0.f;
            const float inv = none ? 0.f : 1.0f / l;
            const float ls = none ? -INFINITY : mx[m] - HEAD + __builtin_amdgcn_logf(l);
            const int i = token_of(a, row[m]), h = hk * a.G + row[m] - i * a.G;
            const int64_t at = ((int64_t)split * a.nbh + bh) * a.nrow + row[m];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int d0 = 16 * d + 4 * g;
                if (d0 >= a.D) continue;
                const f32x4 x = none ? f32x4{0.f, 0.f, 0.f, 0.f} : o[d][m] * inv;
                if (a.nsplit > 1) *(float4*)(a.part + at * a.D + d0) = make_float4(x[0], x[1], x[2], x[3]);
                else put4<IO>((E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2] + d0, x);
            }
            if (g != 0) continue;
            if (a.nsplit > 1) a.part_lse[at] = ls;
            else if (a.lse) a.lse[((int64_t)b * a.H + h) * a.Lq + i] = ls * LN2;
        }
    }
}

// Joins the splits of a row: o = sum_s 2^(lse_s - lse) o_s.  One workgroup a row: thread s weighs split s,
// then COLS threads side by side sum the splits for four values each, 256 / COLS splits at a time.
constexpr int NT = 256;
__device__ __forceinline__ float over_block(float x, float (&sh)[NT / 64], bool max)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const float y = __shfl_xor(x, m);
        x = max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    return max ? fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3])) : (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <class IO, int COLS>
__global__ __launch_bounds__(NT) void cached_join(AttnArgs a)
{
    __shared__ float weight[NT], wave[NT / 64];
    __shared__ f32x4 part[NT];
    const int64_t total = (int64_t)a.nbh * a.nrow, at = blockIdx.x;
    const int t = threadIdx.x, col = t % COLS, d0 = 4 * col;
    const float ls = t < a.nsplit ? a.part_lse[t * total + at] : -INFINITY;
    const float mx = over_block(ls, wave, true);
    const float e = ls == -INFINITY ? 0.f : exp2_hw(ls - mx);
    const float sum = over_block(e, wave, false);
    const bool none = sum == 0.f;   // (a sum of NaN is not empty: the row is NaN)
    weight[t] = none ? 0.f : e / sum;
    __syncthreads();
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    const float* p = a.part + at * a.D + (d0 < a.D ? d0 : 0);
#pragma unroll 4
    for (int s = t / COLS; s < a.nsplit; s += NT / COLS) x += *(const f32x4*)(p + s * total * a.D) * weight[s];
    part[t] = x;
    __syncthreads();
    const int bh = (int)(at / a.nrow), r = (int)(at % a.nrow);
    const int b = bh / a.Hkv, i = r / a.G, h = bh % a.Hkv * a.G + r % a.G;
    if (t < COLS && d0 < a.D) {
#pragma unroll
        for (int k = 1; k < NT / COLS; ++k) x += part[k * COLS + t];
        put4<IO>((typename IO::T*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2] + d0, x);
    }
    if (a.lse && t == 0)
        a.lse[((int64_t)b * a.H + h) * a.Lq + i] = none ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * LN2;
}

// Rows of a workgroup: 16 shared by four waves for the few rows of decoding; else 128, which convert a
// block's codes once for all of them, or 64 where these fill the GPU once (heads up to 64 hold twice the
// workgroups a CU) and 128 would leave half of it empty.  Workgroups of 128 against 64, int8 codes: 16
// heads of 64 on 4, B 3, 1024 tokens over 4096 (384 of 128) 91 and 78 us; 16 on 16, B 8 (1024) 175 and 193;
// heads of 128 on 4, 2048 over 8192 (256) 182 and 173, B 3, 1024 over 4096 (384) 131 and 146; 64 tokens over 4
// caches of 16384 (32, keys split) 59 and 67.
constexpr int FEW = 16;
constexpr int64_t FILL = 512;
int tile_rows(const AttnArgs& a)
{
    if (a.nrow <= FEW) return 16;
    const int64_t w128 = (a.nrow + 127) / 128 * (int64_t)a.nbh, w64 = (a.nrow + 63) / 64 * (int64_t)a.nbh;
    return w128 > (a.D <= 64 ? FILL : FILL / 2) || (a.nrow > 64 && 2 * w64 <= FILL) ? 128 : 64;
}

// Key splits while the rows do not fill the GPU, each of at least SPLIT_MIN keys.  8 caches of up to 65536,
// 4 key heads, one token: 768 workgroups 44.0 us, 512 43.5, 1024 45.5, 1536 44.5; 64 caches of up to 4096 47,
// 48, 46, 47; 4 of up to 10007, 12 heads, 5 tokens, float32: 21, 21, 24, 24.
// Few parts of few rows gain less than the second launch costs, whether the keys or the grid limit them.  One
// sequence, 4 key heads of 64, unsplit and in as many parts as it has 512 keys: 1000 keys 12.1 us and 16.8,
// 2500 (5 parts) 14.3 and 16.8, 3500 (6) 17.9 and 16.9.  B sequences of half to all of T tokens, 4 key heads,
// unsplit and in the parts that the grid has room for (B 47: 5, 48: 4, 64: 3, 96: 2):
//     D x T          B 47           48             64             96
//     64 x 4096      21.5 and 22.8  21.1 and 21.5  25.8 and 28.5  28.8 and 33.6
//     128 x 4096     32.2 and 35.9  32.4 and 37.3  41.0 and 45.6  58.5 and 63.2
//     64 x 8192      35.6 and 33.3  35.5 and 32.5  40.5 and 45.6  54.9 and 60.6
//     128 x 8192     57.6 and 59.2  58.1 and 62.6  79.8 and 81.8  110 and 113
//     64 x 16384     64.5 and 61.1  64.3 and 58.3  79.5 and 79.5  113 and 114
//     128 x 16384    109 and 109    111 and 112    167 and 150    219 and 212
//     64 x 65536     - and 213      241 and 212    342 and 311    410 and 390
//     128 x 65536    - and 387      421 and 420    590 and 545    794 and 766
// (39 sequences of 8192, 5 parts: 34.5 and 29.1, 53.7 and 51.0.)
constexpr int64_t FILL_FEW = 768, SPLIT_MIN = 512;
constexpr int64_t SPLIT_MAX = NT;   // the join weighs one split a thread
constexpr int64_t SPLIT_FROM = 3000;   // keys
int64_t least_room(int64_t keys) { return keys >= 16384 ? 2 : keys >= 8192 ? 5 : 6; }

int splits(const AttnArgs& a, int sinks)
{
    const int bm = tile_rows(a);
    const bool few = a.nrow <= FEW;
    const int64_t wgs = (a.nrow + bm - 1) / bm * (int64_t)a.nbh, fill = few ? FILL_FEW : FILL;
    const int64_t keys = std::min<int64_t>(a.Lk, (int64_t)a.window + sinks + std::min<int64_t>(a.Lq, bm));
    if (wgs <= 0 || 2 * wgs > fill) return 1;
    const int64_t room = (fill + wgs - 1) / wgs;   // parts that the grid has room for
    if (few && (keys < SPLIT_FROM || room < least_room(keys))) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({room, keys / SPLIT_MIN, SPLIT_MAX}));
}

template <class IO, Code CODE, int J, class S>
hipError_t go(AttnArgs a, const CacheArgs& c, int sinks, hipStream_t st)
{
    a.ntile = (a.nrow + S::BM - 1) / S::BM;
    const int64_t blocks = (int64_t)a.ntile * a.nbh * a.nsplit;
    if (!grid_ok(blocks, 64 * S::NW)) return hipErrorInvalidValue;
    return with_options<IO, false>(a, [&](auto cap, auto bias) {
        hipLaunchKernelGGL((cached_attn<IO, CODE, J, decltype(cap)::value, decltype(bias)::value, S>), dim3((unsigned)blocks),
                           dim3(64 * S::NW), 0, st, a, c, sinks);
        return hipGetLastError();
    });
}

template <class IO, Code CODE, int J>
hipError_t shape(const AttnArgs& a, const CacheArgs& c, int sinks, hipStream_t st)
{
    switch (tile_rows(a)) {
    case 16: return go<IO, CODE, J, Shape<1, 4, true>>(a, c, sinks, st);
    case 64: return go<IO, CODE, J, Shape<1, 4, false>>(a, c, sinks, st);
    default: return go<IO, CODE, J, Shape<2, 4, false>>(a, c, sinks, st);
    }
}

template <class IO, Code CODE>
hipError_t run(AttnArgs a, const CacheArgs& c, int sinks, hipStream_t st)
{
    a.nsplit = splits(a, sinks);
    a.part_lse = a.part + (int64_t)a.nsplit * a.nbh * a.nrow * a.D;
    const hipError_t e = a.D <= 64 ? shape<IO, CODE, 1>(a, c, sinks, st) : shape<IO, CODE, 2>(a, c, sinks, st);
    if (e != hipSuccess || a.nsplit == 1) return e;
    const int64_t rows = (int64_t)a.nbh * a.nrow;
    if (!grid_ok(rows, NT)) return hipErrorInvalidValue;
    if (a.D <= 64) hipLaunchKernelGGL((cached_join<IO, 16>), dim3((unsigned)rows), dim3(NT), 0, st, a);
    else hipLaunchKernelGGL((cached_join<IO, 32>), dim3((unsigned)rows), dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

size_t cached_attn_bytes(const AttnArgs& a, int sinks)
{
    const int ns = splits(a, sinks);
    return ns > 1 ? (size_t)ns * a.nbh * a.nrow * (a.D + 1) * sizeof(float) : 0;
}

hipError_t launch_cached_attn(Store s, Code code, const AttnArgs& a, const CacheArgs& c, int sinks, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.part = (float*)ws;
    if (s == Store::F32)
        return code == Code::I8 ? run<f32_io, Code::I8>(x, c, sinks, st) : run<f32_io, Code::E4M3>(x, c, sinks, st);
    return code == Code::I8 ? run<bf16_io, Code::I8>(x, c, sinks, st) : run<bf16_io, Code::E4M3>(x, c, sinks, st);
}

}  // namespace sc
