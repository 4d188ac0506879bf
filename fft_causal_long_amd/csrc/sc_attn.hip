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
// once for all of them.  A workgroup takes 16, 64 or 128 rows (tile_rows), 16 or 32 a wave, and
// walks tiles of 64 keys (32 for float32, heads over 64 and single waves) that asynchronous loads
// bring into a ring of three LDS places, two tiles ahead.  Scores are made transposed (keys x
// rows): a lane then holds a quarter of the tile's keys of one row per 16-row block, the row's
// statistics are the lane's own but for two shuffles, and the weights are the B operand of the
// second product as they stand (sc_attn.h).  A wave skips tiles none of its rows sees and masks
// only tiles that an edge crosses.  When the rows do not fill the GPU the keys are split over
// workgroups, whose parts attn_join adds.
//
// Measured (MI355X; a large copy moves 5.4 TB/s, reads alone 6.3, a bfloat16 product of 8192^3
// reaches 1135 TFLOP/s), bfloat16:
//  * B 8, L 4096, 16 heads of 64, window 256, bias: 104 us, 2.6 TB/s of q, k, v, o read and written
//    once, where 51 us would be a copy's rate.  The loads and stores alone take 65 us; the vector
//    instructions of the scores (scale, bias, edges, maximum, exponential, sum, rounding: 13 each
//    with what a wave spends outside the tiles) keep a SIMD busy 60% of the time, the matrix
//    products 16%.
//  * B 1, L 8192, 16 heads of 128 on 4 key heads, no window: 331 us, 830 TFLOP/s of the products
//    that the mask leaves: bound by the same vector instructions beside the products.
//  * 8 sequences over ragged caches of up to 65536, one query, 16 heads of 64 on 4 key heads: 88 us,
//    4.8 TB/s, 5 us of it the join: bound by the cache's bytes.
// 32 rows a wave and 4 waves against 16 x 8: 104 and 107 us, 335 and 356; 32 x 8: 161 (fewer
// workgroups a CU, and they wait for each other's barriers).  float32 takes 16 a wave: the operands
// are twice as large.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_attn.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace attn;

constexpr int NT = 256;           // threads of attn_join
constexpr float SLACK = 8.f;      // a row's base may lag its maximum by this (base 2)

// A workgroup's shape: NQ 16-row blocks a wave, NW waves, tiles of BN keys.
template <int NQ_, int NW_, int BN_>
struct Shape {
    static constexpr int NQ = NQ_, NW = NW_, BN = BN_, WM = 16 * NQ, BM = NW * WM;   // rows of a wave, of a workgroup
};

// Waves a SIMD the kernel is compiled for: as many as its registers allow without spills.
template <class IO, int DP, class S>
constexpr int fwd_occupancy = S::NW == 1 ? 1 : IO::SIZE == 2 && DP == 64 ? 3 : 2;

// Weights of bfloat16 storage as the sum of two bfloat16 values, which takes the second product twice:
// for the few rows of decoding, where the cache's bytes leave the arithmetic time, so that o is off by
// its own rounding only (0.0017 of it; 0.0024 with weights of one).  8 sequences over 65536 keys each,
// 16 heads of 64 on 4: 99.4 us with one, 99.8 with two; 64 sequences over 2048 keys, 16 heads of 128 on
// 2: 35.1 and 36.4.  More rows take one: B 8, L 4096, 16 heads of 64, window 256, no bias: 91 us, 108
// with two; L 8192 as above 332 and 421.
template <class IO, class S>
constexpr bool two_weights = IO::SIZE == 2 && S::NW == 1;

template <class IO, int DP, Cap CAP, bool BIAS, class S>
__global__ __launch_bounds__((64 * S::NW), (fwd_occupancy<IO, DP, S>)) void attn_fwd(AttnArgs a)
{
    using E = typename IO::T;
    constexpr int NQ = S::NQ, NW = S::NW, WM = S::WM, BM = S::BM, BN = S::BN;
    using R = Ring<IO, DP, 64 * NW, BN>;
    constexpr int KK = DP / 32, ND = DP / 16, KB = BN / 16;   // 16-key blocks of a tile
    constexpr bool TWO = two_weights<IO, S>;
    __shared__ __attribute__((aligned(1024))) typename R::Shared sh;
    __shared__ int4 range[NW];

    uint32_t id = blockIdx.x;
    const int bh = (int)(id % (uint32_t)a.nbh);
    id /= (uint32_t)a.nbh;
    const int split = (int)(id % (uint32_t)a.nsplit);
    // the last rows see most keys: first
    const int tile = a.ntile - 1 - (int)(id / (uint32_t)a.nsplit);
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = seq_len(a, b);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform, so that branches on it are

    // this lane's rows
    int row[NQ], pos[NQ], lo[NQ];
    bool empty[NQ];
    Frag<IO> q[NQ][KK];
    float slope[NQ];
    const int rw = tile * BM + wave * WM;   // the wave's first row
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        row[m] = rw + 16 * m + c;
        const bool in = row[m] < a.nrow;
        const int i = in ? token_of(a, row[m]) : 0, h = in ? hk * a.G + row[m] - i * a.G : hk * a.G;
        pos[m] = n - a.Lq + i;
        lo[m] = in ? first_key(a, b, pos[m], n) : BIG;
        empty[m] = lo[m] == BIG;
        slope[m] = BIAS ? a.slopes[h] * LOG2E : 0.f;
        const E* qp = (const E*)a.q + b * a.qs[0] + (int64_t)i * a.qs[1] + h * a.qs[2];
#pragma unroll
        for (int k = 0; k < KK; ++k) {
            q[m][k] = frag_load<IO>(qp, 32 * k + 8 * g, a.D);
        }
    }
    const RowRange rr = a.doc ? lanes_range(lo, pos) : packed_range(a, n, rw, WM);
    int klo = rr.lo, khi = rr.hi;
    if (a.doc) {
        join_ranges<NW>(range, rr, wave, lane, klo, khi);
    } else {
        const RowRange all = packed_range(a, n, tile * BM, BM);
        klo = all.lo;
        khi = all.hi;
    }
    klo = __builtin_amdgcn_readfirstlane(klo);
    khi = __builtin_amdgcn_readfirstlane(khi);
#pragma unroll
    for (int m = 0; m < NQ; ++m)
        if (empty[m]) {
            // an empty row takes part with q = 0 and nothing masked; its result is dropped
            lo[m] = 0;
            pos[m] = BIG;
        }
    int t0 = khi < 0 ? 0 : klo / BN, t1 = khi < 0 ? 0 : khi / BN + 1;
    if (a.nsplit > 1) {
        const int per = (t1 - t0 + a.nsplit - 1) / a.nsplit;
        t0 = min(t1, t0 + split * per);
        t1 = min(t1, t0 + per);
    }

    const float scale2 = score_scale<CAP>(a), cap2 = a.cap * LOG2E;
    f32x4 o[ND][NQ];
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        mx[m] = -INFINITY;
        sum[m] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    R ring(sh, n, a.D, a.ks[1], a.vs[1]);
    ring.from((const E*)a.k + b * a.ks[0] + hk * a.ks[2], (const E*)a.v + b * a.vs[0] + hk * a.vs[2]);
    if (a.doc) ring.wp[0] = (const uint32_t*)a.doc + (int64_t)b * a.Lk;
    ring.start(t0, t1);
#pragma unroll
    for (int m = 0; m < NQ; ++m)
#pragma unroll
        for (int k = 0; k < KK; ++k) frag_keep<IO>(q[m][k], !empty[m] && 32 * k + 8 * g < a.D);
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
        if (j0 > rr.hi || j0 + BN - 1 < rr.lo) continue;   // no row of this wave sees it

        // scores, keys x rows
        f32x4 s[KB][NQ];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int m = 0; m < NQ; ++m) s[kb][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                const Frag<IO> f = frag_row<IO, DP>(Kt, 16 * kb, k, g, c);
#pragma unroll
                for (int m = 0; m < NQ; ++m) s[kb][m] = mma(f, q[m][k], s[kb][m]);
            }
        }
        const bool edge = j0 < rr.last || j0 + BN - 1 > rr.pos;
        Frag<IO> w[KB / 2][NQ], rest[KB / 2][NQ];
#pragma unroll
        for (int m = 0; m < NQ; ++m) {
            // scores in base 2, less the row's base: the running maximum as it was when a score
            // last passed it by 2^SLACK.  Weights then reach 2^SLACK, which float32 sums and
            // either storage type hold as well as 1, and the accumulators are rescaled a few
            // times a row instead of whenever the maximum moves.
            const float base = mx[m] == -INFINITY ? 0.f : mx[m];
            const float shift = BIAS ? slope[m] * (float)(j0 + 4 * g - pos[m]) - base : -base;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float add = BIAS ? __builtin_fmaf(slope[m], (float)(16 * kb + r), shift) : shift;
                    if constexpr (CAP != UNCAPPED) s[kb][m][r] = __builtin_fmaf(cap2, tanh_of<IO, CAP>(s[kb][m][r] * scale2), add);
                    else s[kb][m][r] = __builtin_fmaf(s[kb][m][r], scale2, add);
                }
            if (edge) {
                keep_branch();
                const int first = lo[m] - j0 - 4 * g;
                const uint32_t span = (uint32_t)(pos[m] - lo[m]);   // keys the row sees, less 1
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if ((uint32_t)(16 * kb + r - first) > span) s[kb][m][r] = -INFINITY;
            }
            if (live != ~0ull) {
                keep_branch();
                const uint64_t mine = live >> (4 * g);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!(mine >> (16 * kb + r) & 1)) s[kb][m][r] = -INFINITY;
            }
            float top = s[0][m][0];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, s[kb][m][r]);
            if (__any(top > (mx[m] == -INFINITY ? -INFINITY : SLACK))) {
                top = gmax(top);
                if (top > (mx[m] == -INFINITY ? -INFINITY : SLACK)) {
                    const float now = base + top, f = exp2_hw(mx[m] - now);
                    sum[m] *= f;
#pragma unroll
                    for (int d = 0; d < ND; ++d) o[d][m] *= f;
                    mx[m] = now;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[kb][m][r] -= top;
                }
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = exp2_hw(s[kb][m][r]);
                    s[kb][m][r] = e;
                    sum[m] += e;
                }
#pragma unroll
            for (int hf = 0; hf < KB / 2; ++hf) {
                w[hf][m] = frag_of<IO>(s[2 * hf][m], s[2 * hf + 1][m]);
                if constexpr (TWO) rest[hf][m] = frag_rest(s[2 * hf][m], s[2 * hf + 1][m], w[hf][m]);
            }
        }
        // o^T += v^T w
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int hf = 0; hf < KB / 2; ++hf) {
                const Frag<IO> f = frag_tr<IO, DP>(Vt, 32 * hf, 16 * d, g, c);
#pragma unroll
                for (int m = 0; m < NQ; ++m) {
                    o[d][m] = mma(f, w[hf][m], o[d][m]);
                    if constexpr (TWO) o[d][m] = mma(f, rest[hf][m], o[d][m]);
                }
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
        const int i = token_of(a, row[m]), h = hk * a.G + row[m] - i * a.G;
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
            put4<IO>(op + d0, none ? f32x4{0.f, 0.f, 0.f, 0.f} : o[d][m] * inv);
        }
        if (a.lse && g == 0) a.lse[((int64_t)b * a.H + h) * a.Lq + i] = ls * LN2;
    }
}

// Joins the splits of a row: o = sum_s 2^(lse_s - lse) o_s.  One workgroup per row: lane s weighs
// split s (at most 64), then each wave sums a quarter of the splits for 64 columns at a time.
template <class IO>
__global__ __launch_bounds__(NT) void attn_join(AttnArgs a)
{
    using E = typename IO::T;
    __shared__ float weight[64], sum4[4][64];
    const int64_t total = (int64_t)a.nbh * a.nrow, at = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float ls = lane < a.nsplit ? a.part_lse[lane * total + at] : -INFINITY;
    float mx = ls;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
    const float e = ls == -INFINITY ? 0.f : exp2_hw(ls - mx);
    float sum = e;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    const bool none = sum == 0.f;   // (a sum of NaN is not empty: the row is NaN)
    if (wave == 0) weight[lane] = none ? 0.f : e / sum;
    const int bh = (int)(at / a.nrow), r = (int)(at % a.nrow);
    const int b = bh / a.Hkv, i = r / a.G, h = bh % a.Hkv * a.G + r % a.G;
    E* op = (E*)a.o + b * a.os[0] + (int64_t)i * a.os[1] + h * a.os[2];
    for (int d0 = 0; d0 < a.D; d0 += 64) {
        __syncthreads();
        const float* p = a.part + at * a.D + min(d0 + lane, a.D - 1);
        float x = 0.f;
#pragma unroll 4
        for (int s = wave; s < a.nsplit; s += 4) x = __builtin_fmaf(weight[s], p[s * total * a.D], x);
        sum4[wave][lane] = x;
        __syncthreads();
        if (wave == 0 && d0 + lane < a.D)
            IO::store(op, d0 + lane, (sum4[0][lane] + sum4[1][lane]) + (sum4[2][lane] + sum4[3][lane]));
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[((int64_t)b * a.H + h) * a.Lq + i] = none ? -INFINITY : (mx + __builtin_amdgcn_logf(sum)) * LN2;
}

// Rows of a workgroup: 16 (one wave) for the few rows of decoding, where waves without rows would
// only share the loads (8 sequences over caches of 65536 keys, 4 key heads of 64: 88.1 us, 90.9
// with 64 rows); 64 where 128 would give no more than 512 workgroups, two a CU (12 heads of 64,
// L 1024: 384 workgroups 23.0 us, 768 of half the rows 17.8; 16 heads of 128, 4 key heads, L 4096:
// 512 135 us, 1024 112; but 768 29.0 us, 1536 30.5 and 4096 104 us, 8192 111).
constexpr int FEW = 16;
constexpr int64_t TWO_A_CU = 512;
int tile_rows(const AttnArgs& a)
{
    if (a.nrow <= FEW) return 16;
    return (a.nrow + 127) / 128 * (int64_t)a.nbh <= TWO_A_CU ? 64 : 128;
}

// Key splits: as many as fill the GPU when the rows alone do not, each of at least SPLIT_MIN keys.
// The caches above take 88 us in 1280 parts (40 a sequence and key head), 1544 us unsplit; 768 and
// 2048 parts are 3% and more slower.  Four sequences of 16384 keys, 2 key heads: 18.7 and 330 us.
constexpr int64_t FILL = 512, FILL_FEW = 1280;
constexpr int64_t SPLIT_MIN = 256;
constexpr int64_t SPLIT_MAX = 64;   // attn_join weighs one split a lane

int splits(const AttnArgs& a)
{
    const int bm = tile_rows(a);
    const int64_t wgs = (a.nrow + bm - 1) / bm * (int64_t)a.nbh, fill = a.nrow <= FEW ? FILL_FEW : FILL;
    const int64_t keys = std::min<int64_t>(a.Lk, (int64_t)a.window + std::min<int64_t>(a.Lq, bm));
    if (wgs <= 0 || 2 * wgs > fill) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(fill + wgs - 1) / wgs, keys / SPLIT_MIN, SPLIT_MAX}));
}

template <class IO, int DP, Cap CAP, bool BIAS, class S>
hipError_t go(const AttnArgs& a, hipStream_t st)
{
    const int64_t blocks = (int64_t)a.ntile * a.nbh * a.nsplit;
    if (!grid_ok(blocks, 64 * S::NW)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_fwd<IO, DP, CAP, BIAS, S>), dim3((unsigned)blocks), dim3(64 * S::NW), 0, st, a);
    return hipGetLastError();
}

template <class IO, int DP, class S>
hipError_t pick(AttnArgs a, hipStream_t st)
{
    a.ntile = (a.nrow + S::BM - 1) / S::BM;
    return with_options<IO, false>(a, [&](auto cap, auto bias) {
        return go<IO, DP, decltype(cap)::value, decltype(bias)::value, S>(a, st);
    });
}

template <class IO, int DP>
hipError_t shape(const AttnArgs& a, hipStream_t st)
{
    constexpr int BN = stage_rows<IO, DP>;
    switch (tile_rows(a)) {
    case 16: return pick<IO, DP, Shape<1, 1, 32>>(a, st);
    case 64: return pick<IO, DP, Shape<1, 4, BN>>(a, st);
    default: break;
    }
    // float32: one block a wave (the score tile and its operands take twice the registers)
    constexpr int NQ = IO::SIZE == 4 ? 1 : 2;
    return pick<IO, DP, Shape<NQ, 8 / NQ, BN>>(a, st);
}

template <class IO>
hipError_t run(AttnArgs a, hipStream_t st)
{
    a.nsplit = splits(a);
    a.part_lse = a.part + (int64_t)a.nsplit * a.nbh * a.nrow * a.D;
    const hipError_t e = a.D <= 64 ? shape<IO, 64>(a, st) : shape<IO, 128>(a, st);
    if (e != hipSuccess || a.nsplit == 1) return e;
    const int64_t rows = (int64_t)a.nbh * a.nrow;
    if (!grid_ok(rows, NT)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_join<IO>), dim3((unsigned)rows), dim3(NT), 0, st, a);
    return hipGetLastError();
}

}  // namespace

size_t attn_fwd_bytes(const AttnArgs& a)
{
    const int ns = splits(a);
    return ns > 1 ? (size_t)ns * a.nbh * a.nrow * (a.D + 1) * sizeof(float) : 0;
}

hipError_t launch_attn(Store s, const AttnArgs& a, void* ws, hipStream_t st)
{
    AttnArgs x = a;
    x.part = (float*)ws;
    return s == Store::F32 ? run<f32_io>(x, st) : run<bf16_io>(x, st);
}

}  // namespace sc
