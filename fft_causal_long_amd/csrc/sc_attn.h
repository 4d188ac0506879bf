// Building blocks of the attention kernels (gfx950): 16 x 16 matrix products whose second
// operand never leaves registers.
//
// A wave's product D = A B of 16 x 16 blocks with a reduction of 32: lane (g, c) = (lane / 16,
// lane % 16) holds A[c][8 g + e], B[8 g + e][c], e < 8, and receives D[4 g + r][c], r < 4.  The
// reduction index may be permuted as long as A and B agree, so two result blocks D0, D1 (rows
// 4 g + r of a 32-row strip's halves) are, rounded, the B operand of a following product whose
// reduction runs over those 32 rows in the order (4 g + r, 16 + 4 g + r): softmax weights go
// from one product to the next without passing through LDS.  The A operand in that order is
// read transposed from a row-major LDS tile (ds_read_b64_tr_b16 for 16-bit elements).
// float32 storage uses the float32 matrix instruction on the same layout, eight of depth 4.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sc_device.h"
#include "sc_internal.h"

namespace sc {
namespace attn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr int NT = 256;   // threads of a workgroup
constexpr int BIG = 0x7fffffff;

// Eight elements of an operand row.
template <class IO>
struct Frag;
template <>
struct Frag<bf16_io> {
    uint4 v;
};
template <>
struct Frag<f32_io> {
    float4 a, b;
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16_io>& a, const Frag<bf16_io>& b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v),
                                                   __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<f32_io>& a, const Frag<f32_io>& b, f32x4 c)
{
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.x, b.a.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.y, b.a.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.z, b.a.z, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a.w, b.a.w, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.x, b.b.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.y, b.b.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.z, b.b.z, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a.b.w, b.b.w, c, 0, 0, 0);
}

// LDS tile row pitch in elements for rows of DP: 16 bytes of padding, so that 16 lanes reading
// 16 bytes each of 16 rows touch every bank once.
template <class IO, int DP>
constexpr int pitch = DP + 16 / IO::SIZE;

// Row r of a tile (or of memory), elements at p[0..7] (16-byte aligned).
template <class IO>
__device__ __forceinline__ Frag<IO> frag_at(const typename IO::T* p)
{
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) {
        f.v = *(const uint4*)p;
    } else {
        f.a = *(const float4*)p;
        f.b = *(const float4*)(p + 4);
    }
    return f;
}

template <class IO>
__device__ __forceinline__ Frag<IO> frag_zero()
{
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) f.v = make_uint4(0, 0, 0, 0);
    else f.a = f.b = make_float4(0, 0, 0, 0);
    return f;
}

// A operand read transposed: column d0 + c of the tile, rows r0 + 4 g + e and r0 + 16 + 4 g + e.
template <class IO, int P>
__device__ __forceinline__ Frag<IO> frag_tr(const typename IO::T* tile, int r0, int d0, int g, int c)
{
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) {
        // lane c of a 16-lane group addresses row c / 4, columns 4 (c % 4) .. + 3, and receives
        // column c of the group's four rows
        const uint16_t* p = tile + (r0 + 4 * g + (c >> 2)) * P + d0 + 4 * (c & 3);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * P));
        const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
        f.v = make_uint4(l.x, l.y, h.x, h.y);
    } else {
        const float* p = tile + (r0 + 4 * g) * P + d0 + c;
        f.a = make_float4(p[0], p[P], p[2 * P], p[3 * P]);
        p += 16 * P;
        f.b = make_float4(p[0], p[P], p[2 * P], p[3 * P]);
    }
    return f;
}

// B operand from two result blocks (the halves of a 32-row strip), rounded to the storage type:
// bfloat16 weights carry a relative error of up to 2^-8 each, as the values they multiply do.
template <class IO>
__device__ __forceinline__ Frag<IO> frag_of(const f32x4& lo, const f32x4& hi)
{
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) {
        f.v = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                         pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
    } else {
        f.a = make_float4(lo[0], lo[1], lo[2], lo[3]);
        f.b = make_float4(hi[0], hi[1], hi[2], hi[3]);
    }
    return f;
}

// sum / max over the four lanes (one per g) that share c
__device__ __forceinline__ float gsum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float gmax(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
// sum over N neighbouring lanes (8, 16 or 32, aligned), by lane permutations in the add itself up
// to 16: quad swaps, then mirrors of 8 and of 16
template <int N>
__device__ __forceinline__ float lane_sum(float v)
{
    auto swapped = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    using std::integral_constant;
    v += swapped(v, integral_constant<int, 0xb1>());    // quad_perm 1, 0, 3, 2
    v += swapped(v, integral_constant<int, 0x4e>());    // quad_perm 2, 3, 0, 1
    v += swapped(v, integral_constant<int, 0x141>());   // row_half_mirror
    if constexpr (N >= 16) v += swapped(v, integral_constant<int, 0x140>());   // row_mirror
    if constexpr (N >= 32) v += __shfl_xor(v, 16);
    return v;
}
__device__ __forceinline__ int wave_min(int v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = min(v, __shfl_xor(v, m));
    return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int wave_max(int v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, __shfl_xor(v, m));
    return __builtin_amdgcn_readfirstlane(v);
}

// Inside a rarely taken block: keeps it a branch.  The compiler would otherwise compute the
// block's selects on every pass (the masks of attn_fwd: 100 of 330 vector instructions a tile).
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// tanh(y).  1 - 2 / (1 + e^2y) is off by about 1e-7 whatever y: below the rounding of bfloat16
// weights even times a cap of 100, so 16-bit storage takes it for every y.  float32 storage
// wants the relative error small too: below 1/2 the odd Taylor series to y^15 (the next term is
// under 1e-8 of the sum).
template <class IO>
__device__ __forceinline__ float tanh_of(float y)
{
    const float t = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + exp2_hw(2.0f * LOG2E * y));
    if constexpr (IO::SIZE == 2) {
        return t;
    } else {
        const float z = y * y;
        float p = -929569.0f / 638512875.0f;
        p = __builtin_fmaf(p, z, 21844.0f / 6081075.0f);
        p = __builtin_fmaf(p, z, -1382.0f / 155925.0f);
        p = __builtin_fmaf(p, z, 62.0f / 2835.0f);
        p = __builtin_fmaf(p, z, -17.0f / 315.0f);
        p = __builtin_fmaf(p, z, 2.0f / 15.0f);
        p = __builtin_fmaf(p, z, -1.0f / 3.0f);
        return z < 0.25f ? __builtin_fmaf(p * z, y, y) : t;
    }
}

// The batch row's length, and a query row's place in it.
__device__ __forceinline__ int seq_len(const AttnArgs& a, int b)
{
    return a.kv_len ? min(max(a.kv_len[b], 0), a.Lk) : a.Lk;
}

// First key that position p may see: past p if its row is empty (p outside the sequence, or its
// document starts after it).
__device__ __forceinline__ int first_key(const AttnArgs& a, int b, int p, int n)
{
    if (p < 0 || p >= n) return BIG;
    int lo = max(0, p - a.window + 1);
    if (a.doc) lo = max(lo, a.doc[(int64_t)b * a.Lk + p]);
    return lo > p ? BIG : lo;
}

// Key j belongs to the sequence and is not padding (its own row is not empty).
__device__ __forceinline__ bool key_live(const AttnArgs& a, int b, int j, int n)
{
    return j < n && (!a.doc || a.doc[(int64_t)b * a.Lk + j] <= j);
}

// What a strip of packed rows sees: its lowest and highest key, the highest first key of a row
// and the lowest position (a key tile at or above `last` and at or below `pos` needs no mask).
// A strip of empty rows has lo = BIG, hi = -1.
struct RowRange {
    int lo, hi, last, pos;
};

// Without documents it follows from the first and the last row: tokens t .. t + count - 1.
__device__ __forceinline__ RowRange token_range(const AttnArgs& a, int n, int t, int count)
{
    const int off = n - a.Lq, p1 = off + min(t + count, a.Lq) - 1;
    if (t >= a.Lq || p1 < 0) return {BIG, -1, 0, BIG};
    const int p0 = max(off + t, 0);
    return {max(0, p0 - a.window + 1), p1, max(0, p1 - a.window + 1), p0};
}
// Packed rows r .. r + rows - 1.
__device__ __forceinline__ RowRange packed_range(const AttnArgs& a, int n, int r, int rows)
{
    if (r >= a.nrow) return {BIG, -1, 0, BIG};
    const int t = r / a.G;
    return token_range(a, n, t, (min(r + rows, a.nrow) - 1) / a.G - t + 1);
}

// The range of a wave's strip from its lanes' rows (lo = BIG: empty).
template <int NR>
__device__ __forceinline__ RowRange lanes_range(const int (&lo)[NR], const int (&pos)[NR])
{
    RowRange x = {BIG, -1, 0, BIG};
#pragma unroll
    for (int m = 0; m < NR; ++m)
        if (lo[m] != BIG) {
            x.lo = min(x.lo, lo[m]);
            x.hi = max(x.hi, pos[m]);
            x.last = max(x.last, lo[m]);
            x.pos = min(x.pos, pos[m]);
        }
    return {wave_min(x.lo), wave_max(x.hi), wave_max(x.last), wave_min(x.pos)};
}

// The key tiles a workgroup walks: 64 keys of k and v, fetched into registers one tile ahead and
// put into LDS rows of pitch<IO, DP>.  Keys past the sequence and padding read as 0, whatever the
// memory holds.
template <class IO, int DP>
struct KeyTiles {
    using E = typename IO::T;
    static constexpr int BN = 64, V = 16 / IO::SIZE, CH = DP / V, NCH = BN * CH / NT, P = pitch<IO, DP>;
    const AttnArgs& a;
    const int32_t* doc;
    const E *kp, *vp;
    int n, r0, d0, lane;   // this thread's pieces: rows r0 + NT / CH i, columns d0 .. d0 + V - 1
    bool din;
    uint4 rk[NCH], rv[NCH];
    int rdoc = 0;

    __device__ __forceinline__ KeyTiles(const AttnArgs& args, int b, int hk, int len, int tid)
        : a(args), doc(args.doc ? args.doc + (int64_t)b * args.Lk : nullptr), n(len), r0(tid / CH),
          d0(tid % CH * V), lane(tid & 63), din(d0 < args.D)
    {
        kp = (const E*)a.k + b * a.ks[0] + hk * a.ks[2] + (din ? d0 : 0);
        vp = (const E*)a.v + b * a.vs[0] + hk * a.vs[2] + (din ? d0 : 0);
    }
    // only where some row sees a key, so n > 0; nothing here waits for a load
    __device__ __forceinline__ void fetch(int j0)
    {
        if (j0 + BN <= n) {
            const E *k = kp + (int64_t)(j0 + r0) * a.ks[1], *v = vp + (int64_t)(j0 + r0) * a.vs[1];
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                rk[i] = *(const uint4*)(k + (int64_t)(NT / CH * i) * a.ks[1]);
                rv[i] = *(const uint4*)(v + (int64_t)(NT / CH * i) * a.vs[1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int64_t j = min(j0 + r0 + NT / CH * i, n - 1);
                rk[i] = *(const uint4*)(kp + j * a.ks[1]);
                rv[i] = *(const uint4*)(vp + j * a.vs[1]);
            }
        }
        if (doc) rdoc = doc[min(j0 + lane, n - 1)];
    }
    // returns which keys of the tile exist and are not padding, bit j - j0
    __device__ __forceinline__ uint64_t put(E* kt, E* vt, int j0)
    {
        const uint64_t live = __ballot(j0 + lane < n && (!doc || rdoc <= j0 + lane));
        if (live == ~0ull && DP == a.D) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int at = (r0 + NT / CH * i) * P + d0;
                *(uint4*)(kt + at) = rk[i];
                *(uint4*)(vt + at) = rv[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int r = r0 + NT / CH * i, at = r * P + d0;
                const bool on = din && live >> r & 1;
                *(uint4*)(kt + at) = on ? rk[i] : make_uint4(0, 0, 0, 0);
                *(uint4*)(vt + at) = on ? rv[i] : make_uint4(0, 0, 0, 0);
            }
        }
        // keys past the sequence lie past every position: no mask of their own
        return doc ? live : ~0ull;
    }
};

// four consecutive results of a row
template <class IO>
__device__ __forceinline__ void put4(typename IO::T* p, const f32x4& x)
{
    if constexpr (IO::SIZE == 2) *(uint2*)p = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
}

}  // namespace attn
}  // namespace sc
