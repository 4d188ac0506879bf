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

// Eight elements of a row in memory (16-byte aligned).
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

// LDS tiles hold rows of DP elements without padding (asynchronous loads write 1024 contiguous
// bytes a wave); the 16-byte chunk k of row r sits at chunk k ^ (r mod SW), so that the rows that
// lanes read together lie in different banks: SW = 8 for rows of 128 bytes, of which two span the
// banks, 16 for longer ones.
template <class IO, int DP>
constexpr int SW = DP * IO::SIZE > 128 ? 16 : 8;

// A operand: row r0 + c, elements 32 k + 8 g .. + 7.  r0 a multiple of 16.
template <class IO, int DP>
__device__ __forceinline__ Frag<IO> frag_row(const typename IO::T* tile, int r0, int k, int g, int c)
{
    const typename IO::T* row = tile + (r0 + c) * DP;
    const int x = c & (SW<IO, DP> - 1);
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) {
        f.v = *(const uint4*)(row + ((4 * k + g) ^ x) * 8);
    } else {
        f.a = *(const float4*)(row + ((8 * k + 2 * g) ^ x) * 4);
        f.b = *(const float4*)(row + ((8 * k + 2 * g + 1) ^ x) * 4);
    }
    return f;
}

// A operand read transposed: column d0 + c of the tile, rows r0 + 4 g + e and r0 + 16 + 4 g + e.
// r0 a multiple of 32, d0 of 16.
template <class IO, int DP>
__device__ __forceinline__ Frag<IO> frag_tr(const typename IO::T* tile, int r0, int d0, int g, int c)
{
    Frag<IO> f;
    if constexpr (IO::SIZE == 2) {
        // lane c of a 16-lane group addresses row c / 4, columns 4 (c % 4) .. + 3, and receives
        // column c of the group's four rows
        const int r = 4 * g + (c >> 2), k = (d0 / 8 + ((c & 3) >> 1)) ^ (r & (SW<IO, DP> - 1));
        const uint16_t* p = tile + (r0 + r) * DP + 8 * k + 4 * (c & 1);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * DP));
        const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
        f.v = make_uint4(l.x, l.y, h.x, h.y);
    } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 4 * g + e, k = (d0 / 4 + (c >> 2)) ^ (r & (SW<IO, DP> - 1));
            const float* p = tile + (r0 + r) * DP + 4 * k + (c & 3);
            x[e] = p[0];
            x[4 + e] = p[16 * DP];
        }
        f.a = make_float4(x[0], x[1], x[2], x[3]);
        f.b = make_float4(x[4], x[5], x[6], x[7]);
    }
    return f;
}

// A wave's rows, element d on: read without a branch (a column past D reads column 0) so that
// nothing waits for a mask, and cleared later where they are not wanted.
template <class IO>
__device__ __forceinline__ Frag<IO> frag_load(const typename IO::T* row, int d, int D)
{
    return frag_at<IO>(row + (d < D ? d : 0));
}
template <class IO>
__device__ __forceinline__ void frag_keep(Frag<IO>& f, bool on)
{
    if constexpr (IO::SIZE == 2) {
        f.v = on ? f.v : make_uint4(0, 0, 0, 0);
    } else {
        f.a = on ? f.a : make_float4(0, 0, 0, 0);
        f.b = on ? f.b : make_float4(0, 0, 0, 0);
    }
}

// ---- asynchronous loads from memory into LDS: every lane's 16 (or 4) bytes go to consecutive
// places from `lds` on (a wave-uniform byte offset under 64 KB).  No register receives them; a
// wave waits for its own with wait_loads, and a barrier then covers the others'.
__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved: nothing else here uses it
__device__ __forceinline__ void load_lds16(const void* p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const void* p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop
// waits until at most N of the wave's loads are in flight; they end in the order of their issue
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// all of the workgroup's LDS reads are done and the asynchronous loads waited for are visible
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What this wave's lanes wrote to LDS comes before what its lanes read next.  The hardware keeps a
// wave's LDS order by itself; this keeps the compiler's, which need not see that a vector read meets
// another lane's scalar write.
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// B operand from two result blocks (the halves of a 32-row strip), rounded to the storage type:
// bfloat16 weights carry a relative error of up to 2^-8 each, as the values they multiply do.  (The rest
// as a second operand, as the forward pass takes it for few rows, would cost the backward pass of the
// window case 322 us for 283, and 1593 for 1320 at L 8192, 16 heads of 128 on 4.)
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

// What frag_of's rounding left of the values, as a second operand: the two together are off by
// (2^-8)^2.
__device__ __forceinline__ Frag<bf16_io> frag_rest(const f32x4& lo, const f32x4& hi, const Frag<bf16_io>& f)
{
    const uint32_t w[4] = {f.v.x, f.v.y, f.v.z, f.v.w};
    f32x4 a, b;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        a[r] = lo[r] - __uint_as_float(r & 1 ? w[r / 2] & 0xffff0000u : w[r / 2] << 16);
        b[r] = hi[r] - __uint_as_float(r & 1 ? w[2 + r / 2] & 0xffff0000u : w[2 + r / 2] << 16);
    }
    return frag_of<bf16_io>(a, b);
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

// A kernel's form for the call's cap.  tanh(y) as 1 - 2 / (1 + e^2y) is off by up to 4 units of 2^-24
// whatever y, and the cap multiplies that.  With SERIES a polynomial takes over near 0, so that the
// error is relative to tanh(y) everywhere, no more than 9 units.  float32 storage always takes it, and
// so does the forward pass, whose lse is float32 whatever the storage.  The backward pass of 16-bit
// storage does without for caps up to 64: a score is then off by no more than 1.5e-5, which results
// rounded to 2^-8 do not show.  There it costs time and registers: B 8, L 4096, 16 heads of 64, window
// 256: 364 us with it, 331 without; L 8192, 16 heads of 128 on 4: 1606 and 1526.  (The forward pass: 122
// and 116, 470 and 432.)
enum Cap { UNCAPPED, CAPPED, SERIES };
constexpr float SERIES_CAP = 64.f;

// float32 storage, below 1/2: the Taylor series to y^15 (the next term is under 1e-8 of the sum).
// 16-bit storage, y^2 below 0.2: y + y^3 (c0 + c1 y^2 + c2 y^4), c fitted for the least maximum of the
// relative error there (5 units).
template <class IO, Cap CAP>
__device__ __forceinline__ float tanh_of(float y)
{
    const float t = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + exp2_hw(2.0f * LOG2E * y));
    if constexpr (CAP != SERIES) {
        return t;
    } else {
        const float z = y * y;
        float p;
        if constexpr (IO::SIZE == 2) {
            p = __builtin_fmaf(-0.046406733f, z, 0.13248634f);
            p = __builtin_fmaf(p, z, -0.333305836f);
        } else {
            p = -929569.0f / 638512875.0f;
            p = __builtin_fmaf(p, z, 21844.0f / 6081075.0f);
            p = __builtin_fmaf(p, z, -1382.0f / 155925.0f);
            p = __builtin_fmaf(p, z, 62.0f / 2835.0f);
            p = __builtin_fmaf(p, z, -17.0f / 315.0f);
            p = __builtin_fmaf(p, z, 2.0f / 15.0f);
            p = __builtin_fmaf(p, z, -1.0f / 3.0f);
        }
        return z < (IO::SIZE == 2 ? 0.2f : 0.25f) ? __builtin_fmaf(p * z, y, y) : t;
    }
}

// Calls f(Cap, BIAS) as constants for the call's options.
template <class IO, bool BWD, class F>
hipError_t with_options(const AttnArgs& a, F&& f)
{
    using std::integral_constant;
    auto bias = [&](auto cap) { return a.slopes ? f(cap, std::true_type()) : f(cap, std::false_type()); };
    if (!(a.cap > 0.f)) return bias(integral_constant<Cap, UNCAPPED>());
    if constexpr (BWD && IO::SIZE == 2)
        if (a.cap <= SERIES_CAP) return bias(integral_constant<Cap, CAPPED>());
    return bias(integral_constant<Cap, SERIES>());
}

// What a raw product is multiplied by: for tanh's argument, no more than the largest float32 where the
// quotient passes it (a 0 stays 0 and everything else saturates, as it does with the quotient), or for
// the score in base 2.
template <Cap CAP>
__device__ __forceinline__ float score_scale(const AttnArgs& a)
{
    return CAP != UNCAPPED ? fminf(a.scale / a.cap, 3.402823466e38f) : a.scale * LOG2E;
}

// The batch row's length, and a query row's place in it.
__device__ __forceinline__ int seq_len(const AttnArgs& a, int b)
{
    return a.kv_len ? min(max(a.kv_len[b], 0), a.Lk) : a.Lk;
}

// Token of a packed row (its head within the group is the remainder).
__device__ __forceinline__ int token_of(const AttnArgs& a, int row) { return a.G == 1 ? row : row / a.G; }

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
    const int t = token_of(a, r);
    return token_range(a, n, t, token_of(a, min(r + rows, a.nrow) - 1) - t + 1);
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

// Rows of one stage (keys, or tokens of a head) of the workgroups that share one among waves, and
// how many stages of BN rows LDS holds: three (48 KB and less), two in flight while one is used;
// float32 heads of 128 leave room for one, whose loads are not hidden.  All under 64 KB, the reach
// of an asynchronous load's LDS offset.
template <class IO, int DP>
constexpr int stage_rows = IO::SIZE == 2 && DP == 64 ? 64 : 32;
template <class IO, int DP, int BN>
constexpr int stages = 3 * 2 * BN * DP * IO::SIZE <= 48 * 1024 ? 3 : 1;

// A ring of stages, each BN rows of two tensors x and y (k and v, or q and dout) and up to three
// 32-bit values a row.  issue(s, t) starts stage s's loads into place t; rows past the last are
// read from the last.  ready() waits until they are in LDS for the whole workgroup; after it the
// place used before is free.
template <class IO, int DP, int NT, int BN = stage_rows<IO, DP>>
struct Ring {
    using E = typename IO::T;
    static constexpr int NS = stages<IO, DP, BN>, V = 16 / IO::SIZE, CH = DP / V;
    static constexpr int NCH = BN * CH / NT, TILE = BN * DP;   // loads a thread and tensor; elements
    static_assert(BN * CH % NT == 0, "whole rounds of loads");
    static constexpr int RPR = NT / CH;                        // rows of a round of loads
    static constexpr int NCOL = RPR >= SW<IO, DP> ? 1 : SW<IO, DP> / RPR;   // rounds until its row repeats mod SW
    struct Shared {
        E x[NS][TILE], y[NS][TILE];
        uint32_t w[3][NS][64];   // a wave writes 64 of them, whatever BN
    };
    static_assert(sizeof(Shared) <= 64 * 1024, "the reach of an asynchronous load");
    Shared& sh;
    const E *xp, *yp;
    const uint32_t* wp[3];   // null: not wanted
    int64_t xs, ys;          // row strides
    int rows, vfirst = 0;    // vfirst: the first row that has values
    int r0, lane, wave, col[NCOL];

    __device__ __forceinline__ Ring(Shared& s, int n, int D, int64_t xs_, int64_t ys_)
        : sh(s), wp{nullptr, nullptr, nullptr}, xs(xs_), ys(ys_), rows(n), r0(threadIdx.x / CH),
          lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6))
    {
        // this thread's chunk of its row of round i; columns past D take the row's first (they meet
        // zeros of the other operand, or results that are not stored)
#pragma unroll
        for (int i = 0; i < NCOL; ++i) {
            const int d = (((int)threadIdx.x % CH) ^ ((r0 + RPR * i) & (SW<IO, DP> - 1))) * V;
            col[i] = d < D ? d : 0;
        }
    }
    __device__ __forceinline__ void from(const E* x, const E* y)
    {
        xp = x;
        yp = y;
    }
    __device__ __forceinline__ void issue(int s, int t) const
    {
        const int64_t b = s * BN + r0;
        const uint32_t lx = lds_offset(sh.x[t]) + wave * 1024, ly = lds_offset(sh.y[t]) + wave * 1024;
        if ((s + 1) * BN <= rows) {
            const E *x = xp + b * xs, *y = yp + b * ys;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                load_lds16(x + i * RPR * xs + col[i % NCOL], __builtin_amdgcn_readfirstlane(lx + i * (NT * 16)));
                load_lds16(y + i * RPR * ys + col[i % NCOL], __builtin_amdgcn_readfirstlane(ly + i * (NT * 16)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int64_t r = min<int64_t>(b + RPR * i, rows - 1);
                load_lds16(xp + r * xs + col[i % NCOL], __builtin_amdgcn_readfirstlane(lx + i * (NT * 16)));
                load_lds16(yp + r * ys + col[i % NCOL], __builtin_amdgcn_readfirstlane(ly + i * (NT * 16)));
            }
        }
        // every wave brings the whole row of values (the same bytes to the same place)
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (wp[k]) load_lds4(wp[k] + max(min(s * BN + lane % BN, rows - 1), vfirst),
                                 __builtin_amdgcn_readfirstlane(lds_offset(sh.w[k][t])));
    }
    // `more`: the next stage's loads are in flight too and may stay so
    __device__ __forceinline__ void ready(bool more) const
    {
        if (!more) {
            wait_loads<0>();
        } else {
            // values wanted: so many more loads a stage
            const int extra = (wp[0] != nullptr) + (wp[1] != nullptr) + (wp[2] != nullptr);
            if (extra == 0) wait_loads<2 * NCH>();
            else if (extra == 1) wait_loads<2 * NCH + 1>();
            else if (extra == 2) wait_loads<2 * NCH + 2>();
            else wait_loads<2 * NCH + 3>();
        }
        stage_barrier();
    }
    // place t's successor, and the place that ready() has freed
    __device__ __forceinline__ static int after(int t) { return t + 1 == NS ? 0 : t + 1; }
    __device__ __forceinline__ static int freed(int t) { return t ? t - 1 : NS - 1; }
    // a walk over stages first .. end - 1: start(first, end), then step() at each
    __device__ __forceinline__ void start(int first, int end) const
    {
        for (int s = first; s < min(end, first + NS - 1); ++s) issue(s, s - first);
    }
    __device__ __forceinline__ void step(int s, int end, int place) const
    {
        if constexpr (NS == 1) {
            __syncthreads();
            issue(s, 0);
            ready(false);
        } else {
            ready(s + 1 < end);
            if (s + NS - 1 < end) issue(s + NS - 1, freed(place));
        }
    }
    // rows whose bit of `live` is clear become 0 in x and y of place t, whatever memory held
    __device__ __forceinline__ void blank(int t, uint64_t live) const
    {
        for (int q = threadIdx.x; q < BN * CH; q += NT)
            if (!(live >> (q / CH) & 1)) {
                *(uint4*)(sh.x[t] + q * V) = make_uint4(0, 0, 0, 0);
                *(uint4*)(sh.y[t] + q * V) = make_uint4(0, 0, 0, 0);
            }
        __syncthreads();
    }
};

// four consecutive results of a row
template <class IO>
__device__ __forceinline__ void put4(typename IO::T* p, const f32x4& x)
{
    if constexpr (IO::SIZE == 2) *(uint2*)p = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
}

// The smallest and the largest key of the waves' ranges (through LDS, NW of them).
template <int NW>
__device__ __forceinline__ void join_ranges(int4 (&sh)[NW], const RowRange& r, int wave, int lane, int& lo, int& hi)
{
    if (lane == 0) sh[wave] = make_int4(r.lo, r.hi, r.last, r.pos);
    __syncthreads();
    lo = BIG;
    hi = -1;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        lo = min(lo, sh[w].x);
        hi = max(hi, sh[w].y);
    }
}

}  // namespace attn
}  // namespace sc
