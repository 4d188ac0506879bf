// The 8-bit cache: 64 tokens of a key head are a block, its k and its v one scale each (gfx950).
//
// A value is code * 2^e.  e is the smallest exponent, in -60 .. 60, that brings the block's largest
// magnitude to 127 (int8 codes, nearest even) or 448 (e4m3, the format's own rounding).  With a power
// of two the division is exact, so a code is the value rounded once in any arithmetic, a growing scale
// costs e4m3 codes nothing until they fall below its normal range, and a scale taken into an exponent
// costs nothing.  What it gives away is the step of int8 codes, up to twice that of amax / 127.
//
// The bytes of a block lie in the order in which the lanes of a matrix product take them, so that a
// wave reads 1024 consecutive bytes, 16 a lane, and needs no exchange.  A 16 x 16 product gives lane
// (g, c) the rows 4 g + r, r < 4.  With key 16 (i / 4) + 4 kb + i % 4 as row i of score block kb, lane
// group g ends up with the weights of keys 16 g .. 16 g + 15, the operand of the second product:
//   k: [kb < 4][16-value chunk of D][i < 16][16 values],  v: [16-value chunk of D][t / 16][d % 16][t % 16]
// int8 codes are held with 128 added: a half-precision value 1024 + byte is then one byte permutation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sc_device.h"
#include "sc_internal.h"

namespace sc {
namespace cache {

constexpr int T = 64;
constexpr int E_LOW = -60, E_HIGH = 60;   // products of scales with sums stay far inside float32

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

// A row's block `blk` in the pool; -1 where there is none (past the row's blocks, or a table entry
// outside the pool).
__device__ __forceinline__ int block_of(const CacheArgs& c, int b, int blk)
{
    if ((uint32_t)blk >= (uint32_t)c.N) return -1;
    if (!c.table) return b * c.N + blk;
    const int p = c.table[(int64_t)b * c.N + blk];
    return (uint32_t)p < (uint32_t)c.P ? p : -1;
}

// Byte of token t's values 16 ch .. 16 ch + 15 in a block of k, and of value d of tokens
// 16 tc .. 16 tc + 15 in one of v (D / 16 = chunks).
__device__ __forceinline__ int k_at(int t, int ch, int chunks)
{
    return ((((t >> 2) & 3) * chunks + ch) * 16 + ((t >> 4) << 2) + (t & 3)) * 16;
}
__device__ __forceinline__ int v_at(int d, int tc) { return (((d >> 4) * 4 + tc) * 16 + (d & 15)) * 16; }

// The exponent for a largest magnitude (0 and subnormals: the lowest).
template <Code CODE>
__device__ __forceinline__ int exponent_of(float top)
{
    const uint32_t u = __float_as_uint(top);
    const int x = (int)(u >> 23) - 127, m = (int)(u & 0x7fffff);
    // 127 = 0x1.fc p6, 448 = 0x1.c p8
    const int e = CODE == Code::I8 ? x - 6 + (m > 0x7e0000) : x - 8 + (m > 0x600000);
    return min(max(e, E_LOW), E_HIGH);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The exponent of a stored scale (whatever memory holds is brought into range).
__device__ __forceinline__ int exponent_of_scale(float scale)
{
    return min(max((int)(__float_as_uint(scale) >> 23 & 255) - 127, E_LOW), E_HIGH);
}

// A magnitude for the largest: infinities and NaN do not count.
__device__ __forceinline__ float magnitude(float x)
{
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

// Four codes of values already divided by the scale.  Infinities take the largest code; NaN is NaN in
// e4m3 and 0 in int8.
template <Code CODE>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (CODE == Code::I8) {
        auto one = [](float x) -> uint32_t {
            const float y = x == x ? fminf(fmaxf(x, -127.f), 127.f) : 0.f;
            return (uint32_t)((int)__builtin_rintf(y) + 128);
        };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    } else {
        auto one = [](float x) { return x == x ? fminf(fmaxf(x, -448.f), 448.f) : x; };
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(one(a), one(b), 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(one(c), one(d), w, true);
    }
}

// Four codes as float32.
template <Code CODE>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4])
{
    if constexpr (CODE == Code::I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)((int)(w >> (8 * i) & 255) - 128);
    } else {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        x[0] = lo[0];
        x[1] = lo[1];
        x[2] = hi[0];
        x[3] = hi[1];
    }
}

// Four codes in half precision (exact: integers up to 127, e4m3 up to 448 and down to 2^-9).
template <Code CODE>
__device__ __forceinline__ void halves4(uint32_t w, half2_t& lo, half2_t& hi)
{
    if constexpr (CODE == Code::I8) {
        const half2_t off = {(_Float16)1152.f, (_Float16)1152.f};
        lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
        hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
    } else {
        lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
    }
}
template <Code CODE>
__device__ __forceinline__ half8_t halves8(uint32_t a, uint32_t b)
{
    half2_t p, q, r, s;
    halves4<CODE>(a, p, q);
    halves4<CODE>(b, r, s);
    return half8_t{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}

}  // namespace cache
}  // namespace sc
