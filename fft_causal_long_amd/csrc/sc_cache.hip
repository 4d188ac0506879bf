// Writing tokens into a cache of 8-bit codes and reading them back (gfx950); layout and rounding in
// sc_cache.h.
//
// A workgroup owns one block of k or of v.  Writing: its new tokens' values go to registers, of k 16 of a
// token a thread (the 16 bytes that lie together in a block), the largest magnitude is found over
// the workgroup, and the codes go out in the block's own order; for v they pass through LDS, where a
// thread collects 16 tokens of a value.  A block that also holds older tokens keeps the larger of its
// scale and the new tokens'; if that is larger than what it had, the older codes are rounded again.
// Otherwise only the 16-byte runs that hold a new token are read and written.  Reading runs the other
// way.  Bound by memory: an element read and a byte written for each value.
//
// Measured (MI355X): B 4, 8192 tokens, 4 heads of 128 bf16, int8: 20.5 us written (4.9 TB/s; a large copy
// moves 5.4), 18 read back (5.6); B 8, 4096 tokens, 16 heads of 64 bf16, e4m3 49 (4.1) and 33 (6.1): rows
// of 128 bytes a head.  The first in float32: 39 (4.3) and 47 (3.5: each lane stores 64 bytes in four
// pieces, so a wave's stores lie 64 bytes apart).  k and v of a block in one workgroup took 53 for 49; the workgroups of a block's heads
// on one die 2 us less there and 2 more in the first; 20 was 30 with the codes of every value checked and
// clamped, since the arithmetic bound it.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "sc_cache.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace cache;

constexpr int NT = 256;

// 16 values as they are stored: of a token (k), or 4 each of 4 tokens (v).
template <class IO>
struct Sixteen {
    static constexpr int N = 4 * IO::SIZE;
    uint32_t w[N];
    __device__ __forceinline__ void load(const typename IO::T* p)
    {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 u = *(const uint4*)((const uint32_t*)p + i);
            w[i] = u.x;
            w[i + 1] = u.y;
            w[i + 2] = u.z;
            w[i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void load4(const typename IO::T* p, int k)
    {
        if constexpr (IO::SIZE == 2) {
            const uint2 u = *(const uint2*)p;
            w[2 * k] = u.x;
            w[2 * k + 1] = u.y;
        } else {
            const uint4 u = *(const uint4*)p;
            w[4 * k] = u.x;
            w[4 * k + 1] = u.y;
            w[4 * k + 2] = u.z;
            w[4 * k + 3] = u.w;
        }
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (IO::SIZE == 2) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else return __uint_as_float(w[i]);
    }
    // bits of the largest magnitude, or more than infinity's with a NaN
    __device__ __forceinline__ uint32_t top() const
    {
        if constexpr (IO::SIZE == 2) {
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
            u16x2 m = {0, 0};
#pragma unroll
            for (int i = 0; i < N; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
            return (uint32_t)std::max(m[0], m[1]) << 16;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) m = std::max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
    // the largest magnitude of the finite ones
    __device__ __forceinline__ uint32_t finite_top() const
    {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, magnitude(at(i)));
        return __float_as_uint(m);
    }
    // codes of values 4 k .. 4 k + 3 at the scale 2^e
    template <Code CODE>
    __device__ __forceinline__ uint32_t codes(int k, int e) const
    {
        const float by = power(-e);
        return encode4<CODE>(at(4 * k) * by, at(4 * k + 1) * by, at(4 * k + 2) * by, at(4 * k + 3) * by);
    }
    // the same where every value is finite and within the code's range: 2 to 3 instructions a value
    template <Code CODE>
    __device__ __forceinline__ uint32_t plain_codes(int k, int e) const
    {
        if constexpr (CODE == Code::I8) {
            // the sum's last byte is the integer, rounded by the addition, plus 128
            const float by = power(-e), off = 12582912.f + 128.f;
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__builtin_fmaf(at(4 * k + i), by, off));
            return __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u),
                                         __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u), 0x05040100u);
        } else if constexpr (IO::SIZE == 2) {
            typedef short s16x2 __attribute__((ext_vector_type(2)));
            s16x2 r = {0, 0};
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w[2 * k]), power(e), false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w[2 * k + 1]), power(e), true);
            return __builtin_bit_cast(uint32_t, r);
        } else {
            const float by = power(-e);
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(at(4 * k) * by, at(4 * k + 1) * by, 0, false);
            return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(at(4 * k + 2) * by, at(4 * k + 3) * by, lo, true);
        }
    }
};

template <class IO>
__device__ __forceinline__ void store16(typename IO::T* p, const float (&x)[16])
{
    constexpr int V = vec_elems<IO>;
#pragma unroll
    for (int i = 0; i < 16 / V; ++i) {
        Lanes<IO> l;
#pragma unroll
        for (int e = 0; e < V; ++e) l.x[e] = x[i * V + e];
        *(uint4*)(p + i * V) = narrow<IO>(l);
    }
}

template <Code CODE>
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float by)
{
    uint4 u;
    u.x = encode4<CODE>(x[0] * by, x[1] * by, x[2] * by, x[3] * by);
    u.y = encode4<CODE>(x[4] * by, x[5] * by, x[6] * by, x[7] * by);
    u.z = encode4<CODE>(x[8] * by, x[9] * by, x[10] * by, x[11] * by);
    u.w = encode4<CODE>(x[12] * by, x[13] * by, x[14] * by, x[15] * by);
    return u;
}
template <Code CODE>
__device__ __forceinline__ void decode16(const uint4& u, float (&x)[16])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[4];
        decode4<CODE>(w[i], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = y[e];
    }
}

// n / chunks for the n < 512 that a block needs, chunks <= 8 (inv = 65536 / chunks + 1: off by less than
// 512 / 65536).
__device__ __forceinline__ int by_chunks(int n, int inv) { return n * inv >> 16; }

// The token and chunk of a block's run in k's order.
__device__ __forceinline__ void k_run(int run, int chunks, int inv, int& t, int& ch)
{
    const int c = run & 15, rest = run >> 4, kb = by_chunks(rest, inv);
    ch = rest - kb * chunks;
    t = 16 * (c >> 2) + 4 * kb + (c & 3);
}

// LDS codes of a block: reading, token by token, rows of D bytes and 4 more, so that the tokens of a column
// lie in different banks; writing, in the block's order with 16 bytes more a 16-value chunk, so that the
// words of a wave's 16 x 4 values and tokens do.
constexpr int PAD = 4, V_PAD = 16;

// word k's byte e <-> word e's byte k
__device__ __forceinline__ void transpose4(uint32_t (&w)[4])
{
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
}

// RUNS: 16-byte runs of a thread, 64 tokens of 4 RUNS chunks over 256 threads
template <class IO, Code CODE, int RUNS>
__global__ __launch_bounds__(NT) void cache_put(CacheArgs c, CacheIo io, int nblk)
{
    using E = typename IO::T;
    __shared__ uint32_t top[NT / 64];
    __shared__ uint32_t codes[T * (64 * RUNS + PAD) / 4];
    uint32_t id = blockIdx.x;
    const bool is_v = id & 1;
    id >>= 1;
    const int h = (int)(id % (uint32_t)c.Hkv);
    id /= (uint32_t)c.Hkv;
    const int b = (int)(id / (uint32_t)nblk), D = c.D, chunks = D / 16, runs = T * chunks;
    const int64_t end = io.len[b], start = end - io.L;   // positions of the new tokens
    const int first = (int)(start > 0 ? start >> 6 : 0), blk = first + (int)(id % (uint32_t)nblk);
    const int64_t at0 = (int64_t)blk * T;
    if (at0 >= end) return;
    const int p = block_of(c, b, blk);
    if (p < 0) return;
    const int from = (int)(start > at0 ? start - at0 : 0), to = (int)(end - at0 < T ? end - at0 : T);   // new tokens
    const int64_t* st = is_v ? io.vst : io.kst;
    const E* src = (const E*)(is_v ? io.v : io.k) + b * st[0] + h * st[2];
    float* scale = (is_v ? c.vs : c.ks) + (int64_t)p * c.Hkv + h;
    uint8_t* out = (uint8_t*)(is_v ? c.v : c.k) + ((int64_t)p * c.Hkv + h) * T * D;

    const int inv = 65536 / chunks + 1;
    const E* row0 = src + (at0 - start) * st[1];   // (token 0 of the block: before the tensor if it is older)

    Sixteen<IO> x[RUNS];
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int run = threadIdx.x + i * NT;
#pragma unroll
        for (int e = 0; e < Sixteen<IO>::N; ++e) x[i].w[e] = 0;
        if (!is_v) {
            int t, ch;
            k_run(run, chunks, inv, t, ch);
            if (run < runs && t >= from && t < to) x[i].load(row0 + t * st[1] + 16 * ch);
        } else {
            const int t4 = by_chunks(run >> 2, inv), dq = run - t4 * 4 * chunks;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * t4 + k;
                if (run < runs && t >= from && t < to) x[i].load4(row0 + t * st[1] + 4 * dq, k);
            }
        }
        bits = std::max(bits, x[i].top());
    }
    const int had = from ? exponent_of_scale(*scale) : E_LOW;
    auto over_all = [&](uint32_t m) {
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = std::max(m, (uint32_t)__shfl_xor((int)m, k));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
        __syncthreads();   // (and every thread has read the old scale)
        return std::max(std::max(top[0], top[1]), std::max(top[2], top[3]));
    };
    bits = over_all(bits);
    // infinities, NaN, values past the largest scale: looked at one by one
    const bool odd = bits > __float_as_uint(CODE == Code::I8 ? 127.f : 448.f) + ((uint32_t)E_HIGH << 23);
    if (odd) {
        bits = 0;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) bits = std::max(bits, x[i].finite_top());
        bits = over_all(bits);
    }
    const int e = max(had, exponent_of<CODE>(__uint_as_float(bits)));
    const bool grown = from && e > had;
    const float shrink = power(had - e);   // of older codes
    if (threadIdx.x == 0) *scale = power(e);
    auto word = [&](const Sixteen<IO>& s, int k) { return odd ? s.template codes<CODE>(k, e) : s.template plain_codes<CODE>(k, e); };

    if (!is_v) {
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int run = threadIdx.x + i * NT;
            int t, ch;
            k_run(run, chunks, inv, t, ch);
            if (run >= runs || (t < from && !grown)) continue;
            if (t < from) {
                float y[16];
                decode16<CODE>(*(const uint4*)(out + run * 16), y);
                *(uint4*)(out + run * 16) = encode16<CODE>(y, shrink);
            } else if (t < to || !from) {
                *(uint4*)(out + run * 16) = make_uint4(word(x[i], 0), word(x[i], 1), word(x[i], 2), word(x[i], 3));
            }
        }
        return;
    }
    // four tokens of a value in a word, in the block's order
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int unit = threadIdx.x + i * NT, t4 = by_chunks(unit >> 2, inv), dq = unit - t4 * 4 * chunks;
        if (unit >= runs) continue;
        uint32_t w[4] = {word(x[i], 0), word(x[i], 1), word(x[i], 2), word(x[i], 3)};
        transpose4(w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 4 * dq + e;
            codes[(v_at(d, t4 >> 2) + (d >> 4) * V_PAD) / 4 + (t4 & 3)] = w[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int run = threadIdx.x + i * NT;   // [chunk][t / 16][d % 16]
        if (run >= runs) continue;
        const int t0 = (run >> 4 & 3) * 16;
        const bool has_new = t0 + 16 > from && t0 < to, has_old = t0 < from;
        if (from && !has_new && !(grown && has_old)) continue;
        const uint4 fresh = *(const uint4*)(codes + (run * 16 + (run >> 6) * V_PAD) / 4);
        uint32_t w[4] = {fresh.x, fresh.y, fresh.z, fresh.w};
        if (has_old) {
            const uint4 u = *(const uint4*)(out + run * 16);
            uint32_t old[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (grown) {
                    float y[4];
                    decode4<CODE>(old[k], y);
                    old[k] = encode4<CODE>(y[0] * shrink, y[1] * shrink, y[2] * shrink, y[3] * shrink);
                }
                const int keep = from - t0 - 4 * k;   // bytes of this word that are older
                const uint32_t mask = keep >= 4 ? ~0u : keep <= 0 ? 0u : (1u << (8 * keep)) - 1;
                w[k] = (old[k] & mask) | (w[k] & ~mask);
            }
        }
        *(uint4*)(out + run * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <class IO, Code CODE, int RUNS>
__global__ __launch_bounds__(NT) void cache_get(CacheArgs c, CacheIo io, int nblk)
{
    using E = typename IO::T;
    __shared__ uint32_t codes[T * (64 * RUNS + PAD) / 4];
    uint32_t id = blockIdx.x;
    const bool is_v = id & 1;
    id >>= 1;
    const int h = (int)(id % (uint32_t)c.Hkv);
    id /= (uint32_t)c.Hkv;
    const int b = (int)(id / (uint32_t)nblk), D = c.D, chunks = D / 16, runs = T * chunks;
    const int64_t end = io.len[b], start = end - io.L;
    const int64_t blk = (start >> 6) + (int64_t)(id % (uint32_t)nblk), at0 = blk * T;   // start may be negative
    if (at0 >= end) return;
    const int p = blk >= 0 && blk < c.N ? block_of(c, b, (int)blk) : -1;
    const int from = (int)(start > at0 ? start - at0 : 0), to = (int)(end - at0 < T ? end - at0 : T);
    const int64_t* st = is_v ? io.vst : io.kst;
    E* dst = (E*)(is_v ? io.vo : io.ko) + b * st[0] + h * st[2];
    const float scale = p < 0 ? 0.f : power(exponent_of_scale((is_v ? c.vs : c.ks)[(int64_t)p * c.Hkv + h]));
    const uint8_t* in = (const uint8_t*)(is_v ? c.v : c.k) + ((int64_t)(p < 0 ? 0 : p) * c.Hkv + h) * T * D;
    const int row = (D + PAD) / 4, inv = 65536 / chunks + 1;
    if (is_v && p >= 0) {
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int run = threadIdx.x + i * NT;
            if (run >= runs) continue;
            const int d = (run >> 6) * 16 + (run & 15), t0 = (run >> 4 & 3) * 16;
            const uint4 u = *(const uint4*)(in + run * 16);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 16; ++k) ((uint8_t*)codes)[(t0 + k) * row * 4 + d] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
        const int run = threadIdx.x + i * NT;
        if (run >= runs) continue;
        const int t = by_chunks(run, inv), ch = run - t * chunks;   // whole rows out
        if (t < from || t >= to) continue;
        float x[16];
        uint4 u = make_uint4(0, 0, 0, 0);
        if (p >= 0) {
            if (is_v) {
                const uint32_t* w = codes + t * row + ch * 4;
                u = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                u = *(const uint4*)(in + k_at(t, ch, chunks));
            }
        }
        decode16<CODE>(u, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = p < 0 ? 0.f : x[e] * scale;
        store16<IO>(dst + (at0 + t - start) * st[1] + 16 * ch, x);
    }
}

// Blocks that L tokens can touch.
int64_t blocks_of(int64_t L) { return (L + T - 2) / T + 1; }

template <class IO, Code CODE>
hipError_t go(const CacheArgs& c, const CacheIo& io, bool put, hipStream_t st)
{
    const int64_t nblk = blocks_of(io.L), wgs = 2 * nblk * c.B * (int64_t)c.Hkv;
    if (!grid_ok(wgs, NT)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)wgs), block(NT);
    if (c.D <= 64) {
        if (put) hipLaunchKernelGGL((cache_put<IO, CODE, 1>), grid, block, 0, st, c, io, (int)nblk);
        else hipLaunchKernelGGL((cache_get<IO, CODE, 1>), grid, block, 0, st, c, io, (int)nblk);
    } else {
        if (put) hipLaunchKernelGGL((cache_put<IO, CODE, 2>), grid, block, 0, st, c, io, (int)nblk);
        else hipLaunchKernelGGL((cache_get<IO, CODE, 2>), grid, block, 0, st, c, io, (int)nblk);
    }
    return hipGetLastError();
}

hipError_t pick(Store s, Code code, const CacheArgs& c, const CacheIo& io, bool put, hipStream_t st)
{
    if (s == Store::F32) return code == Code::I8 ? go<f32_io, Code::I8>(c, io, put, st) : go<f32_io, Code::E4M3>(c, io, put, st);
    return code == Code::I8 ? go<bf16_io, Code::I8>(c, io, put, st) : go<bf16_io, Code::E4M3>(c, io, put, st);
}

}  // namespace

hipError_t launch_cache_write(Store s, Code code, const CacheArgs& c, const CacheIo& io, hipStream_t st)
{
    return pick(s, code, c, io, true, st);
}

hipError_t launch_cache_read(Store s, Code code, const CacheArgs& c, const CacheIo& io, hipStream_t st)
{
    return pick(s, code, c, io, false, st);
}

}  // namespace sc
