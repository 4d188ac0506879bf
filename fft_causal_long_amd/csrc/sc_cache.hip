// Writing tokens into a cache of 8-bit codes and reading them back (gfx950); layout and rounding in
// sc_cache.h.
//
// A workgroup owns one block of k or of v.  Writing: its new tokens' values go to registers, 16 of a
// token a thread (the 16 bytes that lie together in a block of k), the largest magnitude is found over
// the workgroup, and the codes go out in the block's own order; for v they pass through LDS, where a
// thread collects 16 tokens of a value.  A block that also holds older tokens keeps the larger of its
// scale and the new tokens'; if that is larger than what it had, the older codes are rounded again.
// Otherwise only the 16-byte runs that hold a new token are read and written.  Reading runs the other
// way.  Bound by memory: an element read and a byte written for each value.

#include <hip/hip_runtime.h>

#include "sc_cache.h"
#include "sc_rows.h"

namespace sc {

namespace {

using namespace cache;

constexpr int NT = 256;
constexpr int MAX_RUNS = 2;     // 16-byte runs of a thread: 64 tokens of up to 8 chunks over 256 threads

// 16 values of a row (16-byte aligned)
template <class IO>
__device__ __forceinline__ void load16(const typename IO::T* p, float (&x)[16])
{
    constexpr int V = vec_elems<IO>;
    uint4 u[16 / V];
#pragma unroll
    for (int i = 0; i < 16 / V; ++i) u[i] = *(const uint4*)(p + i * V);
#pragma unroll
    for (int i = 0; i < 16 / V; ++i) {
        const Lanes<IO> l = widen<IO>(u[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) x[i * V + e] = l.x[e];
    }
}
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

// The token and chunk of a block's run in k's order.
__device__ __forceinline__ void k_run(int run, int chunks, int& t, int& ch)
{
    const int c = run & 15, rest = run >> 4, kb = rest / chunks;
    ch = rest - kb * chunks;
    t = 16 * (c >> 2) + 4 * kb + (c & 3);
}

// LDS codes of a block token by token: rows of D bytes and 4 more, so that the tokens of a column lie
// in different banks.
constexpr int PAD = 4;

template <class IO, Code CODE>
__global__ __launch_bounds__(NT) void cache_put(CacheArgs c, CacheIo io, int nblk)
{
    using E = typename IO::T;
    __shared__ float top[NT / 64];
    __shared__ uint32_t codes[T * (128 + PAD) / 4];
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

    float x[MAX_RUNS][16], mx = 0.f;
#pragma unroll
    for (int i = 0; i < MAX_RUNS; ++i) {
        const int run = threadIdx.x + i * NT;
        int t, ch;
        k_run(run, chunks, t, ch);
        const bool on = run < runs && t >= from && t < to;
        if (on) load16<IO>(src + (at0 + t - start) * st[1] + 16 * ch, x[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[i][e] = on ? x[i][e] : 0.f;
            mx = fmaxf(mx, magnitude(x[i][e]));
        }
    }
    const int had = from ? exponent_of_scale(*scale) : E_LOW;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = mx;
    __syncthreads();   // (every thread has read the old scale)
    const int e = max(had, exponent_of<CODE>(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))));
    const float by = power(-e);
    const bool grown = from && e > had;
    const float shrink = power(had - e);   // of older codes
    if (threadIdx.x == 0) *scale = power(e);

    if (!is_v) {
#pragma unroll
        for (int i = 0; i < MAX_RUNS; ++i) {
            const int run = threadIdx.x + i * NT;
            int t, ch;
            k_run(run, chunks, t, ch);
            if (run >= runs || (t < from && !grown)) continue;
            if (t < from) {
                decode16<CODE>(*(const uint4*)(out + run * 16), x[i]);
                *(uint4*)(out + run * 16) = encode16<CODE>(x[i], shrink);
            } else if (t < to || !from) {
                *(uint4*)(out + run * 16) = encode16<CODE>(x[i], by);
            }
        }
        return;
    }
    const int row = (D + PAD) / 4;
#pragma unroll
    for (int i = 0; i < MAX_RUNS; ++i) {
        const int run = threadIdx.x + i * NT;
        int t, ch;
        k_run(run, chunks, t, ch);
        if (run >= runs) continue;
        const uint4 u = encode16<CODE>(x[i], by);
        uint32_t* w = codes + t * row + ch * 4;
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MAX_RUNS; ++i) {
        const int run = threadIdx.x + i * NT;   // [chunk][t / 16][d % 16]
        if (run >= runs) continue;
        const int d = (run >> 6) * 16 + (run & 15), t0 = (run >> 4 & 3) * 16;
        const bool has_new = t0 + 16 > from && t0 < to, has_old = t0 < from;
        if (from && !has_new && !(grown && has_old)) continue;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[k] |= (uint32_t)((const uint8_t*)codes)[(t0 + 4 * k + e) * row * 4 + d] << (8 * e);
        }
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

template <class IO, Code CODE>
__global__ __launch_bounds__(NT) void cache_get(CacheArgs c, CacheIo io, int nblk)
{
    using E = typename IO::T;
    __shared__ uint32_t codes[T * (128 + PAD) / 4];
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
    const int row = (D + PAD) / 4;
    if (is_v && p >= 0) {
#pragma unroll
        for (int i = 0; i < MAX_RUNS; ++i) {
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
    for (int i = 0; i < MAX_RUNS; ++i) {
        const int run = threadIdx.x + i * NT;
        if (run >= runs) continue;
        const int t = run / chunks, ch = run - t * chunks;   // whole rows out
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
    if (put) hipLaunchKernelGGL((cache_put<IO, CODE>), dim3((unsigned)wgs), dim3(NT), 0, st, c, io, (int)nblk);
    else hipLaunchKernelGGL((cache_get<IO, CODE>), dim3((unsigned)wgs), dim3(NT), 0, st, c, io, (int)nblk);
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
