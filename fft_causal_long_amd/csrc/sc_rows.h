// Row access shared by the layer kernels (layer norm, gated recurrence, attention): 16-byte
// vectors of float32 or bfloat16 elements, widened exactly to float32 and rounded once on the
// way out (nearest, ties to even).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sc_device.h"

namespace sc {

// Elements of one 16-byte vector.
template <class IO>
constexpr int vec_elems = 16 / IO::SIZE;

template <class IO>
struct Lanes {   // one vector in float32
    float x[vec_elems<IO>];
};

template <class IO>
__device__ __forceinline__ Lanes<IO> widen(const uint4& u)
{
    Lanes<IO> r;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IO::SIZE == 2) {
            r.x[2 * i] = __uint_as_float(w[i] << 16);
            r.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            r.x[i] = __uint_as_float(w[i]);
        }
    }
    return r;
}

template <class IO>
__device__ __forceinline__ uint4 narrow(const Lanes<IO>& v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IO::SIZE == 2) w[i] = pack_bf16x2(v.x[2 * i], v.x[2 * i + 1]);
        else w[i] = __float_as_uint(v.x[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements c .. c+V-1 of the row p of n elements; those at n and beyond read 0.  `whole` says
// that every row starts 16-byte aligned; a vector that the row ends inside, and every vector of
// an unaligned row, is read element by element.
template <class IO>
__device__ __forceinline__ uint4 load_raw(const typename IO::T* p, int c, int n, bool whole)
{
    constexpr int V = vec_elems<IO>;
    if (whole && c + V <= n) return *(const uint4*)(p + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (c + i < n) {
            if constexpr (IO::SIZE == 2) w[i / 2] |= (uint32_t)p[c + i] << (16 * (i & 1));
            else w[i] = __float_as_uint(p[c + i]);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <class IO>
__device__ __forceinline__ void store_raw(typename IO::T* p, int c, int n, bool whole,
                                          const Lanes<IO>& v)
{
    constexpr int V = vec_elems<IO>;
    if (whole && c + V <= n) {
        *(uint4*)(p + c) = narrow<IO>(v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < n) IO::store(p, c + i, v.x[i]);
}

}  // namespace sc
