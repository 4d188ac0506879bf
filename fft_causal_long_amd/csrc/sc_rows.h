// Row access shared by the layer kernels (layer norm, gated recurrence, attention): 16-byte
// vectors of float32 or bfloat16 elements, widened exactly to float32 and rounded once on the
// way out (nearest, ties to even).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sc_device.h"

namespace sc {

// Workgroups go to the eight dies round robin.  Work item of workgroup `id` of `n` such that
// each die takes a run of consecutive items: neighbours that share cache lines or operands then
// share an L2.  (What n leaves over a multiple of 8 stays in place.)
__device__ __forceinline__ uint32_t die_order(uint32_t id, uint32_t n)
{
    const uint32_t per = n >> 3;
    return id < (per << 3) ? (id & 7) * per + (id >> 3) : id;
}

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

// Elements c .. c+V-1 (c < n) of the row p of n elements.  WHOLE: every row starts 16-byte
// aligned and n is a multiple of V, so the vector is one load; a kernel takes one form or the
// other, since a choice at each load would make every load wait for the one before.  Otherwise
// the elements are read one by one, those at n and beyond as 0; STEP apart, so that with STEP lanes
// beside each other every load takes neighbouring elements.
template <class IO, bool WHOLE, int STEP = 1>
__device__ __forceinline__ uint4 load_raw(const typename IO::T* p, int c, int n)
{
    constexpr int V = vec_elems<IO>;
    if constexpr (WHOLE) {
        return *(const uint4*)(p + c);
    } else {
        // each element's own address or the row's last: no branch
        uint32_t w[4];
        if constexpr (IO::SIZE == 2) {
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c0 = c + 2 * i * STEP, c1 = c0 + STEP;
                const u16x2 v = {p[c0 < n ? c0 : n - 1], p[c1 < n ? c1 : n - 1]};
                w[i] = __builtin_bit_cast(uint32_t, v) & (c1 < n ? 0xffffffffu : c0 < n ? 0xffffu : 0u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = c + i * STEP < n;
                const float v = p[in ? c + i * STEP : n - 1];
                w[i] = in ? __float_as_uint(v) : 0u;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <class IO, bool WHOLE, int STEP = 1>
__device__ __forceinline__ void store_raw(typename IO::T* p, int c, int n, const Lanes<IO>& v)
{
    constexpr int V = vec_elems<IO>;
    if constexpr (WHOLE) {
        *(uint4*)(p + c) = narrow<IO>(v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i * STEP < n) IO::store(p, c + i * STEP, v.x[i]);
    }
}

}  // namespace sc
