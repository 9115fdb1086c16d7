// Element types of the row, router and adapter operators: bf16, fp16 and
// float32 rows in 16-byte pieces, widened to float32 for every sum.
#pragma once

#include <type_traits>

#include "moe_common.hpp"

namespace moe {

inline size_t elem_bytes(int dtype) { return dtype == MOE_DT_F32 ? 4 : 2; }

template <int DT>
struct Elem;

// One 16-byte piece as kVec float32 values and back, by the hardware
// conversions (round to nearest even).
template <>
struct Elem<MOE_DT_BF16> {
    typedef uint16_t type;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float load(const type *p)
    {
        return __uint_as_float((uint32_t)*p << 16);
    }
    static __device__ __forceinline__ uint32_t bits_of(float lo, float hi)
    {
        typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
    }
    static __device__ __forceinline__ void store(type *p, float v) { *p = (type)bits_of(v, v); }
    static __device__ __forceinline__ void unpack(const uint4 &q, float *f)
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = bits_of(f[2 * i], f[2 * i + 1]);
        return uint4{o[0], o[1], o[2], o[3]};
    }
};

template <>
struct Elem<MOE_DT_F16> {
    typedef uint16_t type;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float half_of(uint32_t bits)
    {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    }
    static __device__ __forceinline__ uint32_t bits_of(float v)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
    static __device__ __forceinline__ float load(const type *p) { return half_of(*p); }
    static __device__ __forceinline__ void store(type *p, float v) { *p = (type)bits_of(v); }
    static __device__ __forceinline__ void unpack(const uint4 &q, float *f)
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = half_of(w[i]);
            f[2 * i + 1] = half_of(w[i] >> 16);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = bits_of(f[2 * i]) | (bits_of(f[2 * i + 1]) << 16);
        return uint4{o[0], o[1], o[2], o[3]};
    }
};

template <>
struct Elem<MOE_DT_F32> {
    typedef float type;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float load(const type *p) { return *p; }
    static __device__ __forceinline__ void store(type *p, float v) { *p = v; }
    static __device__ __forceinline__ void unpack(const uint4 &q, float *f)
    {
        f[0] = __uint_as_float(q.x);
        f[1] = __uint_as_float(q.y);
        f[2] = __uint_as_float(q.z);
        f[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
    }
};

// A 16-byte store that leaves the L2 first.
__device__ __forceinline__ void store_once(void *p, const uint4 &q)
{
    typedef unsigned int u4v __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(u4v{q.x, q.y, q.z, q.w}, static_cast<u4v *>(p));
}

// A row index from a route table, or -1 where it names no row of the R rows
// (a slot of -1; an index past the buffers is never followed).
__device__ __forceinline__ int checked_row(int row, long R)
{
    return (unsigned)row < (unsigned long)R ? row : -1;
}

// Calls f with the element type as a constant.
template <typename F>
void with_elem(int dtype, F f)
{
    if (dtype == MOE_DT_BF16)
        f(std::integral_constant<int, MOE_DT_BF16>{});
    else if (dtype == MOE_DT_F16)
        f(std::integral_constant<int, MOE_DT_F16>{});
    else
        f(std::integral_constant<int, MOE_DT_F32>{});
}

} // namespace moe
