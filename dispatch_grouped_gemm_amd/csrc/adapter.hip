// Low-rank adapters of many requests beside one shared projection:
//   out[t] = base[t] + scale_l (x[t] A_l^T) B_l^T,   l = ids[t],
// base = x W^T computed here, or given; a row of id -1 (or past the
// adapters) has no second term.
//
// Two launches.  The first ("shrink") makes v[t] = x[t] A_l^T in float32.
// The second computes x W^T in 16x16x32 MFMA tiles and, once a tile's sums
// are complete, adds the adapters' term to them in registers ("expand"), so
// out is written once and rounded once.
//
// Rows come in any order.  Whoever owns a set of rows walks the different
// ids among them: an adapter's product is formed for all the rows of the
// set (the matrix instruction costs the same) and taken only where the id
// matches, so no row ever sees another adapter's values, infinite or NaN.
//
// v keeps float32's precision through the matrix instruction: it enters as
// the sum of two 16-bit values, hi = round(v) and lo = round(v - hi).  fp16
// lacks float32's range, so there v is first divided by a power of two that
// puts the row's largest magnitude below 1, and the product multiplied by it.
#include "elem.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

struct AShape {
    int T, H, N, L, r;
};

// D(16x16) += A(16x32) B(32x16): lane l holds A's row / B's column l mod 16
// at k = 8 (l div 16) .. + 7, and D's column l mod 16 at rows
// 4 (l div 16) .. + 3.
template <int DT>
__device__ __forceinline__ v4f mfma(const uint4 &a, const uint4 &b, v4f c)
{
    if constexpr (DT == MOE_DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                      __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// v as hi + lo, both 16-bit.
template <int DT>
__device__ __forceinline__ void split8(const float *v, uint4 &hi, uint4 &lo)
{
    float h[8], d[8];
    hi = Elem<DT>::pack(v);
    Elem<DT>::unpack(hi, h);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        d[i] = fabsf(h[i]) < INFINITY ? v[i] - h[i] : 0.0f;
    lo = Elem<DT>::pack(d);
}

// ids of the 16 rows that lanes 0..15 (and their copies) hold; -1 where a
// row has no adapter.
__device__ __forceinline__ int adapter_of(const AShape &s, const int32_t *ids, long t)
{
    const int id = t < s.T ? ids[t] : -1;
    return (unsigned)id < (unsigned)s.L ? id : -1;
}

// One wavefront: 16 rows x 16 of the rank over one part of H.
template <int DT>
__global__ void __launch_bounds__(64)
shrink_kernel(AShape s, const uint16_t *__restrict__ x, const int32_t *__restrict__ ids,
              const uint16_t *__restrict__ a, float *__restrict__ v)
{
    const int lane = threadIdx.x;
    const long t = (long)blockIdx.x * 16 + (lane & 15);
    const int j = blockIdx.y * 16 + (lane & 15);
    const int id = adapter_of(s, ids, t);
    const uint16_t *xr = x + (size_t)(t < s.T ? t : s.T - 1) * s.H + 8 * (lane >> 4);
    uint64_t todo = __ballot(id >= 0 && lane < 16);
    while (todo) {
        const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= ~__ballot(id == g);
        const uint16_t *ar =
            a + ((size_t)g * s.r + (j < s.r ? j : s.r - 1)) * s.H + 8 * (lane >> 4);
        v4f c = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int h = 0; h < s.H; h += 32)
            c = mfma<DT>(*reinterpret_cast<const uint4 *>(ar + h),
                         *reinterpret_cast<const uint4 *>(xr + h), c);
        const int j0 = blockIdx.y * 16 + 4 * (lane >> 4);
        if (id == g && j0 < s.r)
            *reinterpret_cast<v4f *>(v + (size_t)t * s.r + j0) = c;
    }
}

// Adds the adapters' term of 16 rows (lane's row: l mod 16, its id) to the
// sums of NF blocks of 16 columns from n0.
template <int DT, int NF>
__device__ __forceinline__ void expand(const AShape &s, const float *__restrict__ v,
                                       const uint16_t *__restrict__ b,
                                       const float *__restrict__ scale, long t, int id, int n0,
                                       v4f *acc)
{
    const int lane = threadIdx.x & 63;
    const int k0 = 8 * (lane >> 4);
    const float *vr = v + (size_t)t * s.r;
    int ex = 0;
    if constexpr (DT == MOE_DT_F16) {
        float m = 0.0f;
        if (id >= 0)
            for (int k = k0; k < s.r; k += 32)
                for (int i = 0; i < 8; ++i)
                    m = fmaxf(m, fabsf(vr[k + i]));
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        if (m > 0.0f && m < INFINITY)
            (void)frexpf(m, &ex);
    }
    const float sc = id < 0 ? 0.0f : scale ? scale[id] : 1.0f;
    uint64_t todo = __ballot(id >= 0 && lane < 16);
    while (todo) {
        const int g = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= ~__ballot(id == g);
        v4f d[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            d[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < s.r; k += 32) {
            const bool in = k + k0 < s.r;
            float f8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f8[i] = in && id == g ? vr[k + k0 + i] : 0.0f;
                if constexpr (DT == MOE_DT_F16)
                    f8[i] = ldexpf(f8[i], -ex);
            }
            uint4 hi, lo;
            split8<DT>(f8, hi, lo);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int n = min(n0 + 16 * f + (lane & 15), s.N - 1);
                uint4 bq = {0, 0, 0, 0};
                if (in)
                    bq = *reinterpret_cast<const uint4 *>(b + ((size_t)g * s.N + n) * s.r + k +
                                                          k0);
                d[f] = mfma<DT>(bq, hi, d[f]);
                d[f] = mfma<DT>(bq, lo, d[f]);
            }
        }
        if (id == g)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[f][i] += sc * ldexpf(d[f][i], ex);
    }
}

// Four wavefronts: 64 rows x 64 columns, each wavefront 16 rows.
template <int DT>
__global__ void __launch_bounds__(kThreads)
project_kernel(AShape s, const uint16_t *__restrict__ x, const uint16_t *__restrict__ w,
               const uint16_t *base, const int32_t *__restrict__ ids,
               const uint16_t *__restrict__ b, const float *__restrict__ scale,
               const float *__restrict__ v, uint16_t *out)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long t0 = (long)blockIdx.x * 64 + wave * 16;
    if (t0 >= s.T)
        return;
    const long t = t0 + (lane & 15);
    const int n0 = blockIdx.y * 64;
    const int id = adapter_of(s, ids, t);
    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
        acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (w) {
        const uint16_t *xr = x + (size_t)(t < s.T ? t : s.T - 1) * s.H + 8 * (lane >> 4);
        const uint16_t *wr[4];
#pragma unroll
        for (int f = 0; f < 4; ++f)
            wr[f] = w + (size_t)min(n0 + 16 * f + (lane & 15), s.N - 1) * s.H + 8 * (lane >> 4);
        for (int h = 0; h < s.H; h += 32) {
            const uint4 xq = *reinterpret_cast<const uint4 *>(xr + h);
#pragma unroll
            for (int f = 0; f < 4; ++f)
                acc[f] = mfma<DT>(*reinterpret_cast<const uint4 *>(wr[f] + h), xq, acc[f]);
        }
    }
    if (!w && t < s.T)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int n = n0 + 16 * f + 4 * (lane >> 4);
            if (n < s.N)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[f][i] = Elem<DT>::load(base + (size_t)t * s.N + n + i);
        }
    expand<DT, 4>(s, v, b, scale, t < s.T ? t : s.T - 1, id, n0, acc);
    if (t >= s.T)
        return;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
        const int n = n0 + 16 * f + 4 * (lane >> 4);
        if (n < s.N)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                Elem<DT>::store(out + (size_t)t * s.N + n + i, acc[f][i]);
    }
}

template <int DT>
hipError_t adapter_of_type(const moe_adapter_shape &sh, const void *x, const void *w,
                           const void *base, const int32_t *ids, const void *a, const void *b,
                           const float *scale, void *out, float *v, hipStream_t st)
{
    const AShape s{sh.T, sh.H, sh.N, sh.L, sh.rank};
    const auto *xe = static_cast<const uint16_t *>(x);
    shrink_kernel<DT><<<dim3((s.T + 15u) / 16u, (s.r + 15) / 16), 64, 0, st>>>(
        s, xe, ids, static_cast<const uint16_t *>(a), v);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    project_kernel<DT><<<dim3((s.T + 63u) / 64u, (s.N + 63) / 64), kThreads, 0, st>>>(
        s, xe, static_cast<const uint16_t *>(w), static_cast<const uint16_t *>(base), ids,
        static_cast<const uint16_t *>(b), scale, v, static_cast<uint16_t *>(out));
    return hipGetLastError();
}

} // namespace

size_t adapter_workspace_bytes(const moe_adapter_shape &s)
{
    return (size_t)s.T * s.rank * sizeof(float);
}

hipError_t launch_adapter_project(const moe_adapter_shape &s, int dtype, const void *x,
                                  const void *w, const void *base, const int32_t *ids,
                                  const void *a, const void *b, const float *scale, void *out,
                                  void *ws, hipStream_t st)
{
    float *v = static_cast<float *>(ws);
    if (dtype == MOE_DT_BF16)
        return adapter_of_type<MOE_DT_BF16>(s, x, w, base, ids, a, b, scale, out, v, st);
    return adapter_of_type<MOE_DT_F16>(s, x, w, base, ids, a, b, scale, out, v, st);
}

} // namespace moe
