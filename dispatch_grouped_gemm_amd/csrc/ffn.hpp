// The dense feed-forward block's parts that its forward and backward launches
// share: the activation and its gradient, what a lane does with 8 neighbouring
// sums, the tile kernels, and the join of K's parts.
#pragma once

#include <algorithm>

#include "tile16.hpp"

namespace moe {

// Pre-activations as they are kept for the backward pass: in the elements'
// type (scale null) or as MX FP8 (codes and an exponent byte per 32 columns).
struct Kept {
    void *rows; // [T, 2I], null: not kept
    uint8_t *scale;
};

__device__ __forceinline__ float not_above(float v, float top) { return v > top ? top : v; }
__device__ __forceinline__ float between(float v, float top)
{
    return v > top ? top : (v < -top ? -top : v); // a NaN stays one
}

// The logistic function by the hardware's exp and reciprocal: a few float32
// ulps (and those of exp, 2^-24 |g|), under the rounding to 16 bits by far.
__device__ __forceinline__ float logistic(float g)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// 8 neighbouring values of a 16-bit row, or of an MX FP8 one.
template <int DT>
__device__ __forceinline__ void load8(const uint16_t *p, float *f)
{
    Elem<DT>::unpack(*reinterpret_cast<const uint4 *>(p), f);
}

template <int DT>
__device__ __forceinline__ void store8(uint16_t *p, const float *f)
{
    *reinterpret_cast<uint4 *>(p) = Elem<DT>::pack(f);
}

__device__ __forceinline__ void load8_mx(const uint8_t *codes, uint8_t scale, float *f)
{
    const uint2 q = *reinterpret_cast<const uint2 *>(codes);
    const int e = (int)scale - 127;
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        f[4 * i] = ldexpf(lo[0], e);
        f[4 * i + 1] = ldexpf(lo[1], e);
        f[4 * i + 2] = ldexpf(hi[0], e);
        f[4 * i + 3] = ldexpf(hi[1], e);
    }
}

// 8 of a block of 32 values as MX FP8; the block's other values are in the
// lanes D, 2 D and 3 D further (xor).
template <int D>
__device__ __forceinline__ void store8_mx(uint8_t *codes, uint8_t *scale, const float *f, bool first)
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor(amax, D));
    amax = fmaxf(amax, __shfl_xor(amax, 2 * D));
    const int e = mx8_block_exponent(amax);
    *reinterpret_cast<uint2 *>(codes) = uint2{mx8_pack4(f[0], f[1], f[2], f[3], e, amax),
                                              mx8_pack4(f[4], f[5], f[6], f[7], e, amax)};
    if (first)
        *scale = (uint8_t)(e + 127);
}

// h = silu(min(g, gl)) clamp(u, ul) of 8 columns j .. j + 7 of row t, from the
// float32 sums; D: lane distance of a block's four pieces.
template <int DT, int D>
struct Activate {
    int I;
    float gl, ul;
    Kept kept;
    uint16_t *h;

    __device__ __forceinline__ void operator()(long t, int j, const float *g, const float *u) const
    {
        if (kept.rows) {
            const long at = t * 2 * I + j;
            if (kept.scale) {
                uint8_t *c = static_cast<uint8_t *>(kept.rows) + at;
                uint8_t *s = kept.scale + at / 32;
                store8_mx<D>(c, s, g, (j & 31) == 0);
                store8_mx<D>(c + I, s + I / 32, u, (j & 31) == 0);
            } else {
                uint16_t *r = static_cast<uint16_t *>(kept.rows) + at;
                store8<DT>(r, g);
                store8<DT>(r + I, u);
            }
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gc = not_above(g[i], gl);
            v[i] = gc * logistic(gc) * between(u[i], ul);
        }
        // h is rounded once to the type: the second product's operand
        store8<DT>(h + t * I + j, v);
    }
};

// dg, du and h of 8 columns of row t from dh and what was kept:
//   du = dh silu(g'),  dg = dh u' s (1 + g' (1 - s)),  s = logistic(g'),
// 0 where the clamp holds the value.
template <int DT>
struct ActivateBack {
    int I;
    float gl, ul;
    Kept kept;
    uint16_t *dgu, *h;

    __device__ __forceinline__ void operator()(long t, int j, const float *dh) const
    {
        float g[8], u[8], v[8];
        const long at = t * 2 * I + j;
        if (kept.scale) {
            const uint8_t *c = static_cast<const uint8_t *>(kept.rows) + at;
            const uint8_t *s = kept.scale + at / 32;
            load8_mx(c, *s, g);
            load8_mx(c + I, s[I / 32], u);
        } else {
            const uint16_t *r = static_cast<const uint16_t *>(kept.rows) + at;
            load8<DT>(r, g);
            load8<DT>(r + I, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gc = not_above(g[i], gl), uc = between(u[i], ul);
            const float s = logistic(gc), silu = gc * s;
            v[i] = silu * uc;
            const float dg = dh[i] * uc * s * (1.0f + gc * (1.0f - s)), du = dh[i] * silu;
            g[i] = g[i] > gl ? 0.0f : dg;
            u[i] = fabsf(u[i]) > ul ? 0.0f : du;
        }
        // rounded once to the type: operands of the products that follow
        store8<DT>(dgu + at, g);
        store8<DT>(dgu + at + I, u);
        if (h)
            store8<DT>(h + t * I + j, v);
    }
};

// 8 columns of a row as they are, added to `base` (may be out itself) or to
// what float32 `out32` holds; rounded once.
template <int DT>
struct Put {
    long ld;
    const uint16_t *base;
    uint16_t *out;
    float *out32;
    bool accumulate; // out32 += instead of =

    __device__ __forceinline__ void operator()(long m, int n, const float *f) const
    {
        const long at = m * ld + n;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = f[i];
        if (out32) {
            v4f *o = reinterpret_cast<v4f *>(out32 + at);
            v4f lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (accumulate) {
                lo += o[0];
                hi += o[1];
            }
            o[0] = lo;
            o[1] = hi;
            return;
        }
        if (base) {
            float b[8];
            load8<DT>(base + at, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += b[i];
        }
        store_once(out + at, Elem<DT>::pack(v));
    }
};

// A product's sizes and operands: C [M, N] over K; tiles tm x tn, K in
// `splits` parts.  kPairs: N is 2I rows of W13 and a tile's columns are half
// gate, half up of the same I.
struct Product {
    Operand a, b;
    long M, K;
    int N, tm, tn, splits, whole;
    float *parts; // [splits][M][N], null: the sums go to the functor
};

template <typename T, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__device__ __forceinline__ void product_tile(const Product &p, const F &f, long m0, int in,
                                             int part, uint8_t *lds)
{
    const int n0 = in * (kPairs ? T::kBN / 2 : T::kBN);
    const int I = p.N / 2;
    const int steps = (int)((p.K + 63) / 64);
    const int first = (int)((long)steps * part / p.splits);
    const int end = (int)((long)steps * (part + 1) / p.splits);
    T tile;
    tile.run(
        lds, p.a, [&](int i) { return min(m0 + i, p.M - 1); }, m0, p.M, p.b,
        [&](int i) -> long {
            const int b = (i >> 4) & 3;
            if (!kPairs)
                return min(n0 + 64 * (i >> 6) + tile_column(b, i & 15), p.N - 1);
            return (b >> 1) * (long)I + min(n0 + 32 * (i >> 6) + tile_column(b & 1, i & 15), I - 1);
        },
        n0, p.N, p.K, first, end - first);
    const int lane = threadIdx.x & 63, wave = tile_wave();
    const int wm = wave / T::kWN, wn = wave % T::kWN;
    const int q = 8 * (lane >> 4);
#pragma unroll
    for (int m = 0; m < T::MF; ++m) {
        const long row = m0 + (wm * T::MF + m) * 16 + (lane & 15);
        if (row >= p.M)
            continue;
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[h][i] = tile.acc[m][2 * h][i];
                v[h][4 + i] = tile.acc[m][2 * h + 1][i];
            }
        if (p.parts) {
            float *o = p.parts + ((long)part * p.M + row) * p.N;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = kPairs ? n0 + 32 * wn + q : n0 + 64 * wn + 32 * h + q;
                if (n < (kPairs ? I : p.N)) {
                    v4f *d = reinterpret_cast<v4f *>(o + n + (kPairs ? h * I : 0));
                    d[0] = tile.acc[m][2 * h];
                    d[1] = tile.acc[m][2 * h + 1];
                }
            }
        } else if constexpr (kPairs) {
            const int n = n0 + 32 * wn + q;
            if (n < I)
                f(row, n, v[0], v[1]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = n0 + 64 * wn + 32 * h + q;
                if (n < p.N)
                    f(row, n, v[h]);
            }
        }
    }
}

// `whole` tiles of 256 x 256, then each tile left over as two of 128 rows.
template <int DT, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
product_large_kernel(Product p, F f)
{
    using T = Tile<DT, 256, 256, 2, 4, 2, ADOWN, BDOWN>;
    using H = Tile<DT, 128, 256, 2, 4, 2, ADOWN, BDOWN>;
    __shared__ __align__(1024) uint8_t lds[T::kLds];
    const int b = blockIdx.x;
    int im, in;
    if (b < p.whole) {
        tile_place(tile_run(b, p.whole), p.tm, p.tn, &im, &in);
        product_tile<T, kPairs, ADOWN, BDOWN>(p, f, im * 256l, in, 0, lds);
        return;
    }
    const int h = tile_run(b - p.whole, gridDim.x - p.whole);
    tile_place(p.whole + (h >> 1), p.tm, p.tn, &im, &in);
    const long m0 = im * 256l + 128 * (h & 1);
    if (m0 < p.M)
        product_tile<H, kPairs, ADOWN, BDOWN>(p, f, m0, in, 0, lds);
}

template <int DT, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
product_small_kernel(Product p, F f)
{
    using T = Tile<DT, 128, 128, 2, 2, 2, ADOWN, BDOWN>;
    __shared__ __align__(1024) uint8_t lds[T::kLds];
    const int tiles = p.tm * p.tn, q = tile_run(blockIdx.x, tiles * p.splits);
    const int part = q / tiles;
    int im, in;
    tile_place(q - part * tiles, p.tm, p.tn, &im, &in);
    product_tile<T, kPairs, ADOWN, BDOWN>(p, f, im * 128l, in, part, lds);
}

// The functor on the sum of the parts' planes, added in their order; four
// neighbouring threads take a block of 32 columns.
template <bool kPairs, typename F>
__global__ void __launch_bounds__(256) join_kernel(Product p, F f)
{
    const int cols = (kPairs ? p.N / 2 : p.N) / 8;
    const long i = blockIdx.x * 256l + threadIdx.x;
    const long row = i / cols;
    const int n = (int)(i - row * cols) * 8;
    if (row >= p.M)
        return;
    float v[2][8];
#pragma unroll
    for (int h = 0; h < (kPairs ? 2 : 1); ++h) {
        v4f lo = {0, 0, 0, 0}, hi = lo;
        for (int s = 0; s < p.splits; ++s) {
            const v4f *o = reinterpret_cast<const v4f *>(p.parts + (s * p.M + row) * p.N + n +
                                                         h * (p.N / 2));
            lo += o[0];
            hi += o[1];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[h][k] = lo[k];
            v[h][4 + k] = hi[k];
        }
    }
    if constexpr (kPairs)
        f(row, n, v[0], v[1]);
    else
        f(row, n, v[0]);
}

constexpr int kTileCus = 256; // workgroups that fill an MI355X; the workspace goes by it

inline long tiles_up(long n, long by) { return (n + by - 1) / by; }

// How a product of M x N over K is cut (kPairs: N the 2I rows of W13).
struct Cut {
    bool large;
    int splits;
};

inline Cut product_cut(long M, long N, long K)
{
    const long n = tiles_up(M, 128) * tiles_up(N, 128);
    const bool large = tiles_up(M, 256) * tiles_up(N, 256) >= kTileCus;
    const long steps = tiles_up(K, 64);
    int splits = 1;
    if (!large && n <= 256)
        splits = (int)std::max(1l, std::min({512 / n, 8l, steps / 8}));
    return Cut{large, splits};
}

inline size_t product_parts_bytes(long M, long N, long K)
{
    const Cut c = product_cut(M, N, K);
    return c.splits > 1 ? (size_t)c.splits * M * N * sizeof(float) : 0;
}

// join: the functor with the lane distance of the join kernel.
template <int DT, bool kPairs, bool ADOWN, bool BDOWN, typename F, typename J>
hipError_t launch_product(Product p, const F &f, const J &join, float *parts, hipStream_t st)
{
    const Cut c = product_cut(p.M, p.N, p.K);
    p.splits = c.splits;
    p.parts = c.splits > 1 ? parts : nullptr;
    if (c.large) {
        p.tm = (int)tiles_up(p.M, 256);
        p.tn = (int)tiles_up(p.N, 256);
        const int cus = kTileCus, left = (int)((long)p.tm * p.tn % cus);
        const int halves = 2 * left <= cus ? left : 0;
        p.whole = p.tm * p.tn - halves;
        product_large_kernel<DT, kPairs, ADOWN, BDOWN>
            <<<p.tm * p.tn + halves, 512, 0, st>>>(p, f);
        return hipGetLastError();
    }
    p.tm = (int)tiles_up(p.M, 128);
    p.tn = (int)tiles_up(p.N, 128);
    product_small_kernel<DT, kPairs, ADOWN, BDOWN>
        <<<p.tm * p.tn * p.splits, 256, 0, st>>>(p, f);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.parts)
        return e;
    const long threads = p.M * ((kPairs ? p.N / 2 : p.N) / 8);
    join_kernel<kPairs><<<(unsigned)tiles_up(threads, 256), 256, 0, st>>>(p, join);
    return hipGetLastError();
}

} // namespace moe
