// The dense feed-forward block's parts that its forward and backward launches
// share: the activation and its gradient, what a lane does with 8 neighbouring
// sums, the tile kernels, and the join of K's parts.
#pragma once

#include "ffn_plan.hpp"
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

// 8 (or 4) neighbouring values of a 16-bit row, or of an MX FP8 one.
template <int DT>
__device__ __forceinline__ void store8(uint16_t *p, const float *f)
{
    *reinterpret_cast<uint4 *>(p) = Elem<DT>::pack(f);
}

template <int DT>
__device__ __forceinline__ void store4(uint16_t *p, const v4f &v)
{
    const float f[8] = {v[0], v[1], v[2], v[3], 0.0f, 0.0f, 0.0f, 0.0f};
    const uint4 q = Elem<DT>::pack(f);
    *reinterpret_cast<uint2 *>(p) = uint2{q.x, q.y};
}

// (an exponent byte of 255 is NaN: the codes of NaN then, whatever the exponent)
__device__ __forceinline__ void from_mx(const uint2 &codes, uint32_t scale, float *f)
{
    const int e = (int)scale - 127;
    const uint32_t nan = scale == 255 ? 0x7f7f7f7fu : 0u;
    const uint32_t w[2] = {codes.x | nan, codes.y | nan};
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
// lanes D, 2 D and 3 D further (xor).  An infinity or NaN becomes the code of a
// NaN and has no part in the block's exponent, so it is not lost between the passes.
template <int D>
__device__ __forceinline__ void store8_mx(uint8_t *codes, uint8_t *scale, const float *f, bool first)
{
    const auto block = [](float v) {
        v = fmaxf(v, __shfl_xor(v, D));
        return fmaxf(v, __shfl_xor(v, 2 * D));
    };
    float amax = 0.0f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, fabsf(f[i]));
        sum += f[i] - f[i]; // 0, or NaN
    }
    uint32_t lost[2] = {0, 0};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = f[i];
    if (__any(sum != 0.0f))
        amax = mx8_finite<8>(f, v, lost);
    amax = block(amax);
    const int e = mx8_block_exponent(amax);
    *reinterpret_cast<uint2 *>(codes) =
        uint2{mx8_pack4(v[0], v[1], v[2], v[3], e, amax) | lost[0],
              mx8_pack4(v[4], v[5], v[6], v[7], e, amax) | lost[1]};
    if (first)
        *scale = (uint8_t)(e + 127);
}

// What a lane does with 8 neighbouring columns of a row once their sums are
// complete.  Pre is what it reads for them, fetched for several rows ahead.

// h = silu(min(g, gl)) clamp(u, ul) of 8 columns j .. j + 7 of row t, from the
// float32 sums; D: lane distance of a block's four pieces.
template <int DT, int D>
struct Activate {
    int I;
    float gl, ul;
    Kept kept;
    uint16_t *h;

    struct Pre {};
    __device__ __forceinline__ void fetch(long, int, Pre *) const {}
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
        for (int i = 0; i < 8; ++i)
            v[i] = one(g[i], u[i]);
        // h is rounded once to the type: the second product's operand
        store8<DT>(h + t * I + j, v);
    }
    __device__ __forceinline__ float one(float g, float u) const
    {
        const float gc = not_above(g, gl);
        return gc * logistic(gc) * between(u, ul);
    }
    // four columns; kept in the elements' type or not at all
    __device__ __forceinline__ void four(long t, int j, const v4f &g, const v4f &u) const
    {
        if (kept.rows) {
            uint16_t *r = static_cast<uint16_t *>(kept.rows) + t * 2 * I + j;
            store4<DT>(r, g);
            store4<DT>(r + I, u);
        }
        store4<DT>(h + t * I + j,
                   v4f{one(g[0], u[0]), one(g[1], u[1]), one(g[2], u[2]), one(g[3], u[3])});
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

    struct Pre {
        uint4 g, u; // 16-bit rows; MX FP8: 8 codes in x and y, the exponent in z
    };
    __device__ __forceinline__ void fetch(long t, int j, Pre *p) const
    {
        const long at = t * 2 * I + j;
        if (kept.scale) {
            const uint8_t *c = static_cast<const uint8_t *>(kept.rows) + at;
            const uint8_t *s = kept.scale + at / 32;
            const uint2 g = *reinterpret_cast<const uint2 *>(c);
            const uint2 u = *reinterpret_cast<const uint2 *>(c + I);
            p->g = uint4{g.x, g.y, s[0], 0};
            p->u = uint4{u.x, u.y, s[I / 32], 0};
        } else {
            const uint16_t *r = static_cast<const uint16_t *>(kept.rows) + at;
            p->g = *reinterpret_cast<const uint4 *>(r);
            p->u = *reinterpret_cast<const uint4 *>(r + I);
        }
    }
    __device__ __forceinline__ void operator()(long t, int j, const float *dh, const Pre &p) const
    {
        float g[8], u[8], v[8];
        if (kept.scale) {
            from_mx(uint2{p.g.x, p.g.y}, p.g.z, g);
            from_mx(uint2{p.u.x, p.u.y}, p.u.z, u);
        } else {
            Elem<DT>::unpack(p.g, g);
            Elem<DT>::unpack(p.u, u);
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
        const long at = t * 2 * I + j;
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

    struct Pre {
        uint4 base;
    };
    __device__ __forceinline__ void fetch(long m, int n, Pre *p) const
    {
        if (base)
            p->base = *reinterpret_cast<const uint4 *>(base + m * ld + n);
    }
    __device__ __forceinline__ void operator()(long m, int n, const float *f, const Pre &p) const
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
            Elem<DT>::unpack(p.base, b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += b[i];
        }
        store_once(out + at, Elem<DT>::pack(v));
    }
    // four columns of a 16-bit row
    __device__ __forceinline__ void four(long m, int n, v4f v) const
    {
        const long at = m * ld + n;
        if (base)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] += Elem<DT>::load(base + at + i);
        store4<DT>(out + at, v);
    }
};

// A product's sizes and operands: C [M, N] over K; tiles tm x tn, K in
// `splits` parts.
struct Product {
    Operand a, b;
    long M, K;
    int N, tm, tn, splits;
    float *parts; // [splits][M][N]: a part's sums, to be joined
};

// The part's steps and the tile's sums.  kPairs: b's rows are W13's 2I and a
// wavefront's columns half gate, half up of the same I.
template <typename T, bool kPairs, bool ADOWN, bool BDOWN>
__device__ __forceinline__ void tile_sums(T &tile, const Product &p, long m0, int n0, int part,
                                          uint8_t *lds)
{
    const int I = p.N / 2;
    const int steps = (int)((p.K + 63) / 64);
    const int first = (int)((long)steps * part / p.splits);
    const int end = (int)((long)steps * (part + 1) / p.splits);
    constexpr int W = 16 * T::NF; // columns of a wavefront
    tile.run(
        lds, p.a, [&](int i) { return min(m0 + i, p.M - 1); }, m0, p.M, p.b,
        [&](int i) -> long {
            const int b = (i % W) >> 4;
            if (!kPairs)
                return min(n0 + i / W * W + tile_column(b, i & 15), p.N - 1);
            return (b >> 1) * (long)I +
                   min(n0 + i / W * 32 + tile_column(b & 1, i & 15), I - 1);
        },
        n0, p.N, p.K, first, end - first);
}

// A lane's 8 columns of block pair h in a row block's sums.
__device__ __forceinline__ void eight(const v4f *acc, int h, float *v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = acc[2 * h][i];
        v[4 + i] = acc[2 * h + 1][i];
    }
}

// One tile of C, whole K, through the functor.
template <typename T, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__device__ __forceinline__ void whole_tile(const Product &p, const F &f, long m0, int in,
                                           uint8_t *lds)
{
    static_assert(!kPairs || T::NF == 4, "two blocks of gates, two of up");
    const int n0 = in * (kPairs ? T::kBN / 2 : T::kBN);
    T tile;
    tile_sums<T, kPairs, ADOWN, BDOWN>(tile, p, m0, n0, 0, lds);
    const int lane = threadIdx.x & 63, wave = tile_wave();
    const int wm = wave / T::kWN, wn = wave % T::kWN;
    const long row0 = m0 + wm * T::MF * 16 + (lane & 15);
    if constexpr (kPairs) {
        const int n = n0 + 32 * wn + 8 * (lane >> 4);
        if (n >= p.N / 2)
            return;
#pragma unroll
        for (int m = 0; m < T::MF; ++m) {
            float g[8], u[8];
            eight(tile.acc[m], 0, g);
            eight(tile.acc[m], 1, u);
            if (row0 + 16 * m < p.M)
                f(row0 + 16 * m, n, g, u);
        }
    } else {
        // what a row block needs is fetched GM blocks ahead of it: its loads would
        // otherwise wait for the stores before them
        constexpr int NH = T::NF / 2;
        const int n = n0 + 16 * T::NF * wn + 8 * (lane >> 4);
        typename F::Pre pre[T::GM][NH];
        const auto fetch = [&](int m) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
                if (n + 32 * h < p.N)
                    f.fetch(min(row0 + 16 * m, p.M - 1), n + 32 * h, &pre[m % T::GM][h]);
        };
#pragma unroll
        for (int m = 0; m < T::GM; ++m)
            fetch(m);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < T::MF; ++m) {
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                float v[8];
                eight(tile.acc[m], h, v);
                if (row0 + 16 * m < p.M && n + 32 * h < p.N)
                    f(row0 + 16 * m, n + 32 * h, v, pre[m % T::GM][h]);
            }
            if (m + T::GM < T::MF)
                fetch(m + T::GM);
        }
    }
}

// The tiles there are; what each costs: product_cost (ffn_plan.hpp).  Where B's k lies
// down its rows, its transpose reads run at half the rate of A's: wavefronts then share
// B's columns among two rows of them, not four (dh, two rows and four, us: 1,021 x 1,408
// over 2,304 by 64 x 128 16.5 and 18.2, by 128 x 128 22.2 and 23.4; 4,096 x 2,304 over
// 5,120 by 128 x 128 152 and 156, by 192 x 128 127 and 122).
template <int DT, bool ADOWN, bool BDOWN>
struct Tiles {
    static constexpr int WM = BDOWN ? 2 : 4, WN = 8 / WM;
    using Huge = Tile<DT, 256, 256, 2, 4, 2, ADOWN, BDOWN>;
    using Tall = Tile<DT, 192, 256, 2, 4, 2, ADOWN, BDOWN>; // this and Slim: k along A's rows
    using Wide = Tile<DT, 128, 256, 2, 4, 3, ADOWN, BDOWN>;
    using Slim = Tile<DT, 192, 128, WM, WN, 4, ADOWN, BDOWN>;
    using Even = Tile<DT, 128, 128, WM, WN, 4, ADOWN, BDOWN>;
    using Flat = Tile<DT, 64, 128, WM, WN, 4, ADOWN, BDOWN>;
    using Small = Tile<DT, 64, 64, 4, 2, 4, ADOWN, BDOWN>;
    using Few = Tile<DT, 32, 64, 2, 2, 6, ADOWN, BDOWN>;
};

template <typename T, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__global__ void __launch_bounds__(T::kThreads, 1) product_kernel(Product p, F f)
{
    __shared__ __align__(1024) uint8_t lds[T::kLds];
    int im, in;
    tile_place(tile_run(blockIdx.x, gridDim.x), p.tm, p.tn, &im, &in);
    whole_tile<T, kPairs, ADOWN, BDOWN>(p, f, (long)im * T::kBM, in, lds);
}

// `whole` tiles of 256 x 256, and behind them those left over, which would leave CUs
// idle for a tile's time, as kCut smaller tiles TL each.  (Some of the small ones first,
// so that the CUs' epilogues are out of step: 8,191 x 7,168 over 2,048 then reads 828 MB
// past the L2s, not 525, since tiles that share rows no longer ask for them together,
// and takes as long.)
template <typename T, typename TL, bool kPairs, bool ADOWN, bool BDOWN, typename F>
__global__ void __launch_bounds__(T::kThreads, 1) product_rest_kernel(Product p, int whole, F f)
{
    constexpr int kMost = TL::kLds > T::kLds ? TL::kLds : T::kLds;
    constexpr int kDownward = T::kBM / TL::kBM, kCut = kDownward * (T::kBN / TL::kBN);
    __shared__ __align__(1024) uint8_t lds[kMost];
    const int b = blockIdx.x;
    int im, in;
    if (b < whole) {
        tile_place(tile_run(b, whole), p.tm, p.tn, &im, &in);
        whole_tile<T, kPairs, ADOWN, BDOWN>(p, f, (long)im * T::kBM, in, lds);
        return;
    }
    const int h = tile_run(b - whole, gridDim.x - whole), part = h % kCut;
    tile_place(whole + h / kCut, p.tm, p.tn, &im, &in);
    const long m0 = (long)im * T::kBM + part % kDownward * TL::kBM;
    in = in * (T::kBN / TL::kBN) + part / kDownward;
    if (m0 < p.M && in * (kPairs ? TL::kBN / 2 : TL::kBN) < (kPairs ? p.N / 2 : p.N))
        whole_tile<TL, kPairs, ADOWN, BDOWN>(p, f, m0, in, lds);
}

// One of `splits` parts of K of a tile, as float32 sums in its plane.
template <typename T, bool ADOWN, bool BDOWN>
__global__ void __launch_bounds__(T::kThreads, 1) parts_kernel(Product p)
{
    __shared__ __align__(1024) uint8_t lds[T::kLds];
    const int tiles = p.tm * p.tn, q = tile_run(blockIdx.x, tiles * p.splits);
    const int part = q / tiles;
    int im, in;
    tile_place(q - part * tiles, p.tm, p.tn, &im, &in);
    T tile;
    tile_sums<T, false, ADOWN, BDOWN>(tile, p, (long)im * T::kBM, in * T::kBN, part, lds);
    const int lane = threadIdx.x & 63, wave = tile_wave();
    const int wm = wave / T::kWN, wn = wave % T::kWN;
    const int n = in * T::kBN + 16 * T::NF * wn + 8 * (lane >> 4);
#pragma unroll
    for (int m = 0; m < T::MF; ++m) {
        const long row = (long)im * T::kBM + (wm * T::MF + m) * 16 + (lane & 15);
        if (row >= p.M)
            continue;
        v4f *o = reinterpret_cast<v4f *>(p.parts + ((long)part * p.M + row) * p.N + n);
#pragma unroll
        for (int h = 0; h < T::NF / 2; ++h)
            if (n + 32 * h < p.N) {
                o[8 * h] = tile.acc[m][2 * h];
                o[8 * h + 1] = tile.acc[m][2 * h + 1];
            }
    }
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
    typename F::Pre pre;
    f.fetch(row, n, &pre);
    float v[2][8];
    constexpr int S = kPairs ? 2 : 1;
    v4f part[S][2][kMostParts];
#pragma unroll
    for (int s = 0; s < kMostParts; ++s)
#pragma unroll
        for (int h = 0; h < S; ++h)
            if (s < p.splits) {
                const v4f *o = reinterpret_cast<const v4f *>(p.parts + (s * p.M + row) * p.N + n +
                                                             h * (p.N / 2));
                part[h][0][s] = o[0];
                part[h][1][s] = o[1];
            }
#pragma unroll
    for (int h = 0; h < S; ++h) {
        v4f lo = part[h][0][0], hi = part[h][1][0];
#pragma unroll
        for (int s = 1; s < kMostParts; ++s)
            if (s < p.splits) {
                lo += part[h][0][s];
                hi += part[h][1][s];
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
        f(row, n, v[0], pre);
}

// Launches a product; join: the functor with the lane distance of the join
// kernel.
template <int DT, bool kPairs, bool ADOWN, bool BDOWN, typename F, typename J>
hipError_t launch_product(Product p, const Cut &c, const F &f, const J &join, float *parts,
                          hipStream_t st)
{
    using S = Tiles<DT, ADOWN, BDOWN>;
    p.tm = (int)tiles_down(c.kind, p.M);
    p.tn = (int)tiles_across(c.kind, p.N);
    p.splits = c.splits;
    p.parts = parts;
    const int n = p.tm * p.tn;
    const auto whole = [&](auto t) {
        using T = decltype(t);
        product_kernel<T, kPairs, ADOWN, BDOWN><<<n, T::kThreads, 0, st>>>(p, f);
    };
    const auto part = [&](auto t) {
        using T = decltype(t);
        parts_kernel<T, ADOWN, BDOWN><<<n * c.splits, T::kThreads, 0, st>>>(p);
    };
    if (c.splits > 1) {
        if (c.kind == kEven)
            part(typename S::Even{});
        else if (c.kind == kFlat)
            part(typename S::Flat{});
        else if (c.kind == kSmall)
            part(typename S::Small{});
        else
            part(typename S::Few{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        const long threads = p.M * ((kPairs ? p.N / 2 : p.N) / 8);
        join_kernel<kPairs><<<(unsigned)tiles_up(threads, 256), 256, 0, st>>>(p, join);
        return hipGetLastError();
    }
    const auto rest = [&](auto t) {
        using L = decltype(t);
        const int left = n % kTileCus, small = huge_rest(n) * left;
        product_rest_kernel<typename S::Huge, L, kPairs, ADOWN, BDOWN>
            <<<n - left + small, 512, 0, st>>>(p, n - left, f);
    };
    if (c.kind == kHuge && huge_rest(n) == 2) {
        rest(typename S::Wide{});
    } else if (c.kind == kHuge && huge_rest(n) == 4) {
        rest(typename S::Even{});
    } else if (c.kind == kHuge) {
        whole(typename S::Huge{});
    } else if (c.kind == kTall) {
        whole(typename S::Tall{});
    } else if (c.kind == kSlim) {
        whole(typename S::Slim{});
    } else if (c.kind == kWide) {
        whole(typename S::Wide{});
    } else if (c.kind == kEven) {
        whole(typename S::Even{});
    } else if (c.kind == kFlat) {
        whole(typename S::Flat{});
    } else if constexpr (!kPairs) {
        if (c.kind == kSmall)
            whole(typename S::Small{});
        else
            whole(typename S::Few{});
    }
    return hipGetLastError();
}

} // namespace moe
