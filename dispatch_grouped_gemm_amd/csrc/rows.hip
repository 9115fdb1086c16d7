// Rows to their experts and back, with gradients, on the dispatch's route
// table route_row[T*K] (the row of slot (t, k), or -1):
//   permute             rows[route_row[t,k]] = x[t]
//   permute_backward    dx[t] = sum_k drows[route_row[t,k]]
//   unpermute           out[t] = sum_k w[t,k] rows[route_row[t,k]]
//   unpermute_backward  drows[route_row[t,k]] = w[t,k] dout[t],
//                       dw[t,k] = <dout[t], rows[route_row[t,k]]>
// All four walk the tokens: a token's row is read or written once however
// many experts it goes to, each of its expert rows once, and no two slots
// share a row, so there are no atomics and every sum has a fixed order.
// Sums are float32, k ascending, rounded once.
//
// Bound by memory, HBM bytes those of the formulas (within 2%).  8,192 tokens of
// 7,168 bf16 values and 6 experts each, from memory (three sets in turn): permute
// 156 us (822 MB, 5.3 TB/s), its gradient 150 (5.5), unpermute 150 (5.5), its
// gradients 314 (1.53 GB, 4.9); a large copy reaches 5.1.  128 tokens take 2.7 to
// 3.4 us, a launch.
#include "elem.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 8;

// Which 16-byte pieces of which token a thread takes (T H < 2^32, so there are
// fewer than 2^30).  One piece, wherever it lies; or (kPair) two, 64 apart, where
// a wavefront lies inside one token: its slots and weights are then read once
// per wavefront (scalar loads) and skipped slots by scalar branches.
//
// kPair is for ranks that hold few of the experts, where most slots go elsewhere
// and a thread's overhead counts; with many here single pieces keep more loads
// and stores in flight.  The sums take pairs up to half of the experts, the
// copies up to a quarter (us from memory, six sets of buffers in turn; K 6, even
// routing; single pieces, then pairs):
//   experts here             1/8           1/4           1/2           all
//   8,192 x 7,168 bf16
//     unpermute              63.3  41.9    70.0  54.9    89.8  87.2    149   154
//     permute                44.0  39.5    56.3  58.5    88.5  95.2    157   166
//   4,096 x 5,120 float32
//     unpermute                            49.0  39.0    63.7  62.5    106   109
//     permute                              40.1  40.0    61.8  66.1    110   116
struct Place {
    int t, p;
};
template <bool kPair>
__device__ __forceinline__ Place place_of(int T, int pieces)
{
    const unsigned i = blockIdx.x * kThreads + threadIdx.x;
    if constexpr (kPair) {
        const unsigned per = (unsigned)pieces / 128, wave = i >> 6;
        const int t = __builtin_amdgcn_readfirstlane((int)min(wave / per, (unsigned)T));
        return Place{t, (int)((wave - t * per) * 128 + (threadIdx.x & 63))};
    } else {
        const unsigned t = i / (unsigned)pieces;
        return Place{(int)t, (int)(i - t * (unsigned)pieces)};
    }
}

// The stores leave the L2 first: what these kernels write is large and read
// by another kernel, which would else find its own reads behind the lines
// still to be written (permute and its gradient, one after the other at 8,192
// tokens of 7,168 bf16 values and 6 experts each: 304 us, with ordinary
// stores 339; unpermute and its gradients 460, and 476).
__device__ __forceinline__ void store_piece(void *base, size_t piece, const uint4 &q)
{
    store_once(static_cast<uint4 *>(base) + piece, q);
}

// A thread stores its pieces of a token's row K times.
template <int DT, bool kPair>
__global__ void __launch_bounds__(kThreads)
permute_kernel(int T, int H, int K, long R, const void *__restrict__ x,
               const int32_t *__restrict__ route_row, void *__restrict__ rows)
{
    constexpr int P = kPair ? 2 : 1;
    const int pieces = H / Elem<DT>::kVec;
    const Place at = place_of<kPair>(T, pieces);
    if (at.t >= T)
        return;
    uint4 v[P];
#pragma unroll
    for (int j = 0; j < P; ++j)
        v[j] = static_cast<const uint4 *>(x)[(size_t)at.t * pieces + at.p + 64 * j];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        const int row = k < K ? checked_row(route_row[(size_t)at.t * K + k], R) : -1;
        if (row >= 0)
#pragma unroll
            for (int j = 0; j < P; ++j)
                store_piece(rows, (size_t)row * pieces + at.p + 64 * j, v[j]);
    }
}

// A thread sums its pieces of a token's expert rows: all loaded, then added
// in ascending k.
template <int DT, bool kPair, bool kWeights>
__global__ void __launch_bounds__(kThreads)
unpermute_kernel(int T, int H, int K, long R, const void *__restrict__ rows,
                 const float *__restrict__ w, const int32_t *__restrict__ route_row,
                 void *__restrict__ out)
{
#pragma clang fp contract(off)
    constexpr int V = Elem<DT>::kVec, P = kPair ? 2 : 1;
    const int pieces = H / V;
    const Place at = place_of<kPair>(T, pieces);
    if (at.t >= T)
        return;
    int row[kMaxK];
    float wk[kMaxK];
    uint4 q[kMaxK][P];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        row[k] = k < K ? checked_row(route_row[(size_t)at.t * K + k], R) : -1;
        wk[k] = kWeights && k < K ? w[(size_t)at.t * K + k] : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < kMaxK; ++k)
        if (row[k] >= 0)
#pragma unroll
            for (int j = 0; j < P; ++j)
                q[k][j] =
                    static_cast<const uint4 *>(rows)[(size_t)row[k] * pieces + at.p + 64 * j];
    float acc[P][V];
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[j][i] = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        if (row[k] < 0)
            continue;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float f[V];
            Elem<DT>::unpack(q[k][j], f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float pr = kWeights ? wk[k] * f[i] : f[i];
                acc[j][i] = acc[j][i] + pr;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
        store_piece(out, (size_t)at.t * pieces + at.p + 64 * j, Elem<DT>::pack(acc[j]));
}

// A workgroup takes one token: its dout row read once, its expert rows read
// for the weights' gradients (kDots) and their gradients written (kRows).  A
// piece of every expert row is loaded before the first is used: loaded and used
// in turn, 8,192 tokens of 2,560 bf16 values take 126 us instead of 114, the
// weights' gradients alone 71 instead of 55.  A thread writes a piece of drows
// after it has read the same piece of rows, and no other thread reads it: drows
// may be rows itself.
template <int DT, bool kRows, bool kDots, bool kWeights>
__global__ void __launch_bounds__(kThreads)
unpermute_backward_kernel(int T, int H, int K, long R, const void *__restrict__ dout,
                          const void *rows, const float *__restrict__ w,
                          const int32_t *__restrict__ route_row, void *drows,
                          float *__restrict__ dw)
{
    constexpr int V = Elem<DT>::kVec;
    __shared__ float part[kThreads / 64][kMaxK];
    const int pieces = H / V;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        int row[kMaxK];
        float wk[kMaxK], dot[kMaxK];
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
            row[k] = k < K ? checked_row(route_row[(size_t)t * K + k], R) : -1;
            wk[k] = kWeights && row[k] >= 0 ? w[(size_t)t * K + k] : 1.0f;
            dot[k] = 0.0f;
        }
        for (int p = threadIdx.x; p < pieces; p += kThreads) {
            uint4 q[kMaxK];
            const uint4 go = static_cast<const uint4 *>(dout)[(size_t)t * pieces + p];
            if (kDots)
#pragma unroll
                for (int k = 0; k < kMaxK; ++k)
                    if (row[k] >= 0)
                        q[k] = static_cast<const uint4 *>(rows)[(size_t)row[k] * pieces + p];
            float g[V];
            Elem<DT>::unpack(go, g);
#pragma unroll
            for (int k = 0; k < kMaxK; ++k) {
                if (row[k] < 0)
                    continue;
                const size_t at = (size_t)row[k] * pieces + p;
                if (kDots) {
                    float f[V];
                    Elem<DT>::unpack(q[k], f);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        dot[k] += g[j] * f[j];
                }
                if (kRows) {
                    float d[V];
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        d[j] = kWeights ? wk[k] * g[j] : g[j];
                    store_piece(drows, at, Elem<DT>::pack(d));
                }
            }
        }
        if (!kDots)
            continue;
#pragma unroll
        for (int k = 0; k < kMaxK; ++k) {
            float v = dot[k];
#pragma unroll
            for (int d = 32; d; d >>= 1)
                v += __shfl_xor(v, d);
            if (lane == 0)
                part[wave][k] = v;
        }
        __syncthreads();
        if ((int)threadIdx.x < K) {
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < kThreads / 64; ++u)
                v += part[u][threadIdx.x];
            dw[(size_t)t * K + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

// Calls f with whether threads take pairs of pieces, and the grid; `few`: pairs
// are for ranks that hold 1 / few of the experts or less.
template <typename F>
void with_place(const moe_shape &s, int dtype, int few, F f)
{
    const long pieces = s.H * (long)elem_bytes(dtype) / 16;
    const auto grid = [&](int P) {
        return (unsigned)((s.T * pieces / P + kThreads - 1) / kThreads);
    };
    if ((long)few * s.E_local <= s.E_total && pieces % 128 == 0)
        f(std::true_type{}, grid(2));
    else
        f(std::false_type{}, grid(1));
}

} // namespace

hipError_t launch_permute(const moe_shape &s, int dtype, const void *x, const int32_t *route_row,
                          void *rows, hipStream_t st)
{
    const long R = moe_row_capacity(&s);
    with_place(s, dtype, 4, [&](auto pair, unsigned grid) {
        constexpr bool kPair = decltype(pair)::value;
        // a copy: both 16-bit types alike
        const auto k = dtype == MOE_DT_F32 ? permute_kernel<MOE_DT_F32, kPair>
                                           : permute_kernel<MOE_DT_BF16, kPair>;
        k<<<grid, kThreads, 0, st>>>(s.T, s.H, s.K, R, x, route_row, rows);
    });
    return hipGetLastError();
}

hipError_t launch_unpermute(const moe_shape &s, int dtype, const void *rows, const float *w,
                            const int32_t *route_row, void *out, hipStream_t st)
{
    const long R = moe_row_capacity(&s);
    with_elem(dtype, [&](auto dt) {
        with_place(s, dtype, 2, [&](auto pair, unsigned grid) {
            constexpr int DT = decltype(dt)::value;
            constexpr bool kPair = decltype(pair)::value;
            const auto k = w ? unpermute_kernel<DT, kPair, true> : unpermute_kernel<DT, kPair, false>;
            k<<<grid, kThreads, 0, st>>>(s.T, s.H, s.K, R, rows, w, route_row, out);
        });
    });
    return hipGetLastError();
}

hipError_t launch_unpermute_backward(const moe_shape &s, int dtype, const void *dout,
                                     const void *rows, const float *w, const int32_t *route_row,
                                     void *drows, float *dw, hipStream_t st)
{
    const long R = moe_row_capacity(&s);
    with_elem(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const auto go = [&](auto kernel) {
            kernel<<<min(s.T, 1 << 20), kThreads, 0, st>>>(s.T, s.H, s.K, R, dout, rows, w,
                                                           route_row, drows, dw);
        };
        if (drows && dw)
            go(w ? unpermute_backward_kernel<DT, true, true, true>
                 : unpermute_backward_kernel<DT, true, true, false>);
        else if (drows)
            go(w ? unpermute_backward_kernel<DT, true, false, true>
                 : unpermute_backward_kernel<DT, true, false, false>);
        else
            go(unpermute_backward_kernel<DT, false, true, false>);
    });
    return hipGetLastError();
}

} // namespace moe
