// The router: each token's K experts and their weights from its logits, and
// the logits' gradient.
//
// Forward, per token: the eligible logits are those above -inf (NaN is not);
// the K largest are chosen, equal ones by the lower expert id, in falling
// order; with m the largest,
//   w_k = exp(l_k - m) / sum exp(l_j - m),
// the sum over the chosen (renormalize) or over every eligible expert.  A
// logit equal to m counts exp(0) = 1, also where m is +inf.  Slots left over
// (fewer eligible experts than K) get id -1 and weight 0.
// Backward: with p the weights' softmax (over the chosen, or all) and g_e
// the gradient of expert e's weight (0 where it was not chosen),
//   dl_e = p_e (g_e - sum_k w_k g_k).
//
// Choosing is exact: a logit becomes a whole number that orders as the
// floats do (-0 made +0 first), so ties are ties.  Bound by memory for many
// tokens, by launch latency for few.
#include "elem.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 8;
constexpr int kMaxPer = 16; // 64 lanes x 16: up to 1024 experts

// Order-preserving whole number of an eligible logit (never 0); 0 for -inf
// and NaN.
__device__ __forceinline__ uint32_t key_of(float v)
{
    if (!(v > -INFINITY))
        return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float exp_to_max(float v, float m)
{
    return expf(v == m ? 0.0f : v - m);
}

__device__ __forceinline__ float wave_sum_f(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// One wavefront per token, expert e in lane e mod 64.
template <int DT, int PER>
__global__ void __launch_bounds__(kThreads)
route_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
             int32_t *__restrict__ ids, float *__restrict__ w)
{
    const int t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= T)
        return;
    const auto *l = static_cast<const typename Elem<DT>::type *>(logits) + (size_t)t * E;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        key[i] = e < E ? key_of(Elem<DT>::load(l + e)) : 0u;
    }
    float all = 0.0f, m = 0.0f, mine = 0.0f, sum = 0.0f;
    int my_id = -1;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * 64 + lane;
            }
        uint64_t b = ((uint64_t)best << 32) | (uint32_t)~at;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)b, d);
            b = o > b ? o : b;
        }
        const uint32_t won = (uint32_t)(b >> 32);
        if (won == 0u)
            break;
        const int e = (int)~(uint32_t)b;
        const float v = value_of(won);
        if (k == 0) {
            m = v;
            if (!renorm) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (key[i])
                        s += exp_to_max(value_of(key[i]), m);
                all = wave_sum_f(s);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == i * 64 + lane)
                key[i] = 0u;
        const float ek = exp_to_max(v, m);
        sum += ek;
        if (lane == k) {
            mine = ek;
            my_id = e;
        }
    }
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        ids[o] = my_id;
        w[o] = my_id >= 0 ? mine / (renorm ? sum : all) : 0.0f;
    }
}

template <int DT, int PER>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
                      const int32_t *__restrict__ ids, const float *__restrict__ w,
                      const float *__restrict__ dw, void *__restrict__ dlogits)
{
    const int t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= T)
        return;
    int id[kMaxK];
    float wk[kMaxK], g[kMaxK], dot = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        const size_t o = (size_t)t * K + k;
        id[k] = k < K ? ids[o] : -1;
        if ((unsigned)id[k] >= (unsigned)E)
            id[k] = -1;
        wk[k] = id[k] >= 0 ? w[o] : 0.0f;
        g[k] = id[k] >= 0 ? dw[o] : 0.0f;
        dot += wk[k] * g[k];
    }
    auto *dl = static_cast<typename Elem<DT>::type *>(dlogits) + (size_t)t * E;
    if (renorm) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 64 + lane;
            float d = 0.0f;
#pragma unroll
            for (int k = 0; k < kMaxK; ++k)
                if (id[k] == e)
                    d += wk[k] * (g[k] - dot);
            if (e < E)
                Elem<DT>::store(dl + e, d);
        }
        return;
    }
    const auto *l = static_cast<const typename Elem<DT>::type *>(logits) + (size_t)t * E;
    float v[PER], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        v[i] = e < E ? Elem<DT>::load(l + e) : -INFINITY;
        if (v[i] > m)
            m = v[i];
    }
#pragma unroll
    for (int d = 32; d; d >>= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = v[i] > -INFINITY ? exp_to_max(v[i], m) : 0.0f;
        s += v[i];
    }
    s = wave_sum_f(s);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        float ge = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
            if (id[k] == e)
                ge += g[k];
        if (e < E)
            Elem<DT>::store(dl + e, v[i] > 0.0f ? v[i] / s * (ge - dot) : 0.0f);
    }
}

// Calls f with the smallest instantiated count of experts per lane.
template <typename F>
void per_lane(int E, F f)
{
    const int per = (E + 63) / 64;
    if (per <= 2)
        f(std::integral_constant<int, 2>{});
    else if (per <= 4)
        f(std::integral_constant<int, 4>{});
    else if (per <= 8)
        f(std::integral_constant<int, 8>{});
    else
        f(std::integral_constant<int, kMaxPer>{});
}

unsigned grid_of(const moe_shape &s) { return ((unsigned)s.T + 3) / 4; }

} // namespace

bool route_supported(const moe_shape &s) { return s.E_total <= 64 * kMaxPer; }

hipError_t launch_route(const moe_shape &s, int dtype, bool renorm, const void *logits,
                        int32_t *ids, float *w, hipStream_t st)
{
    with_elem(dtype, [&](auto dt) {
        per_lane(s.E_total, [&](auto per) {
            route_kernel<decltype(dt)::value, decltype(per)::value>
                <<<grid_of(s), kThreads, 0, st>>>(s.T, s.E_total, s.K, renorm, logits, ids, w);
        });
    });
    return hipGetLastError();
}

hipError_t launch_route_backward(const moe_shape &s, int dtype, bool renorm, const void *logits,
                                 const int32_t *ids, const float *w, const float *dw,
                                 void *dlogits, hipStream_t st)
{
    with_elem(dtype, [&](auto dt) {
        per_lane(s.E_total, [&](auto per) {
            route_backward_kernel<decltype(dt)::value, decltype(per)::value>
                <<<grid_of(s), kThreads, 0, st>>>(s.T, s.E_total, s.K, renorm, logits, ids, w, dw,
                                                  dlogits);
        });
    });
    return hipGetLastError();
}

} // namespace moe
