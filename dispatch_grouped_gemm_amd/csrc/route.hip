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
// floats do (-0 made +0 first), so ties are ties.
//
// Sixteen lanes share a token and hold its logits in registers: a reduction
// then takes four lane rotations inside a row of the wavefront, and four
// tokens share every instruction.  Bound by memory for many tokens, by
// launch latency for few.
#include "elem.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16; // of a token
constexpr int kMaxK = 8;
constexpr int kMaxPer = 64; // 16 lanes x 64: up to 1024 experts

// Value of the lane N places on in the same row of 16.
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, true);
}

template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f)
{
    v = f(v, ror<8>(v));
    v = f(v, ror<4>(v));
    v = f(v, ror<2>(v));
    return f(v, ror<1>(v));
}

__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    return row_reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

__device__ __forceinline__ uint32_t row_min(uint32_t v)
{
    return row_reduce(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

__device__ __forceinline__ float row_sum(float v)
{
    return __uint_as_float(row_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// Value of lane k of the same row of 16.
template <int k>
__device__ __forceinline__ uint32_t row_lane(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + k, 0xf, 0xf, true);
}

// exp(l - m) of a lane's logits in place (0 for -inf) and their sum; m the
// largest of the token.  The hardware exponential of (l - m) log2 e: off by
// |l - m| 2^-24 and an ulp, relatively.
template <int PER>
__device__ __forceinline__ float exps(float *l, float m)
{
    float s = 0.0f;
    if (__any(m == INFINITY)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            l[i] = __expf(l[i] == m ? 0.0f : l[i] - m);
            s += l[i];
        }
    } else {
        const float z = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            l[i] = __expf(l[i] - z);
            s += l[i];
        }
    }
    return s;
}

// Which expert register i of a lane holds: whole 16-byte pieces where the
// rows allow them (kVec), else single logits.
template <int DT, bool kVec>
__device__ __forceinline__ int expert_of(int i, int lane)
{
    constexpr int V = Elem<DT>::kVec;
    return kVec ? ((i / V) * kLanes + lane) * V + i % V : i * kLanes + lane;
}

// The lane that holds expert e (16 or more for e < 0), and its register.
template <int DT, bool kVec>
__device__ __forceinline__ int lane_of(int e)
{
    const int l = kVec ? e / Elem<DT>::kVec % kLanes : e % kLanes;
    return e < 0 ? kLanes : l;
}
template <int DT, bool kVec>
__device__ __forceinline__ int register_of(int e)
{
    constexpr int V = Elem<DT>::kVec;
    return kVec ? e / (V * kLanes) * V + e % V : e / kLanes;
}

// A token's logits; -inf past the last expert.
template <int DT, int PER, bool kVec>
__device__ __forceinline__ void load_logits(const void *logits, size_t row, int E, int lane,
                                            float *l)
{
    const auto *p = static_cast<const typename Elem<DT>::type *>(logits) + row * E;
    if constexpr (kVec) {
        constexpr int V = Elem<DT>::kVec;
#pragma unroll
        for (int j = 0; j < PER / V; ++j) {
            const int e = (j * kLanes + lane) * V;
            if (e < E) {
                Elem<DT>::unpack(*reinterpret_cast<const uint4 *>(p + e), l + j * V);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    l[j * V + i] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kLanes + lane;
            l[i] = e < E ? Elem<DT>::load(p + e) : -INFINITY;
        }
    }
}

template <int DT, int PER, bool kVec>
__global__ void __launch_bounds__(kThreads)
route_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
             int32_t *__restrict__ ids, float *__restrict__ w)
{
    const int lane = threadIdx.x & (kLanes - 1);
    const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= T)
        return; // a whole row of lanes
    float l[PER];
    load_logits<DT, PER, kVec>(logits, t, E, lane, l);
    // The ordering keys, a NaN as -inf; 0 once chosen.  A 16-bit logit's key
    // takes the high half and its expert, complemented, the low one: one
    // maximum finds the winner and settles ties.
    constexpr bool kWide = DT == MOE_DT_F32;
    // the largest key of a logit of -inf
    constexpr uint32_t kNone = kWide                  ? 0x007fffffu
                               : DT == MOE_DT_BF16 ? 0x007fffffu
                                                      : 0x03ffffffu;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        l[i] = fmaxf(l[i], -INFINITY); // the other operand of a NaN
        const float z = l[i] + 0.0f;
        if constexpr (DT == MOE_DT_F16) {
            const uint32_t b = Elem<MOE_DT_F16>::bits_of(z) << 16;
            key[i] = ((b ^ (uint32_t)((int32_t)b >> 31)) | (~b & 0x80000000u)) & 0xffff0000u;
        } else {
            const uint32_t b = __float_as_uint(z);
            key[i] = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
        }
        if constexpr (!kWide)
            key[i] = (key[i] & 0xffff0000u) | (0xffffu - expert_of<DT, kVec>(i, lane));
    }
    const auto value_of = [](uint32_t k) {
        if constexpr (kWide) {
            return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
        } else {
            const uint32_t b = k & 0x80000000u ? (k >> 16) & 0x7fffu : ~(k >> 16) & 0xffffu;
            return DT == MOE_DT_BF16 ? __uint_as_float(b << 16) : Elem<MOE_DT_F16>::half_of(b);
        }
    };
    float m = 0.0f, all = 0.0f, mine = 0.0f;
    int my_id = -1;
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            best = max(best, key[i]);
        const uint32_t won = row_max(best);
        const bool found = won > kNone;
        int e;
        if constexpr (kWide) {
            // the lane's first register of that key, then the lowest expert;
            // only that register of that lane is done with
            int at = PER;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                at = key[i] == won ? i : at;
            const uint32_t mine_e = at < PER ? (uint32_t)expert_of<DT, kVec>(at, lane) : ~0u;
            e = (int)row_min(mine_e);
            at = mine_e == (uint32_t)e ? at : PER;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = at == i ? 0u : key[i];
        } else {
            e = 0xffff - (int)(won & 0xffffu);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                key[i] = key[i] == won ? 0u : key[i];
        }
        const float v = value_of(won);
        if (k == 0) {
            m = v;
            if (!renorm) {
                all = row_sum(exps<PER>(l, m));
            }
        }
        if (lane == k && found) {
            mine = expf(v == m ? 0.0f : v - m);
            my_id = e;
        }
    }
    const float sum = renorm ? row_sum(mine) : all;
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        ids[o] = my_id;
        w[o] = my_id >= 0 ? mine / sum : 0.0f;
    }
}

template <int DT, int PER, bool kVec>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
                      const int32_t *__restrict__ ids, const float *__restrict__ w,
                      const float *__restrict__ dw, void *__restrict__ dlogits)
{
    constexpr int V = Elem<DT>::kVec;
    const int lane = threadIdx.x & (kLanes - 1);
    const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= T)
        return;
    // lane k: the slot k; no expert in the lanes past K
    int id = -1;
    float wk = 0.0f, g = 0.0f;
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        id = ids[o];
        if ((unsigned)id < (unsigned)E) {
            wk = w[o];
            g = dw[o];
        } else {
            id = -1;
        }
    }
    const float dot = row_sum(wk * g);
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        d[i] = 0.0f;
    // what slot k adds to its expert: w (g - dot), or g alone
    const float add = renorm ? wk * (g - dot) : g;
    // the slots whose expert this lane holds, and one of them a turn: a lane
    // rarely holds more than two, and a turn costs what a slot would
    uint32_t held = 0;
#define MOE_SLOT(k)                                                                              \
    held |= (uint32_t)(lane_of<DT, kVec>((int)row_lane<k>((uint32_t)id)) == lane) << k
    MOE_SLOT(0);
    MOE_SLOT(1);
    MOE_SLOT(2);
    MOE_SLOT(3);
    MOE_SLOT(4);
    MOE_SLOT(5);
    MOE_SLOT(6);
    MOE_SLOT(7);
#undef MOE_SLOT
    while (__any(held != 0)) {
        const int k = __ffs(held) - 1;
        const int e = __shfl(id, max(k, 0), kLanes);
        const float a = __shfl(add, max(k, 0), kLanes);
        const int at = k >= 0 ? register_of<DT, kVec>(e) : PER;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] += at == i ? a : 0.0f;
        held &= held - 1;
    }
    if (!renorm) {
        float l[PER];
        load_logits<DT, PER, kVec>(logits, t, E, lane, l);
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            l[i] = fmaxf(l[i], -INFINITY); // a NaN is not eligible
            m = fmaxf(m, l[i]);
        }
        m = __uint_as_float(row_reduce(__float_as_uint(m), [](uint32_t a, uint32_t b) {
            return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        }));
        const float s = row_sum(exps<PER>(l, m));
        const float r = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] = l[i] * r * (d[i] - dot);
    }
    auto *dl = static_cast<typename Elem<DT>::type *>(dlogits) + (size_t)t * E;
    if constexpr (kVec) {
#pragma unroll
        for (int j = 0; j < PER / V; ++j) {
            const int e = (j * kLanes + lane) * V;
            if (e < E)
                *reinterpret_cast<uint4 *>(dl + e) = Elem<DT>::pack(d + j * V);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kLanes + lane;
            if (e < E)
                Elem<DT>::store(dl + e, d[i]);
        }
    }
}

// Calls f with the smallest instantiated count of experts per lane.
template <typename F>
void per_lane(int E, F f)
{
    const int per = (E + kLanes - 1) / kLanes;
    if (per <= 8)
        f(std::integral_constant<int, 8>{});
    else if (per <= 16)
        f(std::integral_constant<int, 16>{});
    else if (per <= 24)
        f(std::integral_constant<int, 24>{});
    else if (per <= 32)
        f(std::integral_constant<int, 32>{});
    else
        f(std::integral_constant<int, kMaxPer>{});
}

// Whether the rows of E logits are whole 16-byte pieces on 16-byte borders.
bool whole_pieces(int E, int dtype, const void *p, const void *q)
{
    return E * elem_bytes(dtype) % 16 == 0 && (((uintptr_t)p | (uintptr_t)q) & 15) == 0;
}

unsigned grid_of(const moe_shape &s)
{
    constexpr unsigned per = kThreads / kLanes;
    return ((unsigned)s.T + per - 1) / per;
}

} // namespace

bool route_supported(const moe_shape &s) { return s.E_total <= kLanes * kMaxPer; }

hipError_t launch_route(const moe_shape &s, int dtype, bool renorm, const void *logits,
                        int32_t *ids, float *w, hipStream_t st)
{
    with_elem(dtype, [&](auto dt) {
        per_lane(s.E_total, [&](auto per) {
            constexpr int DT = decltype(dt)::value, PER = decltype(per)::value;
            const auto k = whole_pieces(s.E_total, dtype, logits, nullptr)
                               ? route_kernel<DT, PER, true>
                               : route_kernel<DT, PER, false>;
            k<<<grid_of(s), kThreads, 0, st>>>(s.T, s.E_total, s.K, renorm, logits, ids, w);
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
            constexpr int DT = decltype(dt)::value, PER = decltype(per)::value;
            const auto k = whole_pieces(s.E_total, dtype, logits, dlogits)
                               ? route_backward_kernel<DT, PER, true>
                               : route_backward_kernel<DT, PER, false>;
            k<<<grid_of(s), kThreads, 0, st>>>(s.T, s.E_total, s.K, renorm, logits, ids, w, dw,
                                               dlogits);
        });
    });
    return hipGetLastError();
}

} // namespace moe
