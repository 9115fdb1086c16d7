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
// tokens share every instruction.
//
// Measured at 65,536 tokens of 384 experts, 6 chosen, the softmax over all, from
// memory (four sets of inputs in turn): bf16 22 us forward (50 MB read;
// instructions bound it) and 22 backward (100 MB read and written at 4.5 TB/s),
// float32 32 and 33 (6.1 TB/s); renormalized 20 and 15, 33 and 18.  Of 512 experts
// 23 and 18; of 1,024, 8 chosen, 42 and 31 (from 513 on a lane holds 64 logits).
// Few tokens are bound by launch latency: 128 take 3.9 us, 8,192 in float32 7.8
// and 5.1.
#include "elem.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16; // of a token
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

// What the wavefront wrote to LDS before is what it reads behind.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

// The same of a 16-bit type as they are, registers 2 i and 2 i + 1 in dword i.
template <int DT, int PER, bool kVec>
__device__ __forceinline__ void load_pairs(const void *logits, size_t row, int E, int lane,
                                           uint32_t *b)
{
    constexpr uint32_t kNegInf = DT == MOE_DT_BF16 ? 0xff80u : 0xfc00u;
    const uint16_t *p = static_cast<const uint16_t *>(logits) + row * E;
    if constexpr (kVec) {
#pragma unroll
        for (int j = 0; j < PER / 8; ++j) {
            const int e = (j * kLanes + lane) * 8;
            uint4 q = {kNegInf * 0x10001u, kNegInf * 0x10001u, kNegInf * 0x10001u,
                       kNegInf * 0x10001u};
            if (e < E)
                q = *reinterpret_cast<const uint4 *>(p + e);
            b[4 * j] = q.x;
            b[4 * j + 1] = q.y;
            b[4 * j + 2] = q.z;
            b[4 * j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER / 2; ++i) {
            const int e = 2 * i * kLanes + lane, f = e + kLanes;
            b[i] = (e < E ? p[e] : kNegInf) | (f < E ? p[f] : kNegInf) << 16;
        }
    }
}

// Numbers that order as two 16-bit logits do, side by side: the sign and the
// magnitude as a two's complement (-0 and +0 the same), moved up until the
// positive NaNs wrap to below -inf, where the negative ones are.
template <int DT>
struct Order16 {
    static constexpr uint32_t kUp = 0x8000u + (DT == MOE_DT_BF16 ? 0x7fu : 0x3ffu);
    // that of -inf
    static constexpr uint32_t kNone = kUp - (DT == MOE_DT_BF16 ? 0x7f80u : 0x7c00u);
    static __device__ __forceinline__ uint32_t of(uint32_t pair)
    {
        typedef uint16_t u2v __attribute__((ext_vector_type(2)));
        typedef int16_t s2v __attribute__((ext_vector_type(2)));
        const u2v sign = __builtin_bit_cast(u2v, __builtin_bit_cast(s2v, pair) >> (int16_t)15);
        const u2v size = __builtin_bit_cast(u2v, pair) & (uint16_t)0x7fff;
        return __builtin_bit_cast(uint32_t, (size ^ sign) - sign + (uint16_t)kUp);
    }
    static __device__ __forceinline__ float value(uint32_t number)
    {
        const int v = (int)number - (int)kUp;
        const uint32_t b = (uint32_t)(v < 0 ? 0x8000 - v : v);
        if constexpr (DT == MOE_DT_BF16)
            return __uint_as_float(b << 16);
        else
            return Elem<MOE_DT_F16>::half_of(b);
    }
};

// One of the two logits of a dword.
template <int DT>
__device__ __forceinline__ float half_pair(uint32_t pair, int high)
{
    if constexpr (DT == MOE_DT_BF16)
        return __uint_as_float(high ? pair & 0xffff0000u : pair << 16);
    else
        return Elem<MOE_DT_F16>::half_of(high ? pair >> 16 : pair);
}

// Writes a token's slots; `all` is the sum over every eligible expert, used
// unless renorm.
__device__ __forceinline__ void store_slots(int t, int K, int lane, bool renorm, float all,
                                            int my_id, float mine, int32_t *ids, float *w)
{
    const float sum = renorm ? row_sum(mine) : all;
    if (lane < K) {
        const size_t o = (size_t)t * K + lane;
        ids[o] = my_id;
        w[o] = my_id >= 0 ? mine / sum : 0.0f;
    }
}

// The second of three in order, v_med3_u32 where a >= b.
__device__ __forceinline__ uint32_t middle(uint32_t a, uint32_t b, uint32_t c)
{
    return max(min(a, b), min(max(a, b), c));
}

// Puts a key among the three largest, in falling order.
__device__ __forceinline__ void keep(uint32_t (&top)[3], uint32_t key)
{
    top[2] = middle(top[1], top[2], key);
    top[1] = middle(top[0], top[1], key);
    top[0] = max(top[0], key);
}

// 16-bit logits.  A logit's key is its number in the high half and its
// expert, complemented, in the low one: no two are alike, none is 0, and a
// maximum finds the winner and settles ties.  A lane keeps its three largest
// keys that are still to be chosen (three instructions a key, once), so that
// a round is one maximum over the 16 lanes; a lane that has given all three
// looks through its keys again, below the last winner.  (65,536 tokens, inputs in
// the cache: with a maximum over every key in each round 6 of 384 bf16 experts
// took 25 us, so 20; float32 33 and 26.)
template <int DT, int PER, bool kVec>
__global__ void __launch_bounds__(kThreads)
route_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
             int32_t *__restrict__ ids, float *__restrict__ w)
{
    const int lane = threadIdx.x & (kLanes - 1);
    const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= T)
        return; // a whole row of lanes
    uint32_t b[PER / 2], key[PER];
    load_pairs<DT, PER, kVec>(logits, t, E, lane, b);
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
        const uint32_t n = Order16<DT>::of(b[i / 2]);
        key[i] = n << 16 | (0xffffu - expert_of<DT, kVec>(i, lane));
        key[i + 1] = (n & 0xffff0000u) | (0xffffu - expert_of<DT, kVec>(i + 1, lane));
    }
    float m = 0.0f, all = 0.0f, mine = 0.0f;
    int my_id = -1;
    uint32_t top[3] = {0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < PER; ++i)
        keep(top, key[i]);
    for (int k = 0; k < K; ++k) {
        const uint32_t won = row_max(top[0]);
        const bool gave = top[0] == won;
        top[0] = gave ? top[1] : top[0];
        top[1] = gave ? top[2] : top[1];
        top[2] = gave ? 0u : top[2];
        if (k + 1 < K && __any(top[0] == 0u)) {
            top[0] = top[1] = top[2] = 0u;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                keep(top, key[i] < won ? key[i] : 0u);
        }
        const float v = Order16<DT>::value(won >> 16);
        if (k == 0) {
            m = v;
            if (!renorm) {
                float l[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) // the other operand of a NaN
                    l[i] = fmaxf(half_pair<DT>(b[i / 2], i & 1), -INFINITY);
                all = row_sum(exps<PER>(l, m));
            }
        }
        if (lane == k && won >> 16 > Order16<DT>::kNone) {
            mine = expf(v == m ? 0.0f : v - m);
            my_id = 0xffff - (int)(won & 0xffffu);
        }
    }
    store_slots(t, K, lane, renorm, all, my_id, mine, ids, w);
}

// float32 logits: a key is a whole number that orders as the logit does, a
// NaN's that of -inf; equal ones go by the expert.  A lane keeps its three
// first, by key and expert, as above.
struct Chosen {
    uint32_t key[3];
    int e[3];
};

// The lane's keys come with rising experts, so an equal one goes behind.
__device__ __forceinline__ void keep(Chosen &c, uint32_t key, int e)
{
    const bool b0 = key > c.key[0], b1 = key > c.key[1], b2 = key > c.key[2];
    c.e[2] = b1 ? c.e[1] : b2 ? e : c.e[2];
    c.e[1] = b0 ? c.e[0] : b1 ? e : c.e[1];
    c.e[0] = b0 ? e : c.e[0];
    c.key[2] = middle(c.key[1], c.key[2], key);
    c.key[1] = middle(c.key[0], c.key[1], key);
    c.key[0] = max(c.key[0], key);
}

template <int PER, bool kVec>
__global__ void __launch_bounds__(kThreads)
route_f32_kernel(int T, int E, int K, bool renorm, const void *__restrict__ logits,
                 int32_t *__restrict__ ids, float *__restrict__ w)
{
    constexpr uint32_t kNone = 0x007fffffu; // the key of -inf
    const int lane = threadIdx.x & (kLanes - 1);
    const int t = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= T)
        return; // a whole row of lanes
    float l[PER];
    load_logits<MOE_DT_F32, PER, kVec>(logits, t, E, lane, l);
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        l[i] = fmaxf(l[i], -INFINITY); // the other operand of a NaN
        const uint32_t b = __float_as_uint(l[i] + 0.0f);
        key[i] = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    }
    float m = 0.0f, all = 0.0f, mine = 0.0f;
    int my_id = -1;
    Chosen c = {};
#pragma unroll
    for (int i = 0; i < PER; ++i)
        keep(c, key[i], expert_of<MOE_DT_F32, kVec>(i, lane));
    for (int k = 0; k < K; ++k) {
        const uint32_t won = row_max(c.key[0]);
        const uint32_t mine_e = c.key[0] == won ? (uint32_t)c.e[0] : ~0u;
        const int e = (int)row_min(mine_e);
        const bool gave = mine_e == (uint32_t)e;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            c.key[i] = gave ? i < 2 ? c.key[i + 1] : 0u : c.key[i];
            c.e[i] = gave && i < 2 ? c.e[i + 1] : c.e[i];
        }
        if (k + 1 < K && __any(c.key[0] == 0u)) {
            c = Chosen{};
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int f = expert_of<MOE_DT_F32, kVec>(i, lane);
                const bool left = (key[i] < won) | ((key[i] == won) & (f > e));
                keep(c, left ? key[i] : 0u, f);
            }
        }
        const float v = __uint_as_float(won & 0x80000000u ? won & 0x7fffffffu : ~won);
        if (k == 0) {
            m = v;
            if (!renorm)
                all = row_sum(exps<PER>(l, m));
        }
        if (lane == k && won > kNone) {
            mine = expf(v == m ? 0.0f : v - m);
            my_id = e;
        }
    }
    store_slots(t, K, lane, renorm, all, my_id, mine, ids, w);
}

// (dlogits may be logits itself: a lane writes the experts that it has read)
template <int DT, int PER, bool kVec>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(int T, int E, int K, bool renorm, const void *logits,
                      const int32_t *__restrict__ ids, const float *__restrict__ w,
                      const float *__restrict__ dw, void *dlogits)
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
    // what slot k adds to its expert: w (g - dot), or g alone
    const float add = renorm ? wk * (g - dot) : g;
    // the token's experts in LDS, zeroed, then written by the slots; slots of
    // the same expert all write their sum.  A wavefront's LDS operations run
    // in order, and no other touches its tokens.  (Finding each slot's register
    // by comparisons took 23 us where this takes 10: 65,536 x 384 bf16 in the
    // cache, renormalized.)
    __shared__ __align__(16) float room[kThreads / kLanes][kLanes * PER];
    float *mine = room[threadIdx.x / kLanes];
#pragma unroll
    for (int i = 0; i < PER; i += 4)
        *reinterpret_cast<float4 *>(mine + (i / 4 * kLanes + lane) * 4) =
            float4{0.0f, 0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
#define MOE_SLOT(k)                                                                              \
    sum += (int)row_lane<k>((uint32_t)id) == id ? __uint_as_float(row_lane<k>(__float_as_uint(add))) \
                                                : 0.0f
    MOE_SLOT(0);
    MOE_SLOT(1);
    MOE_SLOT(2);
    MOE_SLOT(3);
    MOE_SLOT(4);
    MOE_SLOT(5);
    MOE_SLOT(6);
    MOE_SLOT(7);
#undef MOE_SLOT
    wave_fence();
    if (id >= 0)
        mine[id] = sum;
    wave_fence();
    float d[PER];
    if constexpr (kVec) {
#pragma unroll
        for (int j = 0; j < PER; j += 4) {
            const int e = (j / V * kLanes + lane) * V + j % V;
            const float4 q = *reinterpret_cast<const float4 *>(mine + e);
            d[j] = q.x;
            d[j + 1] = q.y;
            d[j + 2] = q.z;
            d[j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] = mine[i * kLanes + lane];
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
            const bool whole = whole_pieces(s.E_total, dtype, logits, nullptr);
            const auto k = [&] {
                if constexpr (DT == MOE_DT_F32)
                    return whole ? route_f32_kernel<PER, true> : route_f32_kernel<PER, false>;
                else
                    return whole ? route_kernel<DT, PER, true> : route_kernel<DT, PER, false>;
            }();
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
