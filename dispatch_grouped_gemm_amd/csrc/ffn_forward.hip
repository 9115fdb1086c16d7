// The dense feed-forward block that every token takes beside the experts:
//   g | u = x W13^T,  h = silu(min(g, gl)) clamp(u, ul),  out = h W2^T (+ base).
// Two products in MFMA tiles; the first one's tiles hold gate and up rows of
// the same columns, so the activation and the product with u are done on the
// float32 sums in registers, and h is written once.
#include "ffn.hpp"

namespace moe {

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t h_bytes(const moe_ffn_shape &s) { return align256((size_t)s.T * s.I * 2); }

// ---------------------------------------------------------------------------
// Few rows (up to 64): 16 MB rows by 32 rows of a weight, bound by reading the
// weight once.  Eight wavefronts: two take 16 weight rows each, four a quarter
// of every step's 256 k, so a CU has a whole tile's K without parts of it in
// memory, and the activation is done where the sums meet, in LDS.  A step is
// 512 neighbouring bytes of every row; NS stages keep 72 KB or more in flight.
// The first product takes 16 gate rows and the 16 up rows of the same I.  One row
// of 5,120 bf16 values by 2,304: 11.9 us (47 MB) and 6.2 (24 MB).
// ---------------------------------------------------------------------------
template <int MB, int NB>
struct FewRows {
    static constexpr int kStepK = 256, kRow = 2 * kStepK; // bytes of a row's step
    static constexpr int kX = 16 * MB * kRow, kW = 32 * NB * kRow, kStage = kX + kW;
    static constexpr int NS = MB == 4 ? (NB == 2 ? 2 : 3) : NB == 2 ? 3 : MB == 1 ? 5 : 4;
    static constexpr int kLds = NS * kStage;
    static constexpr int UX = kX / 1024 / 8, UW = kW / 1024 / 8, U = UX + UW;
    static_assert(UX * 8192 == kX && UW * 8192 == kW, "whole loads");
};

struct FewProduct {
    const uint16_t *x, *w;
    int T, K;
};

// The sums of weight rows w_row(0 .. 32 NB - 1), in LDS: few_sum(b, m) is then a
// lane's rows 16 m + lane mod 16 by columns 4 (lane div 16) .. + 3 of block b of 16.
template <int DT, int MB, int NB, typename R>
__device__ __forceinline__ void few_sums(const FewProduct &p, R w_row, uint8_t *lds)
{
    using F = FewRows<MB, NB>;
    const int lane = threadIdx.x & 63, wave = tile_wave();
    const int slice = wave & 3, block = (wave >> 2) * NB;
    const uint32_t l0 = lds_addr(lds);
    // a load: two rows' steps, pieces stored at piece ^ (row mod 16), so that the
    // 16 rows that an operand read touches lie in different banks
    const uint8_t *base[F::U];
    uint32_t row[F::U];
    int k8[F::U];
#pragma unroll
    for (int u = 0; u < F::U; ++u) {
        const int q = u < F::UX ? wave * F::UX + u : wave * F::UW + u - F::UX;
        const int i = 2 * q + (lane >> 5);
        k8[u] = ((lane & 31) ^ (i & 15)) * 8;
        const auto of = [&](int r) { return u < F::UX ? (long)min(r, p.T - 1) : w_row(r); };
        base[u] = uniform_ptr(reinterpret_cast<const uint8_t *>((u < F::UX ? p.x : p.w) +
                                                                of(2 * q) * p.K));
        row[u] = (uint32_t)((of(i) - of(2 * q)) * p.K * 2);
    }
    const int steps = (p.K + F::kStepK - 1) / F::kStepK;
    const auto load = [&](int step, int buf) {
        step = min(step, steps - 1);
#pragma unroll
        for (int u = 0; u < F::U; ++u) {
            // past a row's end its last piece, which no product takes
            const uint32_t v = row[u] + 2 * min(step * F::kStepK + k8[u], p.K - 8);
            if (u < F::UX)
                g2lds<16>(base[u], v, l0 + buf * F::kStage + (wave * F::UX + u) * 1024);
            else
                g2lds<16, true>(base[u], v, l0 + buf * F::kStage + F::kX +
                                                (wave * F::UW + u - F::UX) * 1024);
        }
    };
    const int i = lane & 15;
    const auto read = [&](const uint8_t *rows, int half) {
        return *reinterpret_cast<const uint4 *>(
            rows + i * F::kRow + ((8 * slice + 4 * half + (lane >> 4)) ^ i) * 16);
    };
    v4f acc[NB][MB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            acc[n][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < F::NS - 1; ++s)
        load(s, s);
    int buf = 0;
    for (int s = 0; s < steps; ++s) {
        // the step has landed; the one before it is done with everywhere, and its
        // stage takes the next load
        tile_wait<(F::NS - 2) * F::U>();
        raw_barrier();
        const uint8_t *st = lds + buf * F::kStage;
        uint4 wq[2][NB], xq[2][MB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
                wq[h][n] = read(st + F::kX + (block + n) * 16 * F::kRow, h);
#pragma unroll
            for (int m = 0; m < MB; ++m)
                xq[h][m] = read(st + m * 16 * F::kRow, h);
        }
        load(s + F::NS - 1, buf == 0 ? F::NS - 1 : buf - 1);
        buf = buf + 1 == F::NS ? 0 : buf + 1;
        // (K is a multiple of 32: a half's k are all there or none)
        const int k = s * F::kStepK + 64 * slice;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (k + 32 * h < p.K)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[n][m] = mfma16<DT>(wq[h][n], xq[h][m], acc[n][m]);
    }
    tile_wait<0>();
    raw_barrier();
    v4f *part = reinterpret_cast<v4f *>(lds); // [block][m][slice][lane]
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            part[(((block + n) * MB + m) * 4 + slice) * 64 + lane] = acc[n][m];
    __syncthreads();
}

template <int MB>
__device__ __forceinline__ v4f few_sum(const uint8_t *lds, int b, int m)
{
    const v4f *q = reinterpret_cast<const v4f *>(lds) + (b * MB + m) * 256 + (threadIdx.x & 63);
    return ((q[0] + q[64]) + q[128]) + q[192];
}

template <int DT, int MB>
__global__ void __launch_bounds__(512) few_gate_up_kernel(FewProduct p, Activate<DT, 16> f)
{
    __shared__ __align__(1024) uint8_t lds[FewRows<MB, 1>::kLds];
    const int j0 = tile_run(blockIdx.x, gridDim.x) * 16, lane = threadIdx.x & 63;
    few_sums<DT, MB, 1>(p, [&](int i) { return (long)(i >> 4) * f.I + j0 + (i & 15); }, lds);
    const int wave = tile_wave();
    const long t = 16 * wave + (lane & 15);
    if (wave < MB && t < p.T)
        f.four(t, j0 + 4 * (lane >> 4), few_sum<MB>(lds, 0, wave), few_sum<MB>(lds, 1, wave));
}

// The same sums by 32 columns, whose MX FP8 blocks are then whole: a wavefront
// has a row's block in the four lanes 16 apart.
template <int DT, int MB>
__global__ void __launch_bounds__(512) few_gate_up_mx_kernel(FewProduct p, Activate<DT, 16> f)
{
    __shared__ __align__(1024) uint8_t lds[FewRows<MB, 2>::kLds];
    const int j0 = tile_run(blockIdx.x, gridDim.x) * 32, lane = threadIdx.x & 63;
    few_sums<DT, MB, 2>(p, [&](int i) { return (long)(i >> 5) * f.I + j0 + (i & 31); }, lds);
    const int wave = tile_wave();
    const long t = 16 * wave + (lane & 15);
    if (wave >= MB || t >= p.T)
        return;
    // 8 neighbouring columns a lane: those of two lanes of the sums
    float v[2][8];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = lane >> 4, b = 2 * n + (c >> 1), from = 2 * (c & 1) + i;
            const v4f *q = reinterpret_cast<const v4f *>(lds) + (b * MB + wave) * 256 +
                           16 * from + (lane & 15);
            const v4f s = ((q[0] + q[64]) + q[128]) + q[192];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[n][4 * i + k] = s[k];
        }
    f(t, j0 + 8 * (lane >> 4), v[0], v[1]);
}

template <int DT, int MB>
__global__ void __launch_bounds__(512) few_out_kernel(FewProduct p, Put<DT> f)
{
    __shared__ __align__(1024) uint8_t lds[FewRows<MB, 1>::kLds];
    const int n0 = tile_run(blockIdx.x, gridDim.x) * 32, lane = threadIdx.x & 63;
    few_sums<DT, MB, 1>(p, [&](int i) { return (long)(n0 + i); }, lds);
    const int wave = tile_wave(), m = wave % MB, b = wave / MB;
    const long t = 16 * m + (lane & 15);
    if (b < 2 && t < p.T) // (eight wavefronts: 2 MB at most)
        f.four(t, n0 + 16 * b + 4 * (lane >> 4), few_sum<MB>(lds, b, m));
}

// How a forward call is cut.
struct ForwardPlan {
    bool few_gate_up, few_out;
    Cut gate_up, out;
    size_t bytes;
};

ForwardPlan plan_of(const moe_ffn_shape &s)
{
    ForwardPlan p{};
    p.gate_up = product_cut(s.T, 2l * s.I, s.H, true);
    p.out = product_cut(s.T, s.H, s.I, false);
    p.few_gate_up = few_rows_pay(s.T, 2l * s.I, s.H, p.gate_up);
    p.few_out = few_rows_pay(s.T, s.H, s.I, p.out);
    p.bytes = h_bytes(s) +
              std::max(p.few_gate_up ? 0 : product_parts_bytes(p.gate_up, s.T, 2l * s.I),
                       p.few_out ? 0 : product_parts_bytes(p.out, s.T, s.H));
    return p;
}

// f with the 16-row blocks of T as a constant.
template <typename F>
hipError_t with_blocks(int T, F f)
{
    const int n = few_blocks(T);
    if (n == 1)
        f(std::integral_constant<int, 1>{});
    else if (n == 2)
        f(std::integral_constant<int, 2>{});
    else
        f(std::integral_constant<int, 4>{});
    return hipGetLastError();
}

template <int DT>
hipError_t forward_of_type(const moe_ffn_shape &s, const ForwardPlan &plan, const uint16_t *x,
                           const uint16_t *w13, const uint16_t *w2, const uint16_t *base,
                           const Kept &kept, uint16_t *out, uint8_t *ws, hipStream_t st)
{
    uint16_t *h = reinterpret_cast<uint16_t *>(ws);
    float *parts = reinterpret_cast<float *>(ws + h_bytes(s));
    const Activate<DT, 16> act{s.I, s.gate_limit, s.up_limit, kept, h};
    const Put<DT> put{s.H, base, out, nullptr, false};
    Product p{};
    p.M = s.T;
    hipError_t e;
    if (plan.few_gate_up) {
        const FewProduct q{x, w13, s.T, s.H};
        e = with_blocks(s.T, [&](auto mb) {
            constexpr int MB = decltype(mb)::value;
            if (kept.scale)
                few_gate_up_mx_kernel<DT, MB><<<s.I / 32, 512, 0, st>>>(q, act);
            else
                few_gate_up_kernel<DT, MB><<<s.I / 16, 512, 0, st>>>(q, act);
        });
    } else {
        p.a = Operand{x, s.H};
        p.b = Operand{w13, s.H};
        p.N = 2 * s.I;
        p.K = s.H;
        e = launch_product<DT, true, kAlong, kAlong>(
            p, plan.gate_up, act, Activate<DT, 1>{s.I, s.gate_limit, s.up_limit, kept, h}, parts,
            st);
    }
    if (e != hipSuccess)
        return e;
    if (plan.few_out)
        return with_blocks(s.T, [&](auto mb) {
            few_out_kernel<DT, decltype(mb)::value>
                <<<s.H / 32, 512, 0, st>>>(FewProduct{h, w2, s.T, s.I}, put);
        });
    p.a = Operand{h, s.I};
    p.b = Operand{w2, s.I};
    p.N = s.H;
    p.K = s.I;
    return launch_product<DT, false, kAlong, kAlong>(p, plan.out, put, put, parts, st);
}

} // namespace

size_t ffn_forward_bytes(const moe_ffn_shape &s)
{
    const ProductSides sides[] = {{2l * s.I, s.H, true}, {s.H, s.I, false}};
    return most_bytes(s.T, sides, [q = s](long M) mutable {
        q.T = (int32_t)M;
        return plan_of(q).bytes;
    });
}

hipError_t launch_ffn_forward(const moe_ffn_shape &s, int dtype, const void *x, const void *w13,
                              const void *w2, const void *base, void *gate_up,
                              uint8_t *gate_up_scale, void *out, void *ws, size_t ws_bytes,
                              bool *fits, hipStream_t st)
{
    const ForwardPlan plan = plan_of(s);
    *fits = ws_bytes >= plan.bytes;
    if (!*fits)
        return hipSuccess;
    const auto u16 = [](const void *p) { return static_cast<const uint16_t *>(p); };
    const Kept kept{gate_up, gate_up_scale};
    uint16_t *o = static_cast<uint16_t *>(out);
    uint8_t *w = static_cast<uint8_t *>(ws);
    if (dtype == MOE_DT_BF16)
        return forward_of_type<MOE_DT_BF16>(s, plan, u16(x), u16(w13), u16(w2), u16(base), kept, o,
                                            w, st);
    return forward_of_type<MOE_DT_F16>(s, plan, u16(x), u16(w13), u16(w2), u16(base), kept, o, w,
                                       st);
}

} // namespace moe
