// The residual joint around a block, one pass over the rows:
//   z   = y rho(y) w_post                 (w_post given, else y)
//   res = skip x + scale logistic(gate_t) z     (y given, else x)
//   normed = res rho(res) w_pre,  rho(v) = 1 / sqrt(mean v^2 + eps),
// the second norm of res as it is stored (rounded to the type), so that the
// backward pass, which has res, computes with the same values.  Sums are
// float32.  normed may also, or only, be written as MX FP8 rows, the experts'
// input, with the codes that moe_quant_mxfp8 makes of the rounded normed, and
// those of NaN where it is not finite.  The norm's gradient, with hat = v rho
// and g = w d,
//   rho (g - hat mean(g hat)),
// keeps every factor as near 1 as hat is: rho^3 leaves float32's range at rows
// of 1e-13 and of 1e14, rho alone and the gradient do not.
//
// Bound by HBM: a workgroup holds its row's 16-byte pieces in registers from
// the one read to the write, so every array moves once (8,192 x 7,168 bf16, all
// of it: 86 us, 5.5 TB/s; its gradients 167 us, 4.2 TB/s; 4,095 x 5,120 float32,
// gradients of the second norm alone 77 us, 4.4 TB/s).
#include <algorithm>

#include "elem.hpp"

namespace moe {

namespace {

struct NShape {
    int T, H;
    float eps, skip, scale;
};

// Sum over a row's wavefronts, `waves` from `first` on; every thread gets it.
// `slot` alternates between calls, so one barrier a sum is enough (and none
// where a row is one wavefront).
template <int N>
__device__ __forceinline__ void sum_all(float *v, float (*lds)[16][N], int slot, int first,
                                        int waves)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n)
            v[n] += __shfl_xor(v[n], d);
    if (waves == 1)
        return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n)
            lds[slot][threadIdx.x >> 6][n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
        v[n] = 0.0f;
    for (int w = first; w < first + waves; ++w)
#pragma unroll
        for (int n = 0; n < N; ++n)
            v[n] += lds[slot][w][n];
}

__device__ __forceinline__ float rho_of(float squares, const NShape &s)
{
    return rsqrtf(squares / (float)s.H + s.eps);
}

__device__ __forceinline__ float logistic_of(float v) { return 1.0f / (1.0f + expf(-v)); }

struct Forward {
    const void *x, *y, *w_post, *w_pre;
    const float *gate;
    void *res, *normed;
    uint8_t *codes, *exps;
};

// A row's pieces in thread order: piece p = i * threads + thread.
template <int DT, int NP>
__global__ void __launch_bounds__(1024) norm_forward_kernel(NShape s, Forward p)
{
    using E = Elem<DT>;
    using V = typename E::type;
    constexpr int kV = E::kVec;
    __shared__ float lds[2][16][1];
    const long t = blockIdx.x;
    const int pieces = s.H / kV;
    // everything is asked for at once: few rows wait for one latency, not for four
    uint4 xq[NP], yq[NP], post[NP], pre[NP], rq[NP];
    const auto row = [&](const void *v) { return static_cast<const uint4 *>(v) + t * pieces; };
    const float gate = p.gate ? p.gate[t] : 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        xq[i] = yq[i] = post[i] = pre[i] = uint4{0, 0, 0, 0};
        if (at < pieces) {
            xq[i] = row(p.x)[at];
            if (p.y)
                yq[i] = row(p.y)[at];
            if (p.w_post)
                post[i] = static_cast<const uint4 *>(p.w_post)[at];
            if (p.w_pre)
                pre[i] = static_cast<const uint4 *>(p.w_pre)[at];
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (p.y) {
        float a = p.gate ? s.scale * logistic_of(gate) : s.scale;
        if (p.w_post) {
            float sq[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float f[kV];
                E::unpack(yq[i], f);
#pragma unroll
                for (int k = 0; k < kV; ++k)
                    sq[0] += f[k] * f[k];
            }
            sum_all<1>(sq, lds, 0, 0, blockDim.x >> 6);
            a *= rho_of(sq[0], s);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * blockDim.x + threadIdx.x;
            float x[kV], y[kV], w[kV];
            E::unpack(xq[i], x);
            E::unpack(yq[i], y);
            E::unpack(post[i], w);
#pragma unroll
            for (int k = 0; k < kV; ++k)
                x[k] = s.skip * x[k] + a * (p.w_post ? y[k] * w[k] : y[k]);
            xq[i] = E::pack(x);
            if (p.res && at < pieces)
                const_cast<uint4 *>(row(p.res))[at] = xq[i];
            if (at >= pieces)
                xq[i] = uint4{0, 0, 0, 0};
        }
    }
    if (!p.normed && !p.codes)
        return;
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float f[kV];
        E::unpack(xq[i], f);
#pragma unroll
        for (int k = 0; k < kV; ++k)
            sq[0] += f[k] * f[k];
    }
    sum_all<1>(sq, lds, 1, 0, blockDim.x >> 6);
    const float rho = rho_of(sq[0], s);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int at = i * blockDim.x + threadIdx.x;
        float f[kV], w[kV];
        E::unpack(xq[i], f);
        E::unpack(pre[i], w);
#pragma unroll
        for (int k = 0; k < kV; ++k)
            f[k] = at < pieces ? f[k] * rho * w[k] : 0.0f; // (rho may be infinite)
        rq[i] = E::pack(f);
        if (p.normed && at < pieces)
            const_cast<uint4 *>(row(p.normed))[at] = rq[i];
        if (p.codes) {
            E::unpack(rq[i], f); // the rounded values, as a quantiser of normed has them
            float v[kV];
            uint32_t lost[kV / 4];
            float amax = mx8_finite<kV>(f, v, lost);
#pragma unroll
            for (int d = 1; d < 32 / kV; d <<= 1)
                amax = fmaxf(amax, __shfl_xor(amax, d));
            if (at < pieces) {
                const int e = mx8_block_exponent(amax);
                uint32_t *o = reinterpret_cast<uint32_t *>(p.codes + t * s.H) + at * (kV / 4);
#pragma unroll
                for (int k = 0; k < kV / 4; ++k)
                    o[k] = mx8_pack4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], e, amax) |
                           lost[k];
                if (at % (32 / kV) == 0)
                    p.exps[t * (s.H / 32) + at / (32 / kV)] = (uint8_t)(e + 127);
            }
        }
    }
}

struct Backward {
    const void *dnormed, *dres, *res, *y, *w_post, *w_pre;
    const float *gate;
    void *dx, *dy;
    float *dgate, *part_pre, *part_post; // [groups][H]
};

// A workgroup takes `teams` rows at a time (a short row, of one piece a thread,
// alone would leave the CU waiting for its sums), every groups-th such set, and keeps its rows' sums
// of the weights' gradients in registers; its teams' meet in LDS at the end, and
// the workgroups' planes are added in their order.
template <int DT, int NP>
__global__ void __launch_bounds__(1024) norm_backward_kernel(NShape s, Backward p, int teams)
{
    using E = Elem<DT>;
    constexpr int kV = E::kVec;
    teams = NP == 1 ? teams : 1;
    __shared__ float l1[2][16][2], l2[2][16][2];
    extern __shared__ __align__(16) float team_sums[];
    const int pieces = s.H / kV, threads = blockDim.x / teams;
    const int team = NP == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / threads) : 0;
    const int tid = threadIdx.x - team * threads, waves = threads >> 6, wave0 = team * waves;
    float sum_pre[NP][kV], sum_post[NP][kV];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int k = 0; k < kV; ++k)
            sum_pre[i][k] = sum_post[i][k] = 0.0f;
    int slot = 0;
    // (a team whose row is past the end goes along: the sums have barriers)
    for (long t0 = (long)blockIdx.x * teams; t0 < s.T; t0 += (long)gridDim.x * teams, slot ^= 1) {
        const bool there = NP > 1 || t0 + team < s.T;
        const long t = there ? t0 + team : s.T - 1;
        const int end = there ? pieces : 0;
        const auto row = [&](const void *v) { return static_cast<const uint4 *>(v) + t * pieces; };
        uint4 rq[NP], nq[NP], dq[NP], yq[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * threads + tid;
            rq[i] = nq[i] = dq[i] = yq[i] = uint4{0, 0, 0, 0};
            if (at < end) {
                if (p.dnormed) {
                    rq[i] = row(p.res)[at];
                    nq[i] = row(p.dnormed)[at];
                }
                if (p.dres)
                    dq[i] = row(p.dres)[at];
                if (p.y)
                    yq[i] = row(p.y)[at];
            }
        }
        // mean res^2 and mean (dn w) hat; mean y^2
        float rho = 0.0f, mean = 0.0f;
        if (p.dnormed) {
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int at = i * threads + tid;
                if (at >= end)
                    continue;
                float r[kV], d[kV], w[kV];
                E::unpack(rq[i], r);
                E::unpack(nq[i], d);
                E::unpack(static_cast<const uint4 *>(p.w_pre)[at], w);
#pragma unroll
                for (int k = 0; k < kV; ++k) {
                    v[0] += r[k] * r[k];
                    v[1] += r[k] * d[k] * w[k];
                }
            }
            sum_all<2>(v, l1, slot, wave0, waves);
            rho = rho_of(v[0], s);
            mean = rho * (v[1] / (float)s.H);
        }
        const float sig = p.gate ? logistic_of(p.gate[t]) : 1.0f, a = s.scale * sig;
        // dr, in place of dn; and the sums that y's gradient and the gate's need
        float dr[NP][kV];
        float v[2] = {0.0f, 0.0f}; // sum y^2, sum dr y w_post
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * threads + tid;
            if (at >= end)
                continue;
            float r[kV], d[kV], w[kV];
            E::unpack(dq[i], dr[i]);
            if (p.dnormed) {
                E::unpack(rq[i], r);
                E::unpack(nq[i], d);
                E::unpack(static_cast<const uint4 *>(p.w_pre)[at], w);
#pragma unroll
                for (int k = 0; k < kV; ++k) {
                    const float hat = r[k] * rho;
                    dr[i][k] += rho * (d[k] * w[k] - hat * mean);
                    sum_pre[i][k] += d[k] * hat;
                }
            }
            if (p.dx) {
#pragma unroll
                for (int k = 0; k < kV; ++k)
                    r[k] = p.y ? s.skip * dr[i][k] : dr[i][k];
                const_cast<uint4 *>(row(p.dx))[at] = E::pack(r);
            }
            if (p.y) {
                E::unpack(yq[i], r);
                if (p.w_post)
                    E::unpack(static_cast<const uint4 *>(p.w_post)[at], w);
#pragma unroll
                for (int k = 0; k < kV; ++k) {
                    v[0] += r[k] * r[k];
                    v[1] += dr[i][k] * (p.w_post ? r[k] * w[k] : r[k]);
                }
            }
        }
        if (!p.y)
            continue;
        if (p.w_post || p.dgate)
            sum_all<2>(v, l2, slot, wave0, waves);
        const float rho_y = p.w_post ? rho_of(v[0], s) : 1.0f;
        if (p.dgate && tid == 0 && there)
            // logistic(-gate), not 1 - sig, which has no bits left for a gate above 17
            p.dgate[t] = s.scale * sig * logistic_of(-p.gate[t]) * (rho_y * v[1]);
        const float mean_y = a * (rho_y * (v[1] / (float)s.H));
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * threads + tid;
            if (at >= end)
                continue;
            float y[kV], w[kV];
            E::unpack(yq[i], y);
            if (p.w_post) {
                E::unpack(static_cast<const uint4 *>(p.w_post)[at], w);
#pragma unroll
                for (int k = 0; k < kV; ++k) {
                    const float hat = y[k] * rho_y, dz = a * dr[i][k];
                    sum_post[i][k] += dz * hat;
                    y[k] = rho_y * (dz * w[k] - hat * mean_y);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kV; ++k)
                    y[k] = a * dr[i][k];
            }
            if (p.dy)
                const_cast<uint4 *>(row(p.dy))[at] = E::pack(y);
        }
    }
    const auto leave = [&](float (*sum)[kV], float *part) {
        if (!part)
            return;
        if (team > 0)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int at = i * threads + tid;
                if (at < pieces)
#pragma unroll
                    for (int k = 0; k < kV; k += 4)
                        *reinterpret_cast<v4f *>(team_sums + (team - 1) * s.H + at * kV + k) =
                            v4f{sum[i][k], sum[i][k + 1], sum[i][k + 2], sum[i][k + 3]};
            }
        __syncthreads();
        if (team == 0)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int at = i * threads + tid;
                if (at < pieces)
#pragma unroll
                    for (int k = 0; k < kV; k += 4) {
                        v4f v = {sum[i][k], sum[i][k + 1], sum[i][k + 2], sum[i][k + 3]};
                        for (int m = 1; m < teams; ++m)
                            v += *reinterpret_cast<const v4f *>(team_sums + (m - 1) * s.H +
                                                                at * kV + k);
                        *reinterpret_cast<v4f *>(part + (long)blockIdx.x * s.H + at * kV + k) = v;
                    }
            }
        __syncthreads();
    };
    leave(sum_pre, p.part_pre);
    leave(sum_post, p.part_post);
}

// out[h] = the sum of the groups' planes: 64 columns a workgroup, 16 wavefronts
// with a part of the planes each, their loads in flight together.
__global__ void __launch_bounds__(1024)
norm_planes_kernel(int H, int groups, const float *part0, const float *part1, float *out0,
                   float *out1)
{
    const float *part = blockIdx.y ? part1 : part0;
    float *out = blockIdx.y ? out1 : out0;
    if (!out)
        return;
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, h = blockIdx.x * 64 + lane;
    float sum = 0.0f;
    if (h < H) {
        const int end = groups * (q + 1) / 16;
        int g = groups * q / 16;
        for (; g + 8 <= end; g += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = part[(long)(g + i) * H + h];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum += v[i];
        }
        for (; g < end; ++g)
            sum += part[(long)g * H + h];
    }
    lds[q][lane] = sum;
    __syncthreads();
    if (q == 0 && h < H) {
        for (int w = 1; w < 16; ++w)
            sum += lds[w][lane];
        out[h] = sum;
    }
}

// Threads and pieces a thread for a row of `pieces`: one up to `one` pieces, then
// two, and four where two would be over 1,024 threads (float32 rows past 8,192).
struct Split {
    int threads, np;
};

Split split_of(int pieces, int one)
{
    const int np = pieces <= one ? 1 : pieces <= 2048 ? 2 : 4;
    return Split{((pieces + np - 1) / np + 63) / 64 * 64, np};
}

template <int DT>
int pieces_of(const moe_norm_shape &s)
{
    return s.H / Elem<DT>::kVec;
}

NShape dev(const moe_norm_shape &s)
{
    return NShape{s.T, s.H, s.eps, s.skip_scale, s.block_scale};
}

// Workgroups of the backward pass: two a CU, and their planes in the workspace.
int groups_of(const moe_norm_shape &s) { return std::min(s.T, 512); }

size_t plane_bytes(const moe_norm_shape &s)
{
    return ((size_t)groups_of(s) * s.H * sizeof(float) + 255) / 256 * 256;
}

} // namespace

size_t norm_workspace_bytes(const moe_norm_shape &s) { return 2 * plane_bytes(s); }

hipError_t launch_norm_forward(const moe_norm_shape &sh, int dtype, const void *x, const void *y,
                               const void *w_post, const float *gate, const void *w_pre,
                               void *res, void *normed, uint8_t *codes, uint8_t *exps,
                               hipStream_t st)
{
    const NShape s = dev(sh);
    const Forward p{x, y, w_post, w_pre, gate, res, normed, codes, exps};
    with_elem(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const Split c = split_of(pieces_of<DT>(sh), 256);
        const auto go = [&](auto np) {
            norm_forward_kernel<DT, decltype(np)::value><<<s.T, c.threads, 0, st>>>(s, p);
        };
        if (c.np == 1)
            go(std::integral_constant<int, 1>{});
        else if (c.np == 2)
            go(std::integral_constant<int, 2>{});
        else if constexpr (DT == MOE_DT_F32)
            go(std::integral_constant<int, 4>{});
    });
    return hipGetLastError();
}

hipError_t launch_norm_backward(const moe_norm_shape &sh, int dtype, const void *dnormed,
                                const void *dres, const void *res, const void *y,
                                const void *w_post, const float *gate, const void *w_pre,
                                void *dx, void *dy, float *dgate, float *dw_post, float *dw_pre,
                                void *ws, hipStream_t st)
{
    const NShape s = dev(sh);
    const int groups = groups_of(sh);
    float *pre = static_cast<float *>(ws);
    float *post = pre ? pre + plane_bytes(sh) / sizeof(float) : nullptr;
    const Backward p{dnormed, dres, res, y, w_post, w_pre, gate, dx, dy, dgate,
                     dw_pre ? pre : nullptr, dw_post ? post : nullptr};
    if (s.T > 0) {
        with_elem(dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            const Split c = split_of(pieces_of<DT>(sh), 512);
            // short rows by several teams, up to 512 threads (5,981 x 608 bf16 rows 21 us,
            // by one 39)
            const int teams =
                c.np > 1 ? 1
                         : std::max(1, std::min(512 / c.threads, (s.T + groups - 1) / groups));
            const auto go = [&](auto np) {
                norm_backward_kernel<DT, decltype(np)::value>
                    <<<groups, teams * c.threads, (teams - 1) * s.H * sizeof(float), st>>>(
                        s, p, teams);
            };
            if (c.np == 1)
                go(std::integral_constant<int, 1>{});
            else if (c.np == 2)
                go(std::integral_constant<int, 2>{});
            else if constexpr (DT == MOE_DT_F32)
                go(std::integral_constant<int, 4>{});
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (dw_pre || dw_post) // of no rows: zeros
        norm_planes_kernel<<<dim3((s.H + 63) / 64, 2), 1024, 0, st>>>(s.H, groups, pre, post,
                                                                    dw_pre, dw_post);
    return hipGetLastError();
}

} // namespace moe
