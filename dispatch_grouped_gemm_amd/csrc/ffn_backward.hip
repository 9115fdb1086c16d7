// The dense feed-forward block's gradients, from dout and the kept
// pre-activations g | u:
//   dh = dout W2,  dg | du from dh, g, u (ffn.hpp),
//   dx = dg | du W13,  dW13 = (dg | du)^T x,  dW2 = dout^T h,
// four products in MFMA tiles.  The first one's epilogue has the activation's
// gradient and forms h again, so neither dh nor h of the forward pass is kept.
// The other three need nothing of each other and are one launch: the tiles of
// the next fill the CUs that the last of one leave idle.
// Operands that these products need transposed are read from LDS transposed.
// An x kept as MX FP8 becomes 16-bit rows in the workspace first.
#include "ffn.hpp"

namespace moe {

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How a backward call is cut, and its workspace: dgu [T, 2I], h [T, I], x [T, H]
// (MX FP8 only) and the parts of dh.
struct BackwardPlan {
    Cut dh;
    size_t dgu, h, x, parts, bytes;
};

BackwardPlan plan_of(const moe_ffn_shape &s)
{
    BackwardPlan l{};
    const size_t T = s.T, H = s.H, I = s.I;
    l.dh = product_cut(s.T, s.I, s.H, false);
    l.dgu = 0;
    l.h = l.dgu + align256(T * 2 * I * 2);
    l.x = l.h + align256(T * I * 2);
    l.parts = l.x + align256(T * H * 2);
    l.bytes = l.parts + product_parts_bytes(l.dh, s.T, s.I);
    return l;
}

// MX FP8 rows as 16-bit ones: 33/32 bytes in and 2 out per value (8,192 x 7,168
// 33 us, 5.4 TB/s).
template <int DT>
__global__ void __launch_bounds__(256)
from_mx_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scale, long pieces,
               uint16_t *__restrict__ out)
{
    for (long i = blockIdx.x * 256l + threadIdx.x; i < pieces; i += gridDim.x * 256l) {
        float f[8];
        from_mx(*reinterpret_cast<const uint2 *>(codes + 8 * i), scale[i / 4], f);
        store8<DT>(out + 8 * i, f);
    }
}

// Up to three products of one launch, in tiles of their own; job 0 may have A
// along its rows (dx), the others have both operands down.  first: a job's first workgroup, each a
// multiple of 8, so that a job's tiles keep their XCDs.
template <int DT>
struct Gradients {
    Product p[3];
    Put<DT> put[3];
    int jobs, along; // along: job 0 is dx
    TileKind kind[3];
    int first[4];
};

template <int DT>
__global__ void __launch_bounds__(512, 1) gradients_kernel(Gradients<DT> g)
{
    using A = Tiles<DT, kAlong, kDown>;
    using D = Tiles<DT, kDown, kDown>;
    __shared__ __align__(1024) uint8_t lds[A::Wide::kLds]; // the largest
    int j = 0;
    while (j + 1 < g.jobs && (int)blockIdx.x >= g.first[j + 1])
        ++j;
    const Product &p = g.p[j];
    const int b = blockIdx.x - g.first[j], n = p.tm * p.tn;
    if (b >= n)
        return;
    int im, in;
    tile_place(tile_run(b, n), p.tm, p.tn, &im, &in);
    const auto dx = [&](auto t) {
        using T = decltype(t);
        whole_tile<T, false, kAlong, kDown>(p, g.put[j], (long)im * T::kBM, in, lds);
    };
    const auto dw = [&](auto t) {
        using T = decltype(t);
        whole_tile<T, false, kDown, kDown>(p, g.put[j], (long)im * T::kBM, in, lds);
    };
    if (j < g.along) {
        if (g.kind[j] == kHuge)
            dx(typename A::Huge{});
        else if (g.kind[j] == kTall)
            dx(typename A::Tall{});
        else if (g.kind[j] == kWide)
            dx(typename A::Wide{});
        else if (g.kind[j] == kEven)
            dx(typename A::Even{});
        else
            dx(typename A::Flat{});
    } else if (g.kind[j] == kHuge) {
        dw(typename D::Huge{});
    } else if (g.kind[j] == kWide) {
        dw(typename D::Wide{});
    } else {
        dw(typename D::Even{});
    }
}

template <int DT>
hipError_t launch_gradients(Gradients<DT> &g, hipStream_t st)
{
    if (g.jobs == 0)
        return hipSuccess;
    Sides sides[3];
    for (int j = 0; j < g.jobs; ++j)
        sides[j] = {g.p[j].M, g.p[j].N, g.p[j].K};
    choose_tiles(sides, g.jobs, g.along, g.kind);
    int n = 0;
    for (int j = 0; j < g.jobs; ++j) {
        g.p[j].tm = (int)tiles_down(g.kind[j], g.p[j].M);
        g.p[j].tn = (int)tiles_across(g.kind[j], g.p[j].N);
        g.p[j].splits = 1;
        g.first[j] = n;
        n += (g.p[j].tm * g.p[j].tn + 7) / 8 * 8;
    }
    gradients_kernel<DT><<<n, 512, 0, st>>>(g);
    return hipGetLastError();
}

template <int DT>
hipError_t backward_of_type(const moe_ffn_shape &s, const BackwardPlan &l, const uint16_t *dout,
                            const void *x_, const uint8_t *x_scale, const uint16_t *w13,
                            const uint16_t *w2,
                            const Kept &kept, uint16_t *dx, void *dw13, void *dw2, bool f32,
                            bool accumulate, uint8_t *ws, hipStream_t st)
{
    uint16_t *dgu = reinterpret_cast<uint16_t *>(ws + l.dgu);
    uint16_t *h = dw2 ? reinterpret_cast<uint16_t *>(ws + l.h) : nullptr;
    float *parts = reinterpret_cast<float *>(ws + l.parts);
    Product p{};
    p.a = Operand{dout, s.H};
    p.b = Operand{w2, s.I};
    p.M = s.T;
    p.N = s.I;
    p.K = s.H;
    const ActivateBack<DT> back{s.I, s.gate_limit, s.up_limit, kept, dgu, h};
    hipError_t e = launch_product<DT, false, kAlong, kDown>(p, l.dh, back, back, parts, st);
    if (e != hipSuccess)
        return e;
    const uint16_t *x = static_cast<const uint16_t *>(x_);
    if (dw13 && x_scale) {
        uint16_t *to = reinterpret_cast<uint16_t *>(ws + l.x);
        const long pieces = (long)s.T * s.H / 8;
        from_mx_kernel<DT><<<(unsigned)std::min(tiles_up(pieces, 256), 4096l), 256, 0, st>>>(
            static_cast<const uint8_t *>(x_), x_scale, pieces, to);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        x = to;
    }
    Gradients<DT> g{};
    const auto job = [&](const Operand &a, const Operand &b, long M, int N, long K, void *out,
                         bool wide) {
        uint16_t *o = static_cast<uint16_t *>(out);
        const bool add = accumulate && out != dx;
        g.p[g.jobs] = Product{a, b, M, K, N, 0, 0, 1, nullptr};
        g.put[g.jobs++] = Put<DT>{N, add && !wide ? o : nullptr, wide ? nullptr : o,
                                  wide ? static_cast<float *>(out) : nullptr, add};
    };
    if (dx) {
        g.along = 1;
        job(Operand{dgu, 2l * s.I}, Operand{w13, s.H}, s.T, s.H, 2l * s.I, dx, false);
    }
    if (dw13)
        job(Operand{dgu, 2l * s.I}, Operand{x, s.H}, 2l * s.I, s.H, s.T, dw13, f32);
    if (dw2)
        job(Operand{dout, s.H}, Operand{h, s.I}, s.H, s.I, s.T, dw2, f32);
    return launch_gradients<DT>(g, st);
}

// The weights' gradients of no rows.
__global__ void __launch_bounds__(256) zero_kernel(uint4 *p, long pieces)
{
    for (long i = blockIdx.x * 256l + threadIdx.x; i < pieces; i += gridDim.x * 256l)
        p[i] = uint4{0, 0, 0, 0};
}

hipError_t zero(void *p, size_t bytes, hipStream_t st)
{
    const long pieces = (long)(bytes / 16);
    zero_kernel<<<(unsigned)std::min(tiles_up(pieces, 256), 4096l), 256, 0, st>>>(
        static_cast<uint4 *>(p), pieces);
    return hipGetLastError();
}

} // namespace

size_t ffn_backward_bytes(const moe_ffn_shape &s)
{
    const ProductSides sides[] = {{s.I, s.H, false}};
    return most_bytes(s.T, sides, [q = s](long M) mutable {
        q.T = (int32_t)M;
        return plan_of(q).bytes;
    });
}

hipError_t launch_ffn_backward(const moe_ffn_shape &s, int dtype, const void *dout, const void *x,
                               const uint8_t *x_scale, const void *w13, const void *w2,
                               const void *gate_up, const uint8_t *gate_up_scale, void *dx,
                               void *dw13, void *dw2, bool f32, bool accumulate, void *ws,
                               size_t ws_bytes, bool *fits, hipStream_t st)
{
    *fits = true;
    const auto u16 = [](const void *p) { return static_cast<const uint16_t *>(p); };
    const Kept kept{const_cast<void *>(gate_up), const_cast<uint8_t *>(gate_up_scale)};
    if (s.T == 0) {
        const size_t one = (size_t)s.H * s.I * (f32 ? 4 : 2);
        hipError_t e = hipSuccess;
        if (dw13 && !accumulate)
            e = zero(dw13, 2 * one, st);
        if (dw2 && !accumulate && e == hipSuccess)
            e = zero(dw2, one, st);
        return e;
    }
    const BackwardPlan plan = plan_of(s);
    *fits = ws_bytes >= plan.bytes;
    if (!*fits)
        return hipSuccess;
    uint16_t *d = static_cast<uint16_t *>(dx);
    uint8_t *w = static_cast<uint8_t *>(ws);
    if (dtype == MOE_DT_BF16)
        return backward_of_type<MOE_DT_BF16>(s, plan, u16(dout), x, x_scale, u16(w13), u16(w2), kept, d,
                                             dw13, dw2, f32, accumulate, w, st);
    return backward_of_type<MOE_DT_F16>(s, plan, u16(dout), x, x_scale, u16(w13), u16(w2), kept, d,
                                        dw13, dw2, f32, accumulate, w, st);
}

} // namespace moe
