// The dense feed-forward block's gradients, from dout and the kept
// pre-activations g | u:
//   dh = dout W2,  dg | du from dh, g, u (ffn.hpp),
//   dx = dg | du W13,  dW13 = (dg | du)^T x,  dW2 = dout^T h,
// four products in MFMA tiles.  The first one's epilogue has the activation's
// gradient and forms h again, so neither dh nor h of the forward pass is kept.
// Operands that these products need transposed are read from LDS transposed.
// An x kept as MX FP8 becomes 16-bit rows in the workspace first.
#include "ffn.hpp"

namespace moe {

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// dgu [T, 2I], h [T, I], x [T, H] (MX FP8 only) and the parts
struct BackLayout {
    size_t dgu, h, x, parts, bytes;
};

BackLayout back_layout(const moe_ffn_shape &s)
{
    BackLayout l{};
    const size_t T = s.T, H = s.H, I = s.I;
    l.dgu = 0;
    l.h = l.dgu + align256(T * 2 * I * 2);
    l.x = l.h + align256(T * I * 2);
    l.parts = l.x + align256(T * H * 2);
    l.bytes = l.parts + std::max({product_parts_bytes(T, I, H), product_parts_bytes(T, H, 2 * I),
                                  product_parts_bytes(2 * I, H, T),
                                  product_parts_bytes(H, I, T)});
    return l;
}

// MX FP8 rows as 16-bit ones: 33/32 bytes in and 2 out per value.
template <int DT>
__global__ void __launch_bounds__(256)
from_mx_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scale, long pieces,
               uint16_t *__restrict__ out)
{
    for (long i = blockIdx.x * 256l + threadIdx.x; i < pieces; i += gridDim.x * 256l) {
        float f[8];
        load8_mx(codes + 8 * i, scale[i / 4], f);
        store8<DT>(out + 8 * i, f);
    }
}

template <int DT>
hipError_t backward_of_type(const moe_ffn_shape &s, const uint16_t *dout, const void *x_,
                            const uint8_t *x_scale, const uint16_t *w13, const uint16_t *w2,
                            const Kept &kept, uint16_t *dx, void *dw13, void *dw2, bool f32,
                            bool accumulate, uint8_t *ws, hipStream_t st)
{
    const BackLayout l = back_layout(s);
    uint16_t *dgu = reinterpret_cast<uint16_t *>(ws + l.dgu);
    uint16_t *h = dw2 ? reinterpret_cast<uint16_t *>(ws + l.h) : nullptr;
    float *parts = reinterpret_cast<float *>(ws + l.parts);
    const auto dw = [&](void *w, long ld) {
        return Put<DT>{ld, accumulate && !f32 ? static_cast<const uint16_t *>(w) : nullptr,
                       f32 ? nullptr : static_cast<uint16_t *>(w),
                       f32 ? static_cast<float *>(w) : nullptr, accumulate};
    };
    Product p{};
    p.a = Operand{dout, s.H};
    p.b = Operand{w2, s.I};
    p.M = s.T;
    p.N = s.I;
    p.K = s.H;
    const ActivateBack<DT> back{s.I, s.gate_limit, s.up_limit, kept, dgu, h};
    hipError_t e = launch_product<DT, false, kAlong, kDown>(p, back, back, parts, st);
    if (e != hipSuccess)
        return e;
    if (dx) {
        p.a = Operand{dgu, 2l * s.I};
        p.b = Operand{w13, s.H};
        p.M = s.T;
        p.N = s.H;
        p.K = 2l * s.I;
        const Put<DT> put{s.H, nullptr, dx, nullptr, false};
        if ((e = launch_product<DT, false, kAlong, kDown>(p, put, put, parts, st)) != hipSuccess)
            return e;
    }
    if (dw13) {
        const uint16_t *x = static_cast<const uint16_t *>(x_);
        if (x_scale) {
            uint16_t *to = reinterpret_cast<uint16_t *>(ws + l.x);
            const long pieces = (long)s.T * s.H / 8;
            from_mx_kernel<DT><<<(unsigned)std::min(tiles_up(pieces, 256), 4096l), 256, 0, st>>>(
                static_cast<const uint8_t *>(x_), x_scale, pieces, to);
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
            x = to;
        }
        p.a = Operand{dgu, 2l * s.I};
        p.b = Operand{x, s.H};
        p.M = 2l * s.I;
        p.N = s.H;
        p.K = s.T;
        const Put<DT> put = dw(dw13, s.H);
        if ((e = launch_product<DT, false, kDown, kDown>(p, put, put, parts, st)) != hipSuccess)
            return e;
    }
    if (dw2) {
        p.a = Operand{dout, s.H};
        p.b = Operand{h, s.I};
        p.M = s.H;
        p.N = s.I;
        p.K = s.T;
        const Put<DT> put = dw(dw2, s.I);
        if ((e = launch_product<DT, false, kDown, kDown>(p, put, put, parts, st)) != hipSuccess)
            return e;
    }
    return hipSuccess;
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

size_t ffn_backward_bytes(const moe_ffn_shape &s) { return back_layout(s).bytes; }

hipError_t launch_ffn_backward(const moe_ffn_shape &s, int dtype, const void *dout, const void *x,
                               const uint8_t *x_scale, const void *w13, const void *w2,
                               const void *gate_up, const uint8_t *gate_up_scale, void *dx,
                               void *dw13, void *dw2, bool f32, bool accumulate, void *ws,
                               hipStream_t st)
{
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
    uint16_t *d = static_cast<uint16_t *>(dx);
    uint8_t *w = static_cast<uint8_t *>(ws);
    if (dtype == MOE_DT_BF16)
        return backward_of_type<MOE_DT_BF16>(s, u16(dout), x, x_scale, u16(w13), u16(w2), kept, d,
                                             dw13, dw2, f32, accumulate, w, st);
    return backward_of_type<MOE_DT_F16>(s, u16(dout), x, x_scale, u16(w13), u16(w2), kept, d,
                                        dw13, dw2, f32, accumulate, w, st);
}

} // namespace moe
