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

template <int DT>
hipError_t forward_of_type(const moe_ffn_shape &s, const uint16_t *x, const uint16_t *w13,
                           const uint16_t *w2, const uint16_t *base, const Kept &kept,
                           uint16_t *out, uint8_t *ws, hipStream_t st)
{
    uint16_t *h = reinterpret_cast<uint16_t *>(ws);
    float *parts = reinterpret_cast<float *>(ws + h_bytes(s));
    Product p{};
    p.a = Operand{x, s.H};
    p.b = Operand{w13, s.H};
    p.M = s.T;
    p.N = 2 * s.I;
    p.K = s.H;
    hipError_t e = launch_product<DT, true, kAlong, kAlong>(
        p, Activate<DT, 16>{s.I, s.gate_limit, s.up_limit, kept, h},
        Activate<DT, 1>{s.I, s.gate_limit, s.up_limit, kept, h}, parts, st);
    if (e != hipSuccess)
        return e;
    p.a = Operand{h, s.I};
    p.b = Operand{w2, s.I};
    p.N = s.H;
    p.K = s.I;
    const Put<DT> put{s.H, base, out, nullptr, false};
    return launch_product<DT, false, kAlong, kAlong>(p, put, put, parts, st);
}

} // namespace

size_t ffn_forward_bytes(const moe_ffn_shape &s)
{
    return h_bytes(s) + std::max(product_parts_bytes(s.T, 2 * s.I, s.H, true),
                                 product_parts_bytes(s.T, s.H, s.I, false));
}

hipError_t launch_ffn_forward(const moe_ffn_shape &s, int dtype, const void *x, const void *w13,
                              const void *w2, const void *base, void *gate_up,
                              uint8_t *gate_up_scale, void *out, void *ws, hipStream_t st)
{
    const auto u16 = [](const void *p) { return static_cast<const uint16_t *>(p); };
    const Kept kept{gate_up, gate_up_scale};
    uint16_t *o = static_cast<uint16_t *>(out);
    uint8_t *w = static_cast<uint8_t *>(ws);
    if (dtype == MOE_DT_BF16)
        return forward_of_type<MOE_DT_BF16>(s, u16(x), u16(w13), u16(w2), u16(base), kept, o, w,
                                            st);
    return forward_of_type<MOE_DT_F16>(s, u16(x), u16(w13), u16(w2), u16(base), kept, o, w, st);
}

} // namespace moe
