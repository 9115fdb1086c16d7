// Products of 16-bit matrices in MFMA tiles,
//   C[m][n] = sum over k of A[m][k] B[n][k]   (float32 sums),
// where each operand lies in memory either with k along its rows (kAlong) or
// with k down its rows (kDown: the transpose, as a gradient needs it).
//
// A tile is BM x BN values of C by WM x WN wavefronts.  Steps of 64 k go from
// global memory to LDS without registers (NS stages) as they lie in memory;
// an operand that has k along its rows is read 16 bytes (8 k) a lane, one that
// has k down its rows by the LDS transpose read, 4 k of 16 columns for 16
// lanes, twice.  The 16-byte pieces of a stage are stored where the rows that
// one read touches lie in different banks: both reads run at their full rate
// (8 waves: 4 clocks a KiB along, 8 down; pieces in order 12 and 26).
//
// Operands are read from LDS one phase ahead of their matrix instructions,
// into a second set of registers, a few reads between every few matrix
// instructions.  The last phase of a step reads the next stage and sends off
// the loads of the step after it, into the stage that all wavefronts have
// just finished reading: one barrier a step.
//
// What of K is no whole step comes first (k of C's sum in any order): its
// missing k are zeroed in LDS once the stage has landed, so that no step
// inside the loop looks at K and nothing of other rows enters a sum.
#pragma once

#include "elem.hpp"

namespace moe {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// D(16x16) += A(16x32) B(32x16): lane l holds A's row / B's column l mod 16
// at k = 8 (l div 16) .. + 7, and D's column l mod 16 at rows
// 4 (l div 16) .. + 3.
template <int DT>
__device__ __forceinline__ v4f mfma16(const uint4 &a, const uint4 &b, v4f c)
{
    if constexpr (DT == MOE_DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                      __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// This thread's wavefront in the workgroup, in a scalar register.
__device__ __forceinline__ int tile_wave()
{
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// s_waitcnt vmcnt(N) lgkmcnt(0).
template <int N>
__device__ __forceinline__ void tile_wait()
{
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

// Column of C that row i (0..15) of a wavefront's block f of 16 B rows stands
// for: a lane then holds 8 neighbouring columns in two blocks' sums.
__device__ __forceinline__ int tile_column(int f, int i)
{
    return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
}

// Place of workgroup b of n in a run that gives each XCD (neighbouring
// workgroups run on different ones) a contiguous part.
__device__ __forceinline__ int tile_run(int b, int n)
{
    const int xcd = b & 7;
    return xcd * (n >> 3) + min(xcd, n & 7) + (b >> 3);
}

// Tile q of tm x tn: down 8 row tiles before the next column tile, so the
// tiles that run together on an XCD share rows and columns in its L2.
__device__ __forceinline__ void tile_place(int q, int tm, int tn, int *im, int *in)
{
    const int group = q / (8 * tn), first = group * 8;
    const int rows = min(8, tm - first), in_group = q - group * 8 * tn;
    *im = first + in_group % rows;
    *in = in_group / rows;
}

constexpr bool kAlong = false, kDown = true; // where an operand's k lies

// An operand: its first element and the pitch of its rows in elements.
struct Operand {
    const uint16_t *p;
    long ld;
};

// ROWS rows (of the tile's side) by 64 k in LDS, either way.
template <int ROWS, bool DOWN, bool PERM>
struct Side {
    static constexpr int kBytes = ROWS * 128;
    static constexpr int kLoads = kBytes / 1024;
    static constexpr int kPitch = DOWN ? 2 * ROWS : 128; // LDS bytes of a row
    static constexpr int kPieces = kPitch / 16;
    static constexpr int kRows = 1024 / kPitch; // LDS rows of a load
    static_assert(kPieces >= 8, "the turns stay inside a row");

    // what the 16-byte piece c of LDS row i is moved by
    static __device__ __forceinline__ int turn(int i)
    {
        if (!DOWN)
            return (i >> 1) & 7;
        if (kPieces == 8) // two rows fill the banks
            return PERM ? 4 * ((i >> 1) & 1) : 2 * (((i >> 1) & 1) | ((i >> 2) & 2));
        return PERM ? 4 * (i & 3) : 2 * ((i & 3) | ((i >> 1) & 4));
    }
    // LDS row and piece of this lane in load u
    static __device__ __forceinline__ int row_of(int u) { return u * kRows + lane() / kPieces; }
    static __device__ __forceinline__ int piece_of(int i)
    {
        return (lane() & (kPieces - 1)) ^ turn(i);
    }
    static __device__ __forceinline__ int lane() { return threadIdx.x & 63; }

    // byte offset of this lane's part of the 16 rows (kDown: columns) of block
    // f from row0, k 0 .. 31 of the stage (the others: Tile::read)
    static __device__ __forceinline__ int at(int row0, int f, int second)
    {
        const int l = lane() & 15, g = lane() >> 4;
        if (!DOWN)
            return (row0 + 16 * f + l) * 128 + ((g ^ turn(l)) * 16);
        const int k = 8 * g + 4 * second + (l >> 2), s = l & 3;
        const int col = row0 + (PERM ? 32 * (f >> 1) + 8 * s + 4 * (f & 1) : 16 * f + 4 * s);
        return k * kPitch + ((col >> 3) ^ turn(k)) * 16 + (col & 7) * 2;
    }
};

typedef short v4s16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s16 lds_v4s16;

__device__ __forceinline__ uint2 read_turned(const uint8_t *p)
{
    const v4s16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s16 *)(p));
    return __builtin_bit_cast(uint2, v);
}

template <int DT, int BM, int BN, int WM, int WN, int NS, bool ADOWN, bool BDOWN>
struct Tile {
    static constexpr int NW = WM * WN, MF = BM / WM / 16, NF = BN / WN / 16;
    static constexpr int kBM = BM, kBN = BN, kWN = WN, kThreads = 64 * NW;
    using SA = Side<BM, ADOWN, false>;
    using SB = Side<BN, BDOWN, true>;
    static constexpr int kStage = SA::kBytes + SB::kBytes, kLds = NS * kStage;
    // loads per wavefront and step, A's first
    static constexpr int UA = SA::kLoads / NW, UB = SB::kLoads / NW, U = UA + UB;
    static constexpr int GM = MF % 4 == 0 ? 4 : MF % 3 == 0 ? 3 : MF; // row blocks of a phase
    static_assert(MF % GM == 0 && NF % 2 == 0 && NF <= 4, "whole groups and pairs of blocks");
    static_assert(UA * NW == SA::kLoads && UB * NW == SB::kLoads, "whole loads");

    v4f acc[MF][NF];

    // This lane's offsets in load v of a side, and the load's base address.
    // rows(i): matrix row of the tile's row i, not falling (along); c0, c_end:
    // the first column here and the end of the matrix's (down, multiples of 8:
    // columns past the end are read from the last piece and not stored).
    template <typename S, bool DOWN, typename Rows>
    static __device__ __forceinline__ uint32_t place(const Operand &o, Rows rows, long c0,
                                                     long c_end, long k0, int v,
                                                     const uint8_t **base)
    {
        const int i = S::row_of(v), c = S::piece_of(i);
        if constexpr (DOWN) {
            *base = uniform_ptr(reinterpret_cast<const uint8_t *>(o.p + k0 * o.ld + c0));
            return (uint32_t)(i * o.ld * 2 + (min(c0 + 8 * c, c_end - 8) - c0) * 2);
        } else {
            const long r0 = rows(v * S::kRows);
            *base = uniform_ptr(reinterpret_cast<const uint8_t *>(o.p + r0 * o.ld + k0));
            return (uint32_t)((rows(i) - r0) * o.ld * 2 + c * 16);
        }
    }

    // The offset where only k below `there` are: what is missing is read from
    // the last row there is (down) or the row's own first half (along, where
    // `there` is 32 or 64).
    template <typename S, bool DOWN>
    static __device__ __forceinline__ uint32_t inside(const Operand &o, uint32_t voff, int v,
                                                      int there)
    {
        const int i = S::row_of(v);
        if constexpr (DOWN)
            return voff - (uint32_t)((i - min(i, there - 1)) * o.ld * 2);
        else
            return S::piece_of(i) * 8 >= there ? voff - 64 : voff;
    }

    template <typename S, bool DOWN>
    static __device__ __forceinline__ void zero_rest(uint8_t *lds, int there)
    {
        if constexpr (DOWN) {
            for (int at = there * S::kPitch + threadIdx.x * 16; at < S::kBytes;
                 at += kThreads * 16)
                *reinterpret_cast<uint4 *>(lds + at) = uint4{0, 0, 0, 0};
        } else {
            for (int at = threadIdx.x; at < S::kBytes / 16; at += kThreads) {
                const int i = at >> 3, c = (at & 7) ^ S::turn(i);
                if (c * 8 >= there)
                    *reinterpret_cast<uint4 *>(lds + at * 16) = uint4{0, 0, 0, 0};
            }
        }
    }

    // 16 rows (columns) by 32 k of a side: block f of the wavefront's, k from
    // 32 half on; off: Side::at of its blocks 0 and 1.
    template <typename S, bool DOWN>
    static __device__ __forceinline__ uint4 read(const uint8_t *p, const int (*off)[2], int f,
                                                 int half)
    {
        if constexpr (!DOWN)
            return *reinterpret_cast<const uint4 *>(p + f * 2048 + (off[0][0] ^ (64 * half)));
        // two blocks are 32 columns, four pieces: the turn, an xor of the piece's
        // number, leaves them one as well; 32 k turn alike
        const int x = (f & ~1) * 32, y = 32 * half * S::kPitch;
        const uint2 lo = read_turned(p + (off[f & 1][0] ^ x) + y);
        const uint2 hi = read_turned(p + (off[f & 1][1] ^ x) + y);
        return uint4{lo.x, lo.y, hi.x, hi.y};
    }

    // acc = the sums over the steps [first, first + steps) of K = k values.
    template <typename RA, typename RB>
    __device__ __forceinline__ void run(uint8_t *lds, const Operand &a, RA rows_a, long a0,
                                        long a_end, const Operand &b, RB rows_b, long b0,
                                        long b_end, long k, int first, int steps)
    {
        const int wave = tile_wave(), last = steps - 1;
        const int ragged = (int)(k - 64 * ((k - 1) / 64)); // k of step 0
        const long k0 = first == 0 ? 0 : ragged + 64l * (first - 1);
        const int there = first == 0 ? ragged : 64;        // k of the first step here
        const uint32_t l0 = lds_addr(lds);
        const long ka = 2 * (ADOWN ? a.ld : 1), kb = 2 * (BDOWN ? b.ld : 1); // bytes of a k

        uint32_t voff[U];
        const uint8_t *base[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < UA)
                voff[u] = place<SA, ADOWN>(a, rows_a, a0, a_end, k0, wave * UA + u, &base[u]);
            else
                voff[u] =
                    place<SB, BDOWN>(b, rows_b, b0, b_end, k0, wave * UB + u - UA, &base[u]);
        }
        const auto lds_of = [&](int u) {
            return l0 + (u < UA ? (wave * UA + u) * 1024
                                : SA::kBytes + (wave * UB + u - UA) * 1024);
        };
        const auto load = [&](int u, int step, int buf) {
            g2lds<16>(base[u] + step * (64 * (u < UA ? ka : kb)), voff[u],
                      lds_of(u) + buf * kStage);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t v = u < UA
                                   ? inside<SA, ADOWN>(a, voff[u], wave * UA + u, there)
                                   : inside<SB, BDOWN>(b, voff[u], wave * UB + u - UA, there);
            g2lds<16>(base[u], v, lds_of(u));
            // the next step begins where this one ends; where there is none, what is
            // loaded ahead is this one again
            if (last > 0)
                base[u] -= (64 - there) * (u < UA ? ka : kb);
            else
                voff[u] = v;
        }
#pragma unroll
        for (int s = 1; s < NS; ++s)
#pragma unroll
            for (int u = 0; u < U; ++u)
                load(u, min(s, last), s);

        int aoff[2][2], boff[2][2];
        const int wm = wave / WN, wn = wave % WN;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                aoff[f][h] = SA::at(wm * MF * 16, f, h);
                boff[f][h] = SB::at(wn * NF * 16, f, h);
            }
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                acc[m][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        // The phases of a step: half k of its 64 values, a group of GM of the
        // wavefront's row blocks.  Phase p multiplies the operands in sets p mod 2
        // (A) and k (B) and reads those of phase p + 1 into the other sets.
        constexpr int G = MF / GM, P = 2 * G;
        static_assert(P % 2 == 0, "the next step starts with A's set 0");
        uint4 ao[2][GM], bo[2][NF];
        const auto read_a = [&](int q, int ph, int buf) {
            ao[ph & 1][q] = read<SA, ADOWN>(lds + buf * kStage, aoff, (ph % G) * GM + q, ph / G);
        };
        const auto read_b = [&](int f, int half, int buf) {
            bo[half][f] = read<SB, BDOWN>(lds + buf * kStage + SA::kBytes, boff, f, half);
        };
        // step s in stage buf: the next stage holds step s + 1 before the last
        // phase, which also sends off the loads of step s + NS into this stage
        const auto step_of = [&](int s, int buf, int next) {
#pragma unroll
            for (int ph = 0; ph < P; ++ph) {
                const bool end = ph + 1 == P;
                const int np = end ? 0 : ph + 1, nbuf = end ? next : buf;
                if (end) {
                    tile_wait<(NS - 2) * U>();
                    raw_barrier();
                }
#pragma unroll
                for (int q = 0; q < GM; ++q) {
                    read_a(q, np, nbuf);
                    if (np % G == 0)
#pragma unroll
                        for (int f = q * NF / GM; f < (q + 1) * NF / GM; ++f)
                            read_b(f, np / G, nbuf);
                    if (end)
#pragma unroll
                        for (int u = q * U / GM; u < (q + 1) * U / GM; ++u)
                            load(u, min(s + NS, last), buf);
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        v4f &c = acc[(ph % G) * GM + q][f];
                        c = mfma16<DT>(bo[ph / G][f], ao[ph & 1][q], c);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        wait_vmcnt<(NS - 1) * U>();
        raw_barrier();
        if (there < 64) {
            zero_rest<SA, ADOWN>(lds, there);
            zero_rest<SB, BDOWN>(lds + SA::kBytes, there);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            raw_barrier();
        }
#pragma unroll
        for (int q = 0; q < GM; ++q)
            read_a(q, 0, 0);
#pragma unroll
        for (int f = 0; f < NF; ++f)
            read_b(f, 0, 0);
        if constexpr (NS == 2) {
            int s = 0;
            for (; s + 2 <= steps; s += 2) {
                step_of(s, 0, 1);
                step_of(s + 1, 1, 0);
            }
            if (s < steps)
                step_of(s, 0, 1);
        } else {
            int buf = 0;
            for (int s = 0; s < steps; ++s) {
                const int next = buf + 1 == NS ? 0 : buf + 1;
                step_of(s, buf, next);
                buf = next;
            }
        }
        tile_wait<0>();
    }
};

} // namespace moe
