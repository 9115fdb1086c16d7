// Low-rank adapters of many requests beside one shared projection:
//   out[t] = base[t] + scale_l (x[t] A_l^T) B_l^T,   l = ids[t],
// base = x W^T computed here, or given; a row of id -1 (or past the
// adapters) has no second term.
//
// "Shrink" makes v[t] = x[t] A_l^T in float32.  "Project" computes x W^T in
// MFMA tiles and, once a tile's sums are complete, adds the adapters' term
// to them in registers ("expand"), so out is written once and rounded once.
// Where the tiles are too few for the CUs, they become parts of H, float32
// planes that a last launch ("add") joins in a fixed order and expands.
//
// Rows come in any order.  Whoever owns a set of rows walks the different
// ids among them: an adapter's product is formed for 16 rows at a time (the
// matrix instruction costs the same for one) and taken only where the id
// matches, so no row ever sees another adapter's values, infinite or NaN.
// Past few rows a first launch orders the rows by adapter, so that a tile
// holds few of them; results do not depend on the places inside one.
//
// v enters the matrix instruction as it is: as the sum of three bf16 values
// with eight of float32's 24 bits each, hi, mid and lo.  fp16 lacks float32's
// range, so there B becomes bf16 instead, the sum of two values (11 bits).
// Products of bf16 values are exact in float32.
#include <algorithm>

#include "elem.hpp"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

struct AShape {
    int T, H, N, L, r;
};

constexpr int kFewRows = 128;       // rows that few_kernel and shrink_few take, in any order
constexpr int kOrderKeys = 1 << 13; // adapters that the order counts in LDS

// Whether the order of a given projection's rows pays for its launch: with it the
// shrink and the add meet few adapters in 16 rows.  H = N, mixed rows, bf16, us
// without and with it:
//   rows, adapters, rank     33         48         64         96
//   H 2,048  16  16        13.3 14.5  14.0 14.5  14.2 14.5  14.9 14.2
//            64  16        15.3 17.1  15.9 16.5  15.9 16.4  16.7 15.9
//            16  64        18.7 18.2  20.1 17.3  20.4 16.9  21.8 15.7
//            64  64        21.7 22.8  24.0 25.8  24.6 24.3  26.6 22.6
//   H 7,168  16  32        17.7 19.2  21.4 19.7  22.4 18.5  23.9 17.7
//            16  64        23.6 23.1  25.1 21.0  25.6 20.6  27.6 19.9
//            64  64        27.7 28.5  28.4 28.4  29.2 27.5  31.1 31.5
bool order_pays(const AShape &s)
{
    return s.T > 64 || (s.T > 40 && (long)s.r * s.H >= 1 << 17);
}

// D(16x16) += A(16x32) B(32x16): lane l holds A's row / B's column l mod 16
// at k = 8 (l div 16) .. + 7, and D's column l mod 16 at rows
// 4 (l div 16) .. + 3.
template <int DT>
__device__ __forceinline__ v4f mfma(const uint4 &a, const uint4 &b, v4f c)
{
    if constexpr (DT == MOE_DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                      __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// This thread's wavefront in the workgroup, in a scalar register: the matrix
// instruction does not look at which lanes are active, so every branch
// around one has to be a scalar branch.
__device__ __forceinline__ int wave_of()
{
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// s_waitcnt vmcnt(N) lgkmcnt(0).
template <int N>
__device__ __forceinline__ void wait_but()
{
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}

__device__ __forceinline__ const uint4 &piece(const uint16_t *p)
{
    return *reinterpret_cast<const uint4 *>(p);
}

// v as the sum of N bf16 values, each what the ones before it lack, cut to its
// upper 16 bits (so none is above that or of another sign); v[i] keeps the rest,
// a NaN where v was infinite.
template <int N>
__device__ __forceinline__ void cut8(float *v, uint4 *out)
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]),
                                         0x07060302);
        out[n] = uint4{w[0], w[1], w[2], w[3]};
        float h[8];
        Elem<MOE_DT_BF16>::unpack(out[n], h);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] -= h[i];
    }
}

// A row and its adapter (-1: none).
struct Row {
    int t, id;
};

// What place i holds, clamped to the last place, there without its adapter;
// order: the places' rows sorted by adapter, or null.
__device__ __forceinline__ Row row_at(const AShape &s, const Row *__restrict__ order,
                                      const int32_t *__restrict__ ids, long i)
{
    const long c = i < s.T ? i : s.T - 1;
    Row r;
    if (order) {
        r = order[c];
    } else {
        r = Row{(int)c, ids[c]};
        r.id = (unsigned)r.id < (unsigned)s.L ? r.id : -1;
    }
    return Row{r.t, i < s.T ? r.id : -1};
}

// Column of the output that row i (0..15) of the block f of 16 weight rows
// stands for: a lane then holds 8 neighbouring columns of its token in two
// blocks' sums, and the four lanes of a token 32 (64 whole bytes).
__device__ __forceinline__ int column_of(int f, int i)
{
    return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3);
}

// Place of workgroup b of n in a run that gives each XCD (neighbouring
// workgroups run on different ones) a contiguous part.
__device__ __forceinline__ int xcd_run(int b, int n)
{
    const int xcd = b & 7;
    return xcd * (n >> 3) + min(xcd, n & 7) + (b >> 3);
}

// ---------------------------------------------------------------------------
// Order: the rows by adapter, those without one last, as a list of rows
// (places inside an adapter in whatever order the claims land), and the
// blocks of up to `block` places that hold one adapter each.  One workgroup:
// a histogram (in LDS, or in the workspace past kOrderKeys adapters), its
// scan, and a claim of a place per row.  A wavefront whose rows share an
// adapter claims with one atomic.  Bound by its chain of loads and atomics:
// 8,191 rows of 16 adapters 10 us, 4,097 of 96 7; past 8,192 rows each claims
// twice, 65,536 take 50 to 54.
// ---------------------------------------------------------------------------
constexpr int kOrderThreads = 1024, kOrderBatch = 8;

// Places first .. first + rows - 1 hold rows of one adapter.
struct Block {
    int id, first, rows, pad;
};

struct OrderOut {
    Row *order;      // T
    int32_t *blocks; // how many
    Block *block;    // T / rows + L at most
    int32_t *count;  // L + 1 of scratch, or null: in LDS
};

__global__ void __launch_bounds__(kOrderThreads)
order_kernel(AShape s, int rows, const int32_t *__restrict__ ids, OrderOut o)
{
    extern __shared__ int lds_count[]; // L + 1
    __shared__ int wsum[2][kOrderThreads / 64];
    int *count = o.count ? o.count : lds_count;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int keys = s.L + 1;
    for (int i = tid; i < keys; i += kOrderThreads)
        count[i] = 0;
    __syncthreads();
    // claims one place of key k for every lane with in set
    const auto claim = [&](int k, bool in) -> int {
        const uint64_t act = __ballot(in);
        if (!act)
            return 0;
        const int first = __builtin_ctzll(act);
        const int k0 = __builtin_amdgcn_readlane(k, first);
        if (__ballot(in && k != k0) == 0) {
            int at = 0;
            if (lane == first)
                at = atomicAdd(&count[k0], __builtin_popcountll(act));
            at = __builtin_amdgcn_readlane(at, first);
            return at + __builtin_popcountll(act & ((1ull << lane) - 1));
        }
        return in ? atomicAdd(&count[k], 1) : 0;
    };
    // f(q, row, its key, whether there is such a row), kOrderBatch loads at once
    const auto walk = [&](auto f) {
        for (long b = 0; b < s.T; b += kOrderThreads * kOrderBatch) {
            int id[kOrderBatch];
#pragma unroll
            for (int q = 0; q < kOrderBatch; ++q)
                id[q] = ids[min(b + q * kOrderThreads + tid, (long)s.T - 1)];
#pragma unroll
            for (int q = 0; q < kOrderBatch; ++q) {
                const long t = b + q * kOrderThreads + tid;
                f(q, (int)t, (unsigned)id[q] < (unsigned)s.L ? id[q] : s.L, t < s.T);
            }
        }
    };
    // a claim's answer is the row's place inside its adapter: up to one batch
    // of rows keeps it, more claim a second time, from the adapters' places on
    const bool one = s.T <= kOrderThreads * kOrderBatch;
    int place[kOrderBatch], key[kOrderBatch];
    walk([&](int q, int, int k, bool in) {
        const int at = claim(k, in);
        if (one) {
            place[q] = at;
            key[q] = k;
        }
    });
    __syncthreads();
    // exclusive scans of the counts and of the blocks, a run of keys a thread
    const int per = (keys + kOrderThreads - 1) / kOrderThreads;
    const int b = min(keys, tid * per), e = min(keys, b + per);
    int sum[2] = {0, 0};
    for (int i = b; i < e; ++i) {
        const int c = count[i];
        sum[0] += c;
        sum[1] += i < s.L ? (c + rows - 1) / rows : 0;
    }
    int inc[2] = {sum[0], sum[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(inc[h], d);
            if (lane >= d)
                inc[h] += u;
        }
        if (lane == 63)
            wsum[h][wave] = inc[h];
    }
    __syncthreads();
    int run = inc[0] - sum[0], at = inc[1] - sum[1];
    for (int w = 0; w < wave; ++w) {
        run += wsum[0][w];
        at += wsum[1][w];
    }
    for (int i = b; i < e; ++i) {
        const int c = count[i];
        count[i] = run;
        if (i < s.L)
            for (int q = 0; q < c; q += rows)
                o.block[at++] = Block{i, run + q, min(rows, c - q), 0};
        run += c;
    }
    if (tid == kOrderThreads - 1)
        *o.blocks = at;
    __syncthreads();
    if (one) {
#pragma unroll
        for (int q = 0; q < kOrderBatch; ++q) {
            const int t = q * kOrderThreads + tid;
            if (t < s.T)
                o.order[count[key[q]] + place[q]] = Row{t, key[q] < s.L ? key[q] : -1};
        }
        return;
    }
    walk([&](int, int t, int k, bool in) {
        const int at = claim(k, in);
        if (in)
            o.order[at] = Row{t, k < s.L ? k : -1};
    });
}

// ---------------------------------------------------------------------------
// Stream: BM rows of x by BN rows of a weight (W or A), bound by reading
// them.  A step is KB bytes (128 or 256) of every row; a load instruction
// moves whole KB-byte pieces of 1024 / KB rows from global memory to LDS, so
// it asks for whole cache lines (a wavefront reading its operands straight
// into registers touches 16 rows by 64 bytes at a time, and half lines come
// from the L2 at a third of the rate: 36 against 105 KB/us a CU).  The 16-byte
// pieces of a row are stored where the 16 rows that one operand read touches
// lie in different banks.
//
// Half the wavefronts load x, half the weight, each into its own ring of
// stages (NX, NR): a wavefront's loads end in order, so in one ring the
// operand that comes from the L2 would wait for the one that comes from
// memory, and the rings' depths could not differ.  Little's law sets them:
// about 2 us of latency from memory at 25 KB/us a CU.
//
// A wavefront multiplies 64 bytes of every step (one matrix instruction deep)
// for a block of WM x WN of the tile; the KB / 64 sums of a block meet in LDS
// at the end, in a fixed order.  kOnce: the weight is read by no other
// workgroup and leaves the L2 first.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int NX, int NR, int KB, bool kOnce = true>
struct Stream {
    static_assert(KB == 128 || KB == 256, "one or two cache lines of a row");
    static constexpr int kSlices = KB / 64, kWaves = kSlices * WM * WN, kThreads = 64 * kWaves;
    static constexpr int kBM = BM, kBN = BN, MF = BM / WM / 16, NF = BN / WN / 16;
    static constexpr int kRows = 1024 / KB; // rows of a load
    // loads per wavefront and step
    static constexpr int UX = BM / kRows / (kWaves / 2), UR = BN / kRows / (kWaves / 2);
    static constexpr int kX = BM * KB, kR = BN * KB; // bytes of a stage
    static constexpr int kLds = NX * kX + NR * kR;
    static_assert(UX * kRows * kWaves / 2 == BM && UR * kRows * kWaves / 2 == BN, "whole loads");
    static_assert(MF * WM * 16 == BM && NF * WN * 16 == BN, "whole blocks");
    static_assert((NX - 2) * UX < 64 && (NR - 2) * UR < 64, "loads that vmcnt can count");
    static_assert(kSlices * (BM / 16) * (BN / 16) * 1024 <= kLds, "the sums reuse the stages");
};

// Place of the 16-byte piece c of row i.
template <int KB>
__device__ __forceinline__ int place_of(int c, int i)
{
    return KB == 256 ? c ^ (i & 15) : c ^ ((i >> 1) & 7);
}

// One wavefront's loads into one ring: U a step, N stages of kStage bytes
// from lds0; kOnce: read once, to leave the L2 first.  Loads past the last
// step repeat it into stages that nobody reads again, so the number in flight
// stays the same to the end.
template <int U, int N, int kStage, int KB, bool kOnce>
struct Ring {
    const uint8_t *next;
    uint32_t voff[U], lds0, slot;
    int left; // steps after the next one

    // `first`: this wavefront's first load of a stage; row(i): number of the
    // stage's row i in the array at p
    template <typename Row>
    __device__ __forceinline__ Ring(const uint16_t *p, int H, int steps, int first, uint32_t lds,
                                    Row row)
        : next(reinterpret_cast<const uint8_t *>(p)), lds0(lds + first * 1024), slot(0),
          left(steps - 1)
    {
        const int lane = threadIdx.x & 63;
        constexpr int kPieces = KB / 16;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = (first + u) * (1024 / KB) + lane / kPieces;
            voff[u] = (uint32_t)row(i) * (uint32_t)(2 * H) +
                      place_of<KB>(lane & (kPieces - 1), i) * 16;
        }
    }
    __device__ __forceinline__ void load()
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            g2lds<16, kOnce>(next, voff[u], lds0 + slot + u * 1024);
        slot = slot + kStage == N * kStage ? 0 : slot + kStage;
        next += left > 0 ? KB : 0;
        --left;
    }
    __device__ __forceinline__ void start()
    {
        for (int k = 0; k < N - 1; ++k)
            load();
    }
    // this wavefront's part of the oldest step has landed, and what it read
    // of the step before is in registers
    __device__ __forceinline__ void wait() { wait_but<(N - 2) * U>(); }
};

// `steps` steps from x and w on.  Rows [0, BM) come from x, columns [0, BN)
// from the rows of w: xrow(i) and wrow(i) give their numbers, w's within
// 2^31 bytes of its base.  Afterwards wavefront v holds the blocks of 16
// rows v, v + kWaves, ... in sum, BN / 16 values a block.
template <int DT, int BM, int BN, int WM, int WN, int NX, int NR, int KB, bool kOnce,
          typename XRow, typename WRow>
__device__ __forceinline__ void stream_tile(Stream<BM, BN, WM, WN, NX, NR, KB, kOnce>, int H, int steps,
                                            const uint16_t *__restrict__ x, XRow xrow,
                                            const uint16_t *__restrict__ w, WRow wrow,
                                            uint8_t *lds, v4f *sum)
{
    using S = Stream<BM, BN, WM, WN, NX, NR, KB, kOnce>;
    constexpr int MF = S::MF, NF = S::NF, kHalf = S::kWaves / 2;
    const int lane = threadIdx.x & 63, wave = wave_of();
    const uint32_t l0 = lds_addr(lds);
    const int slice = wave % S::kSlices, block = wave / S::kSlices;
    const int wm = block / WN, wn = block % WN;
    const int off = (lane & 15) * KB + place_of<KB>(4 * slice + (lane >> 4), lane & 15) * 16;
    v4f acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const auto go = [&](auto ring) {
        ring.start();
        const uint8_t *xl = lds + off + wm * MF * 16 * KB;
        const uint8_t *wl = lds + NX * S::kX + off + wn * NF * 16 * KB;
        int xs = 0, ws = 0;
        for (int k = steps; k > 0; --k) {
            // the step has landed, and the one before it is done with
            // everywhere: its stage takes the next load
            ring.wait();
            raw_barrier();
            uint4 xq[MF], wq[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f)
                wq[f] = *reinterpret_cast<const uint4 *>(wl + ws + 16 * f * KB);
#pragma unroll
            for (int m = 0; m < MF; ++m)
                xq[m] = *reinterpret_cast<const uint4 *>(xl + xs + 16 * m * KB);
            ring.load();
            xs = xs + S::kX == NX * S::kX ? 0 : xs + S::kX;
            ws = ws + S::kR == NR * S::kR ? 0 : ws + S::kR;
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[m][f] = mfma<DT>(wq[f], xq[m], acc[m][f]);
        }
    };
    if (wave < kHalf)
        go(Ring<S::UX, NX, S::kX, KB, false>(x, H, steps, wave * S::UX, l0, xrow));
    else
        go(Ring<S::UR, NR, S::kR, KB, kOnce>(w, H, steps, (wave - kHalf) * S::UR,
                                           l0 + NX * S::kX, wrow));
    wait_vmcnt<0>();
    __syncthreads();
    constexpr int MB = BM / 16, NB = BN / 16;
    v4f *part = reinterpret_cast<v4f *>(lds);
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            part[((slice * MB + wm * MF + m) * NB + wn * NF + f) * 64 + lane] = acc[m][f];
    __syncthreads();
#pragma unroll
    for (int q = 0; q * S::kWaves < MB; ++q) {
        const int m = q * S::kWaves + wave;
        if (m >= MB)
            break;
#pragma unroll
        for (int f = 0; f < NB; ++f) {
            v4f a = part[(m * NB + f) * 64 + lane];
#pragma unroll
            for (int k = 1; k < S::kSlices; ++k)
                a += part[((k * MB + m) * NB + f) * 64 + lane];
            sum[q * NB + f] = a;
        }
    }
}

// ---------------------------------------------------------------------------
// Shrink, few rows (up to kFewRows, in any order): a task is up to 16 rows of
// one adapter by the S::kBN of the rank, and a workgroup takes every blocks-th
// task.  The first of each sixteen rows of an adapter stands for it, so
// every adapter's A is read as few times as its rows allow.
// ---------------------------------------------------------------------------
using FewStream = Stream<16, 16, 1, 1, 16, 16, 256>;  // four wavefronts
using FewStream8 = Stream<16, 32, 1, 2, 8, 12, 256>;  // eight

template <int DT, typename S>
__device__ __forceinline__ void shrink_few(const AShape &s, const uint16_t *__restrict__ x,
                                           const int32_t *__restrict__ ids,
                                           const uint16_t *__restrict__ a, float *__restrict__ v,
                                           int block, int blocks, uint8_t *lds)
{
    static_assert(S::kThreads >= kFewRows, "a thread looks at one row");
    constexpr int kGroups = kFewRows / 64;
    __shared__ int32_t id_of[kFewRows];
    __shared__ uint64_t firsts[kGroups];
    __shared__ int lead[kFewRows], member[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_of();
    int id = -1;
    if (tid < s.T && (unsigned)ids[tid] < (unsigned)s.L)
        id = ids[tid];
    if (tid < kFewRows)
        id_of[tid] = id;
    __syncthreads();
    // rows of the same adapter before this one
    int rank = 0;
    for (int u = 0; u < min(tid, s.T); ++u)
        rank += id_of[u] == id;
    const bool leads = id >= 0 && rank % 16 == 0;
    const uint64_t m = __ballot(leads);
    if (lane == 0 && wave < kGroups)
        firsts[wave] = m;
    __syncthreads();
    int n = 0, at = 0;
    for (int w = 0; w < kGroups; ++w) {
        at += w < wave ? __builtin_popcountll(firsts[w]) : 0;
        n += __builtin_popcountll(firsts[w]);
    }
    if (leads)
        lead[at + __builtin_popcountll(m & ((1ull << lane) - 1))] = tid | rank << 16;
    const int nj = (s.r + S::kBN - 1) / S::kBN;
    for (int task = block; task < n * nj; task += blocks) {
        if (tid < 16)
            member[tid] = -1;
        __syncthreads();
        const int first = __builtin_amdgcn_readfirstlane(lead[task / nj]);
        const int t = first & 0xffff, g = __builtin_amdgcn_readfirstlane(id_of[t]);
        if (id == g && (unsigned)(rank - (first >> 16)) < 16u)
            member[rank - (first >> 16)] = tid;
        __syncthreads();
        const int j0 = task % nj * S::kBN;
        v4f sum[S::kBN / 16];
        stream_tile<DT>(
            S{}, s.H, s.H / 128, x, [&](int i) { return member[i] < 0 ? t : member[i]; },
            a + (size_t)g * s.r * s.H, [&](int i) { return min(j0 + i, s.r - 1); }, lds, sum);
        const int row = member[lane & 15];
        if (wave == 0 && row >= 0)
#pragma unroll
            for (int f = 0; f < S::kBN / 16; ++f) {
                const int j = j0 + 16 * f + 4 * (lane >> 4);
                if (j < s.r)
                    *reinterpret_cast<v4f *>(v + (size_t)row * s.r + j) = sum[f];
            }
        __syncthreads();
    }
}

template <int DT>
__global__ void __launch_bounds__(FewStream::kThreads)
shrink_few_kernel(AShape s, const uint16_t *__restrict__ x, const int32_t *__restrict__ ids,
                  const uint16_t *__restrict__ a, float *__restrict__ v)
{
    __shared__ __align__(1024) uint8_t lds[FewStream::kLds];
    shrink_few<DT, FewStream>(s, x, ids, a, v, blockIdx.x, gridDim.x, lds);
}

// Shrink, many rows, ordered (8,191 rows of 7,168 bf16 values by rank 64: 40 us,
// 130 MB read at 3.2 TB/s): workgroup (a block of up to BM places of one
// adapter, BN of the rank).
template <int DT, int BM, int BN, int WM, int NX, int NR>
__global__ void __launch_bounds__((Stream<BM, BN, WM, 1, NX, NR, 256, false>::kThreads))
shrink_many_kernel(AShape s, const uint16_t *__restrict__ x, OrderOut o,
                   const uint16_t *__restrict__ a, float *__restrict__ v)
{
    using S = Stream<BM, BN, WM, 1, NX, NR, 256, false>;
    __shared__ __align__(1024) uint8_t lds[S::kLds];
    const int n = *o.blocks, lane = threadIdx.x & 63, wave = wave_of();
    const int j0 = blockIdx.y * BN;
    for (int q = blockIdx.x; q < n; q += gridDim.x) {
        // an XCD's blocks lie together: few adapters' A in its L2
        const Block b = o.block[n <= (int)gridDim.x ? xcd_run(q, n) : q];
        v4f sum[BN / 16];
        stream_tile<DT>(
            S{}, s.H, s.H / 128, x,
            [&](int i) { return o.order[b.first + min(i, b.rows - 1)].t; },
            a + (size_t)b.id * s.r * s.H, [&](int i) { return min(j0 + i, s.r - 1); }, lds, sum);
        const int i = 16 * wave + (lane & 15);
        if (wave < BM / 16 && i < b.rows) {
            float *vr = v + (size_t)o.order[b.first + i].t * s.r;
#pragma unroll
            for (int f = 0; f < BN / 16; ++f) {
                const int j = j0 + 16 * f + 4 * (lane >> 4);
                if (j < s.r)
                    *reinterpret_cast<v4f *>(vr + j) = sum[f];
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Expand: adds the adapters' term of 16 rows (the lane's: row) to the sums of
// 16 NF columns from n0 (in column_of's order).
// 32 KK of the rank at a time: the rows' v in bf16 parts, then the adapters among
// the rows, GB at a time with their B in flight together.  No load stands
// behind a branch (a lane or a place without work reads a valid address and
// drops the product): behind one the compiler waits for each by itself.
// ---------------------------------------------------------------------------

// 32 KK of the rank of the lane's row, from c: pieces k0 + 32 k of 8, each as
// hi, mid and lo.
template <int KK>
struct Low {
    uint4 v[KK][3];
    int at[KK];
    bool there[KK];
};

// The scale of a row's adapter.
__device__ __forceinline__ float scale_of(const float *__restrict__ scale, const Row &row)
{
    return scale ? scale[max(row.id, 0)] : 1.0f;
}

template <int KK>
__device__ __forceinline__ Low<KK> low_of(const AShape &s, const float *__restrict__ v,
                                          const Row &row, int c)
{
    const float *vr = v + (size_t)row.t * s.r;
    const int k0 = 8 * ((threadIdx.x & 63) >> 4);
    Low<KK> low;
    v4f vq[KK][2];
#pragma unroll
    for (int k = 0; k < KK; ++k) {
        low.there[k] = c + 32 * k + k0 < s.r;
        low.at[k] = low.there[k] ? c + 32 * k + k0 : 0;
        vq[k][0] = *reinterpret_cast<const v4f *>(vr + low.at[k]);
        vq[k][1] = *reinterpret_cast<const v4f *>(vr + low.at[k] + 4);
    }
#pragma unroll
    for (int k = 0; k < KK; ++k) {
        float f8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f8[i] = low.there[k] && row.id >= 0 ? vq[k][i >> 2][i & 3] : 0.0f;
        cut8<3>(f8, low.v[k]);
    }
    return low;
}

// One block's product with 32 KK of the rank: b as NB bf16 values, v as three,
// the smallest products first.
template <int NB, int KK>
__device__ __forceinline__ v4f product(const uint4 (*b)[NB], const uint4 (*v)[3])
{
    v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int o = NB + 1; o >= 0; --o)
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int h = 0; h < NB; ++h)
                if (o - h >= 0 && o - h < 3)
                    d = mfma<MOE_DT_BF16>(b[k][h], v[k][o - h], d);
    return d;
}

// q's bf16 values, 0 where those of `by` are infinities or NaN.
__device__ __forceinline__ uint4 where_finite(const uint4 &q, const uint4 &by)
{
    const auto one = [](uint32_t x, uint32_t y) {
        const uint32_t lo = (y & 0x7f80u) == 0x7f80u ? 0u : 0xffffu;
        const uint32_t hi = (y & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u;
        return x & (lo | hi);
    };
    return uint4{one(q.x, by.x), one(q.y, by.y), one(q.z, by.z), one(q.w, by.w)};
}

// The same where a factor is infinite or NaN.  Its first bf16 value is too, and
// multiplies the other factor's first value alone, which is 0 only where that
// factor is: the values behind may be 0, and 0 times an infinity a NaN.
template <int NB, int KK>
__device__ __forceinline__ v4f careful(const uint4 (*b)[NB], const uint4 (*v)[3])
{
    uint4 bf[KK][NB], vf[KK][3];
#pragma unroll
    for (int k = 0; k < KK; ++k) {
#pragma unroll
        for (int h = 0; h < NB; ++h)
            bf[k][h] = where_finite(b[k][h], b[k][0]);
#pragma unroll
        for (int h = 0; h < 3; ++h)
            vf[k][h] = where_finite(v[k][h], v[k][0]);
    }
    v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int o = NB + 1; o >= 0; --o)
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int h = 0; h < NB; ++h)
                if (o - h >= 0 && o - h < 3)
                    d = mfma<MOE_DT_BF16>(o ? bf[k][h] : b[k][0], o ? vf[k][o - h] : v[k][0], d);
    return d;
}

// Adds 32 KK of the rank to M blocks of 16 rows; rows[m]: which rows of block
// m have an adapter.  An adapter's B is loaded once for all the blocks.  Returns
// whether a product of this lane's rows is left out, not being finite: those
// are added, and nothing else, by a second call (kAgain).
template <int DT, int M, int NF, int GB, int KK, bool kAgain = false>
__device__ __forceinline__ bool expand_part(const AShape &s, const uint16_t *__restrict__ b,
                                            const Row *row, const uint32_t *rows,
                                            const float *scale, const Low<KK> *low, int n0,
                                            v4f (*acc)[NF])
{
    const int lane = threadIdx.x & 63;
    uint32_t col[NF]; // element of B_l; N * rank is below 2^28
#pragma unroll
    for (int f = 0; f < NF; ++f)
        col[f] = (uint32_t)min(n0 + column_of(f, lane & 15), s.N - 1) * s.r;
    uint32_t todo[M], any = 0;
    bool left_out = false;
#pragma unroll
    for (int m = 0; m < M; ++m)
        any |= todo[m] = rows[m];
    while (any) {
        int g[GB], n = 0;
        uint4 bq[GB][KK][NF];
#pragma unroll
        for (int q = 0; q < GB; ++q) {
            int next = -1;
#pragma unroll
            for (int m = M - 1; m >= 0; --m)
                if (todo[m])
                    next = __builtin_amdgcn_readlane(row[m].id, __builtin_ctz(todo[m]));
            n += next >= 0 ? 1 : 0;
            g[q] = next >= 0 ? next : g[0];
            any = 0;
#pragma unroll
            for (int m = 0; m < M; ++m)
                any |= todo[m] &= ~(uint32_t)__ballot(row[m].id == g[q]);
        }
#pragma unroll
        for (int q = 0; q < GB; ++q) {
            const uint16_t *bg = b + (size_t)g[q] * s.N * s.r;
#pragma unroll
            for (int k = 0; k < KK; ++k)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    bq[q][k][f] = piece(bg + col[f] + low[0].at[k]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < GB; ++q) {
            if (q >= __builtin_amdgcn_readfirstlane(n))
                break;
            constexpr int NB = DT == MOE_DT_F16 ? 2 : 1; // bf16 values of one of B
            uint4 bk[NF][KK][NB];
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    const uint4 p = low[0].there[k] ? bq[q][k][f] : uint4{0, 0, 0, 0};
                    if constexpr (DT == MOE_DT_F16) {
                        float f8[8];
                        Elem<DT>::unpack(p, f8);
                        cut8<NB>(f8, bk[f][k]);
                    } else {
                        bk[f][k][0] = p;
                    }
                }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const bool take = row[m].id == g[q];
                if (M > 1 && !__any(take))
                    continue;
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    v4f d = product<NB, KK>(bk[f], low[m].v);
                    const bool finite =
                        fabsf(d[0]) + fabsf(d[1]) + fabsf(d[2]) + fabsf(d[3]) < INFINITY;
                    left_out |= take && !finite;
                    if constexpr (kAgain)
                        d = careful<NB, KK>(bk[f], low[m].v);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (take && finite != kAgain) // (adding 0 would change a -0)
                            acc[m][f][i] += scale[m] * d[i];
                }
            }
        }
    }
    return left_out;
}

// The whole term for M blocks of 16 rows, 32 KK of the rank at a time.
template <int DT, int M, int NF, int GB, int KK>
__device__ __forceinline__ void expand(const AShape &s, const float *__restrict__ v,
                                       const uint16_t *__restrict__ b,
                                       const float *__restrict__ scale, const Row *row, int n0,
                                       v4f (*acc)[NF])
{
    uint32_t rows[M], any = 0;
    float sc[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        any |= rows[m] = (uint32_t)__ballot(row[m].id >= 0) & 0xffffu;
    if (!any)
        return;
#pragma unroll
    for (int m = 0; m < M; ++m)
        sc[m] = scale_of(scale, row[m]);
    bool left_out = false;
    for (int c = 0; c < s.r; c += 32 * KK) {
        Low<KK> low[M];
#pragma unroll
        for (int m = 0; m < M; ++m)
            low[m] = low_of<KK>(s, v, row[m], c);
        left_out |= expand_part<DT, M, NF, GB, KK>(s, b, row, rows, sc, low, n0, acc);
    }
    if (!__any(left_out))
        return;
    // (what is left out is the products of the same 32 KK)
#pragma unroll
    for (int m = 0; m < M; ++m)
        for (int c = 0; c < s.r; c += 32 * KK) {
            const Low<KK> low = low_of<KK>(s, v, row[m], c);
            expand_part<DT, 1, NF, 1, KK, true>(s, b, row + m, rows + m, sc + m, &low, n0, acc + m);
        }
}

// A lane's sums of 16 NF columns from n0 of row t, rounded and stored in
// pieces of 8 (N is a multiple of 8).  The stores leave the L2 first: with
// ordinary ones the rows and weights that other workgroups read again leave
// earlier (whole calls: adding to 4,097 x 5,120 fp16 values 46 us, so 40; 8,191 x
// 7,168 x 7,168 bf16 728, so 704).
template <int DT, int NF>
__device__ __forceinline__ void store_cols(const AShape &s, uint16_t *out, int t, int n0,
                                           const v4f *acc)
{
    const int n = n0 + 8 * ((threadIdx.x & 63) >> 4);
    uint16_t *o = out + (size_t)t * s.N + n;
#pragma unroll
    for (int p = 0; p < NF / 2; ++p) {
        const v4f a = acc[2 * p], b = acc[2 * p + 1];
        const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        if (n + 32 * p < s.N)
            store_once(o + 32 * p, Elem<DT>::pack(f));
    }
}

// The order of up to kFewRows rows, by one workgroup: a row's place is the
// count of rows before it, by adapter and row, those without one last.  The
// add then meets one or two adapters in 16 rows and reads B once: 128 rows at
// 1,024 x 6,144 with 32 adapters of rank 64 take 31 us, in the caller's order 39,
// of rank 16 18 and 20.
__device__ __forceinline__ void order_few(const AShape &s, const int32_t *__restrict__ ids,
                                          Row *__restrict__ order, int32_t *key)
{
    const int tid = threadIdx.x;
    const int id = tid < s.T && (unsigned)ids[tid] < (unsigned)s.L ? ids[tid] : -1;
    const uint32_t mine = (uint32_t)id; // -1 orders last
    if (tid < s.T)
        key[tid] = id;
    __syncthreads();
    int place = 0;
    for (int u = 0; u < s.T; ++u)
        place += (uint32_t)key[u] < mine || ((uint32_t)key[u] == mine && u < tid);
    if (tid < s.T)
        order[place] = Row{tid, id};
}

// ---------------------------------------------------------------------------
// Project, few rows: W is read once.  One launch makes v and the order (its
// workgroups last) and, beside them, parts of x W^T: a workgroup takes all
// rows (up to BM), BN columns and one of `splits` parts of H, and leaves
// float32 sums; the add launch joins the parts and adds the adapters' term.
// Splitting H gives every CU work without more copies of x than columns ask
// for, and the adapters' chain of loads does not stand at the end of W's.
// order is null for 16 rows, whose add is one block in any order.
// Bound by reading W and A: 1 x 5,120 by 4,608 takes 12 us (4.0 TB/s), 128 x
// 7,168 by 7,168 with 64 adapters of rank 32 33 us (145 MB, 4.5 TB/s); a step
// of the 128-row tile multiplies in a fifth of that time.
// ---------------------------------------------------------------------------
template <int DT, typename S, typename F>
__global__ void __launch_bounds__(S::kThreads)
few_kernel(AShape s, int tn, int splits, const uint16_t *__restrict__ x,
           const uint16_t *__restrict__ w, const int32_t *__restrict__ ids,
           const uint16_t *__restrict__ a, float *__restrict__ v, float *__restrict__ parts,
           Row *__restrict__ order)
{
    static_assert(S::kThreads == F::kThreads, "one launch for both");
    constexpr int kLds = S::kLds > F::kLds ? S::kLds : F::kLds, BM = S::kBM;
    __shared__ __align__(1024) uint8_t lds[kLds];
    const int q = blockIdx.x, other = tn * splits + (order != nullptr);
    if (q >= other) {
        shrink_few<DT, F>(s, x, ids, a, v, q - other, gridDim.x - other, lds);
        return;
    }
    if (q == tn * splits) {
        order_few(s, ids, order, reinterpret_cast<int32_t *>(lds));
        return;
    }
    const int n0 = q % tn * S::kBN, part = q / tn;
    const int all = s.H / 64, first = (long)all * part / splits;
    const int steps = (int)((long)all * (part + 1) / splits) - first;
    constexpr int NB = S::kBN / 16;
    v4f sum[NB * ((BM / 16 + S::kWaves - 1) / S::kWaves)];
    stream_tile<DT>(
        S{}, s.H, steps, x + 64 * first, [&](int r) { return min(r, s.T - 1); },
        w + (size_t)n0 * s.H + 64 * first,
        [&](int r) {
            return min(column_of(r >> 4, r & 15), s.N - 1 - n0);
        },
        lds, sum);
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 0; m * S::kWaves < BM / 16; ++m) {
        const int t = 16 * (m * S::kWaves + wave_of()) + (lane & 15);
        if (t < min(s.T, BM))
#pragma unroll
            for (int f = 0; f < NB; ++f) {
                const int n = n0 + column_of(f, 4 * (lane >> 4));
                if (n < s.N)
                    *reinterpret_cast<v4f *>(parts + ((size_t)part * s.T + t) * s.N + n) =
                        sum[m * NB + f];
            }
    }
}

// ---------------------------------------------------------------------------
// Project, many rows: BM places x BN columns per workgroup, WM x WN
// wavefronts of 16 MF rows x 16 NF columns.  K steps of 64 values (128 bytes
// a row) go from global memory to LDS without registers, two stages.  A
// row's eight 16-byte pieces are stored at piece ^ (row / 2 mod 8): the 16
// rows that one operand read touches then lie in different banks.
//
// Operands are read from LDS one phase ahead of their matrix instructions,
// into a second set of registers, a few reads between every few matrix
// instructions.  The last phase of a step reads the next stage and sends off
// the loads of the step after it, into the stage that all wavefronts have
// just finished reading: one barrier a step, and a step's time for its loads.
// Bound by the matrix instructions and what of the loads they do not cover: at
// 8,191 x 7,168 x 7,168 bf16 they hold the matrix cores for two thirds of 670 to
// 727 us (1.2 PFLOP/s with the adapters' term; 896 tiles are 3.5 rounds of 256 CUs).
// ---------------------------------------------------------------------------

// Tile q of tm x tn: down 8 row tiles before the next column tile, so the
// tiles that run together on an XCD share rows and columns in its L2.
__device__ __forceinline__ void tile_of(int q, int tm, int tn, int *im, int *in)
{
    const int group = q / (8 * tn), first = group * 8;
    const int rows = min(8, tm - first), in_group = q - group * 8 * tn;
    *im = first + in_group % rows;
    *in = in_group / rows;
}

constexpr int kRowBytes = 128; // of a row's step

struct ProjectArgs {
    const uint16_t *x, *w;
    const Row *order; // tiles are of ordered rows
    const uint16_t *b;
    const float *scale, *v;
    uint16_t *out;
    float *parts;
};

// The rows of places m0 .. m0 + BM - 1 by the columns n0 .. n0 + BN - 1: out,
// or (kParts) the float32 sums over `steps` steps (even) from `first` on, as
// plane `part` of p.parts.
template <int DT, int BM, int BN, int WM, int WN, int NS = 2, bool kParts = false>
__device__ __forceinline__ void project_tile(const AShape &s, const ProjectArgs &p, long m0,
                                             int n0, uint8_t *lds, int first, int steps,
                                             int part = 0)
{
    constexpr int NW = WM * WN, MF = BM / WM / 16, NF = BN / WN / 16;
    static_assert(NF % 4 == 0 && (BM + BN) % (8 * NW) == 0, "wavefronts cover the tile");
    constexpr int U = (BM + BN) / 8 / NW; // 1 KiB loads per wavefront and step
    constexpr int kStage = (BM + BN) * kRowBytes;
    const int lane = threadIdx.x & 63, wave = wave_of();

    // this lane's byte offsets: load u covers 8 LDS rows, x's first
    uint32_t voff[U];
    const uint8_t *base[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = (wave * U + u) * 8 + (lane >> 3);
        const int at = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        if ((wave * U + u) * 8 < BM) {
            const long i = min(m0 + row, (long)s.T - 1);
            voff[u] = (uint32_t)p.order[i].t * (uint32_t)(2 * s.H) + at;
            base[u] = reinterpret_cast<const uint8_t *>(p.x);
        } else {
            const int rw = row - BM;
            const int n = column_of(rw >> 4, rw & 15);
            const int nc = min(n, s.N - 1 - n0);
            voff[u] = (uint32_t)nc * (uint32_t)(2 * s.H) + at;
            base[u] = reinterpret_cast<const uint8_t *>(p.w + (size_t)n0 * s.H);
        }
    }
    const uint32_t l0 = lds_addr(lds);
    const auto load = [&](int u, int step, int buf) {
        g2lds<16>(base[u] + (size_t)(first + step) * kRowBytes, voff[u],
                  l0 + buf * kStage + (wave * U + u) * 1024);
    };

    const int wm = wave / WN, wn = wave % WN;
    const int off = (lane & 15) * kRowBytes + (((lane >> 4) ^ ((lane & 15) >> 1)) * 16);
    const uint8_t *xl = lds + wm * MF * 16 * kRowBytes;
    const uint8_t *wl = lds + (BM + wn * NF * 16) * kRowBytes;
    v4f acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // The phases of a step: half k of its 64 values, a group of 4 of the
    // wavefront's row blocks.  Phase p multiplies the operands in sets p mod 2
    // (x) and k (w) and reads those of phase p + 1 into the other sets.
    constexpr int G = MF / 4, P = 2 * G;
    static_assert(MF % 4 == 0, "row blocks in groups of four");
    uint4 xo[2][4], wo[2][NF];
    const auto read_x = [&](int q, int ph, int buf) {
        xo[ph & 1][q] = *reinterpret_cast<const uint4 *>(
            xl + buf * kStage + ((ph % G) * 4 + q) * 16 * kRowBytes + (off ^ (64 * (ph / G))));
    };
    const auto read_w = [&](int f, int k, int buf) {
        wo[k][f] = *reinterpret_cast<const uint4 *>(wl + buf * kStage + f * 16 * kRowBytes +
                                                    (off ^ (64 * k)));
    };
    // step k in stage buf: the next stage holds step k + 1 before the last
    // phase, which also sends off the loads of step k + NS into this stage
    const auto step_of = [&](int k, int buf, int next, int last) {
#pragma unroll
        for (int ph = 0; ph < P; ++ph) {
            const bool end = ph + 1 == P;
            const int np = end ? 0 : ph + 1, nbuf = end ? next : buf;
            if (end) {
                wait_but<(NS - 2) * U>();
                raw_barrier();
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                read_x(q, np, nbuf);
                if (np % G == 0)
#pragma unroll
                    for (int f = q * NF / 4; f < (q + 1) * NF / 4; ++f)
                        read_w(f, np / G, nbuf);
                if (end)
#pragma unroll
                    for (int u = q * U / 4; u < (q + 1) * U / 4; ++u)
                        load(u, min(k + NS, last), buf);
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    v4f &a = acc[(ph % G) * 4 + q][f];
                    a = mfma<DT>(wo[ph / G][f], xo[ph & 1][q], a);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    static_assert(P % 2 == 0, "the next step starts with x's set 0");
    // (loads past the last step repeat it, unused)
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
            load(u, min(k, steps - 1), k);
    wait_vmcnt<(NS - 1) * U>();
    raw_barrier();
#pragma unroll
    for (int q = 0; q < 4; ++q)
        read_x(q, 0, 0);
#pragma unroll
    for (int f = 0; f < NF; ++f)
        read_w(f, 0, 0);
    if constexpr (NS == 2) {
        for (int k = 0; k < steps; k += 2) {
            step_of(k, 0, 1, steps - 1);
            step_of(k + 1, 1, 0, steps - 1);
        }
    } else {
        int buf = 0;
        for (int k = 0; k < steps; ++k) {
            const int next = buf + 1 == NS ? 0 : buf + 1;
            step_of(k, buf, next, steps - 1);
            buf = next;
        }
    }
    wait_but<0>();

    Row row[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
        row[m] = row_at(s, p.order, nullptr, m0 + (wm * MF + m) * 16 + (lane & 15));
    if constexpr (kParts) {
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            if (m0 + (wm * MF + m) * 16 + (lane & 15) >= s.T)
                continue;
            float *o = p.parts + ((size_t)part * s.T + row[m].t) * s.N;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int n = n0 + wn * NF * 16 + column_of(f, 4 * (lane >> 4));
                if (n < s.N)
                    *reinterpret_cast<v4f *>(o + n) = acc[m][f];
            }
        }
        return;
    }
    static_assert(NF == 4 && MF % 4 == 0, "four blocks of rows at a time");
    // 64 of the rank at a time (whole lines of B) where one workgroup has the CU's
    // registers (512 x 7,168 x 7,168 with 64 adapters of rank 64 120 us, by 32 128),
    // else 32, which fit beside the sums (8,191 rows 704, by 64 781)
    constexpr int kRank = NS == 4 ? 2 : 1;
#pragma unroll
    for (int m = 0; m < MF; m += 4) {
        const int n = n0 + wn * NF * 16;
        __builtin_amdgcn_sched_barrier(0);
        expand<DT, 4, NF, MF == 4 ? 2 : 1, kRank>(s, p.v, p.b, p.scale, row + m, n,
                                                  acc + m);
#pragma unroll
        for (int q = m; q < m + 4; ++q)
            if (m0 + (wm * MF + q) * 16 + (lane & 15) < s.T)
                store_cols<DT, NF>(s, p.out, row[q].t, n, acc[q]);
    }
}

// `whole` tiles of 256 x 256, then, where the tiles left over would keep less
// than half the CUs busy for a tile's time, each of them as two of 128 rows.
template <int DT>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
project_large_kernel(AShape s, int tm, int tn, int whole, ProjectArgs p)
{
    __shared__ __align__(1024) uint8_t lds[2 * 512 * kRowBytes];
    const int b = blockIdx.x;
    int im, in;
    if (b < whole) {
        tile_of(xcd_run(b, whole), tm, tn, &im, &in);
        project_tile<DT, 256, 256, 2, 4>(s, p, (long)im * 256, in * 256, lds, 0, s.H / 64);
        return;
    }
    const int h = xcd_run(b - whole, gridDim.x - whole);
    tile_of(whole + (h >> 1), tm, tn, &im, &in);
    const long m0 = (long)im * 256 + 128 * (h & 1);
    if (m0 < s.T)
        project_tile<DT, 128, 256, 2, 4>(s, p, m0, in * 256, lds, 0, s.H / 64);
}

// Tiles of 128 x 128: with NS = 2 stages two workgroups a CU, with 4 one,
// three steps ahead of memory; kParts: `splits` parts of H, joined by the add
// launch.  Which of them: at small_tiles below.
template <int DT, int NS, bool kParts>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
project_small_kernel(AShape s, int tm, int tn, int splits, ProjectArgs p)
{
    __shared__ __align__(1024) uint8_t lds[NS * 256 * kRowBytes];
    const int q = xcd_run(blockIdx.x, tm * tn * splits);
    const int part = q / (tm * tn), pairs = s.H / 128; // steps go in pairs
    const int a = (long)pairs * part / splits, b = (long)pairs * (part + 1) / splits;
    int im, in;
    tile_of(q - part * tm * tn, tm, tn, &im, &in);
    project_tile<DT, 128, 128, 2, 2, NS, kParts>(s, p, (long)im * 128, in * 128, lds, 2 * a,
                                                 2 * (b - a), part);
}

// ---------------------------------------------------------------------------
// Add: out = base + the adapters' term, base a given projection, or (kParts)
// the sum of `parts` float32 planes.  Bound by reading the base or the planes
// and B, and writing out: 4,097 x 5,120 fp16 values 26 us (84 MB, 3.2 TB/s; the
// parts of v and of an fp16 B take the rest).  A
// wavefront takes 16 places and `blocks` blocks of 16 NF columns: their v is
// read once for all of them, up to a rank of 32 KK.
// ---------------------------------------------------------------------------
constexpr int kAddWaves = 4;

template <int DT, int NF, int GB, int KK, bool kParts>
__global__ void __launch_bounds__(64 * kAddWaves)
add_kernel(AShape s, int blocks, int parts, const void *base, const int32_t *__restrict__ ids,
           const Row *__restrict__ order, const uint16_t *__restrict__ b,
           const float *__restrict__ scale, const float *__restrict__ v, uint16_t *out)
{
    const int lane = threadIdx.x & 63, wave = wave_of();
    int n0 = (blockIdx.y * kAddWaves + wave) * 16 * NF * blocks;
    const long i = (long)blockIdx.x * 16 + (lane & 15);
    const Row row = row_at(s, order, ids, i);
    const uint32_t rows = (uint32_t)__ballot(row.id >= 0) & 0xffffu;
    // a given base's pieces of the block at n0, loaded one block ahead
    uint4 ahead[NF / 2];
    const auto load_base = [&](int at) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + (size_t)row.t * s.N;
#pragma unroll
        for (int h = 0; h < NF / 2; ++h)
            ahead[h] = piece(p + min(at + 32 * h + 8 * (lane >> 4), s.N - 8));
    };
    if constexpr (!kParts)
        load_base(n0);
    const float sc = scale_of(scale, row);
    const Low<KK> low = low_of<KK>(s, v, row, 0);
    for (int k = 0; k < blocks && n0 < s.N; ++k, n0 += 16 * NF) {
        v4f acc[NF];
        if constexpr (kParts) {
            const float *p = static_cast<const float *>(base) + (size_t)row.t * s.N;
            const size_t plane = (size_t)s.T * s.N;
            v4f q[4][NF];
#pragma unroll
            for (int f = 0; f < NF; ++f)
                acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            for (int h = 0; h < parts; h += 4) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        q[u][f] = *reinterpret_cast<const v4f *>(
                            p + min(h + u, parts - 1) * plane +
                            min(n0 + column_of(f, 4 * (lane >> 4)), s.N - 4));
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        acc[f] += h + u < parts ? q[u][f] : v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
        } else {
#pragma unroll
            for (int h = 0; h < NF / 2; ++h) {
                float f[8];
                Elem<DT>::unpack(ahead[h], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[2 * h][e] = f[e];
                    acc[2 * h + 1][e] = f[4 + e];
                }
            }
            // (past the wavefront's columns a repeat, dropped)
            load_base(min(n0 + 16 * NF, s.N - 8));
        }
        if (rows) {
            bool left_out =
                expand_part<DT, 1, NF, GB, KK>(s, b, &row, &rows, &sc, &low, n0, &acc);
            for (int c = 32 * KK; c < s.r; c += 32 * KK) {
                const Low<KK> more = low_of<KK>(s, v, row, c);
                left_out |= expand_part<DT, 1, NF, GB, KK>(s, b, &row, &rows, &sc, &more, n0, &acc);
            }
            if (__any(left_out))
                for (int c = 0; c < s.r; c += 32 * KK) {
                    const Low<KK> more = low_of<KK>(s, v, row, c);
                    expand_part<DT, 1, NF, 1, KK, true>(s, b, &row, &rows, &sc, &more, n0, &acc);
                }
        }
        if (i < s.T)
            store_cols<DT, NF>(s, out, row.t, n0, acc);
    }
}

// The numbers of parts below go by the 256 CUs of an MI355X and not by the device,
// since the workspace's size goes by them and is asked for without one.

// Workgroups of few_kernel for the parts of x W^T, one a CU: an eighth of the
// CUs stays free for the shrink, which else starts when the first part ends
// (one row at 4,096 x 4,096 with an adapter of rank 64: 18 us, with 256 35;
// 65 rows, rank 16: 20 and 25).
constexpr int kFewGroups = 224;

// Columns of a workgroup of few_kernel.  Past 64 rows, 128 read x half as
// often; 64 make more workgroups, so fewer and larger parts of H, whose planes
// are written and read.  By 64 and by 128, us (32 adapters of rank 32):
//   rows               72           100          128
//   H 1,024  N 5,120                             18.4  22.7
//   H 2,048  N 5,120   19.1  20.0   20.8  23.1   21.8  23.9
//   H 4,096  N 1,024   16.8  18.6   17.0  19.2   17.8  20.3
//            N 2,304   21.9  20.2   24.4  21.0   25.4  22.5
//            N 4,608   22.6  23.6   27.9  23.8   26.1  27.2
//   H 7,168  N 2,048   21.4  24.2                23.4  27.1
//            N 2,304   27.2  25.1   30.0  25.8   30.1  27.3
//            N 7,168   37.7  35.1   38.6  38.4   41.1  38.8
int few_columns(const moe_adapter_shape &s)
{
    return s.T > 64 && s.H >= 4096 && s.N > 2048 ? 128 : 64;
}

// Parts of H of few_kernel: at most 6 (8 gain less than 1% in a short H and
// lose as much in small N), of at least two steps.
int few_splits(const moe_adapter_shape &s)
{
    const int tn = (s.N + few_columns(s) - 1) / few_columns(s);
    return std::max(1, std::min({kFewGroups / tn, 6, s.H / 128}));
}

// Tiles of 128 x 128 in one of three forms (us, whole calls, mixed or packed rows,
// rank 32): parts of H, up to two workgroups a CU; whole, two workgroups a CU; or
// whole, one deep workgroup a CU.
//   rows, H, N (tiles)          parts  whole  deep
//     300  1,024    520  (15)    20.4   23.0  27.7
//   1,024  1,024  1,024  (64)    30.8   26.3  29.4
//   1,024  2,048  1,024  (64)    35.3   36.4  40.3
//     640  2,048  4,096 (160)    38.8   35.4  39.4
//     640  4,096  4,096 (160)    48.4   55.5  61.1
//     300  4,096  9,216 (216)    59.1   66.2  61.0
//     640  4,480  4,096 (175)    53.7   55.7  61.1
//   2,048  4,096  2,048 (256)    66.5   60.1  66.7
//   2,048  7,168  2,048 (256)    89.9   94.7   100
//     256  4,096 12,800 (200)    74.2   77.2  64.5
//     256  7,168 12,800 (200)     107    128   100
//     512  5,120  6,144 (192)    60.4   68.0  71.2
//     512  5,120  7,168 (224)    79.3   82.3  72.0
//     512  7,168  7,168 (224)     101    119  96.7
//   1,024  7,168  3,584 (224)    83.6   87.5  94.5
// What parts save grows with H, what their planes cost with the tiles: from 18 of
// H a tile they win.  A weight that few tiles of rows share streams best through
// deep rings, once its tiles fill two thirds of the CUs (two tiles of rows) or
// three quarters (four, in a long H).
long small_tiles(const moe_adapter_shape &s)
{
    return (long)((s.T + 127) / 128) * ((s.N + 127) / 128);
}

bool small_deep(const moe_adapter_shape &s)
{
    const long n = small_tiles(s);
    return n <= 256 && ((s.T <= 256 && s.H > 2048 && n > 170) ||
                        (s.T <= 512 && s.H > 4096 && n > 192));
}

int small_splits(const moe_adapter_shape &s)
{
    const long n = small_tiles(s);
    if (n > 256 || s.H < 18 * n || small_deep(s))
        return 1;
    return (int)std::max(1l, std::min({512 / n, 8l, (long)s.H / 256}));
}

size_t parts_bytes(const moe_adapter_shape &s)
{
    const int splits = s.T <= kFewRows ? few_splits(s) : small_splits(s);
    return s.T > kFewRows && splits == 1 ? 0 : (size_t)splits * s.T * s.N * sizeof(float);
}

// The order's arrays in the workspace, from its start; null for one block of rows.
struct OrderLayout {
    OrderOut out;
    size_t bytes;
};

OrderLayout order_layout(const moe_adapter_shape &s, uint8_t *ws)
{
    OrderLayout l{};
    if (s.T <= 16)
        return l;
    const auto take = [&](size_t n) {
        uint8_t *p = ws + l.bytes;
        l.bytes += (n + 255) / 256 * 256;
        return p;
    };
    l.out.order = reinterpret_cast<Row *>(take(sizeof(Row) * s.T));
    l.out.blocks = reinterpret_cast<int32_t *>(take(sizeof(int32_t)));
    l.out.block = reinterpret_cast<Block *>(
        take(sizeof(Block) * ((s.T + 15u) / 16u + (size_t)std::min(s.T, s.L))));
    if (s.L >= kOrderKeys)
        l.out.count = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * ((size_t)s.L + 1)));
    return l;
}

// x A^T of every row, 256-byte aligned ends.
size_t v_bytes(const moe_adapter_shape &s)
{
    return order_layout(s, nullptr).bytes + ((size_t)s.T * s.rank * sizeof(float) + 255) / 256 * 256;
}

int up(long n, int by) { return (int)((n + by - 1) / by); }

// The order, and x A^T of its blocks.
template <int DT>
hipError_t shrink_many(const AShape &s, const uint16_t *x, const int32_t *ids, const OrderOut &o,
                       const uint16_t *a, float *v, hipStream_t st)
{
    // as much of the rank per workgroup as there is (x is read once per
    // block of the rank), but a workgroup for every CU; x comes from memory
    // and gets the deeper ring (8,191 x 7,168 x 7,168 with rank 64, the whole call:
    // by 64 704 us, by 32 710, by 16 733; 4,111 rows of rank 128 431, 437, 462;
    // 257 x 5,120 x 4,608 and 1,024 x 5,120 x 2,048, too few rows for every CU: by
    // 64 53 and 57, by 16 45 and 53)
    const int cus = device_cu_count(), t = up(s.T, 32);
    // blocks there may be (a workgroup takes several past 2^20)
    const auto blocks = [&](int rows) {
        return (int)std::min(up(s.T, rows) + (long)std::min(s.T, s.L), 1l << 20);
    };
    const bool wide = s.r > 16 && t * up(s.r, 32) >= cus;
    order_kernel<<<1, kOrderThreads, o.count ? 0 : (s.L + 1) * sizeof(int), st>>>(
        s, wide ? 32 : 16, ids, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (wide && s.r > 32 && t * up(s.r, 64) >= cus)
        shrink_many_kernel<DT, 32, 64, 2, 8, 6>
            <<<dim3(blocks(32), up(s.r, 64)), 512, 0, st>>>(s, x, o, a, v);
    else if (wide)
        shrink_many_kernel<DT, 32, 32, 2, 10, 8>
            <<<dim3(blocks(32), up(s.r, 32)), 512, 0, st>>>(s, x, o, a, v);
    else
        shrink_many_kernel<DT, 16, 16, 1, 10, 10>
            <<<dim3(blocks(16), up(s.r, 16)), 256, 0, st>>>(s, x, o, a, v);
    return hipGetLastError();
}

template <int DT>
hipError_t adapter_of_type(const moe_adapter_shape &sh, const void *x_, const void *w_,
                           const void *base, const int32_t *ids, const void *a_, const void *b_,
                           const float *scale, void *out_, uint8_t *ws, hipStream_t st)
{
    const AShape s{sh.T, sh.H, sh.N, sh.L, sh.rank};
    const auto *x = static_cast<const uint16_t *>(x_), *w = static_cast<const uint16_t *>(w_);
    const auto *a = static_cast<const uint16_t *>(a_), *b = static_cast<const uint16_t *>(b_);
    auto *out = static_cast<uint16_t *>(out_);
    const OrderLayout ol = order_layout(sh, ws);
    const bool few_rows = w && s.T <= kFewRows;
    const bool ordered = w || order_pays(s);
    const Row *order = ordered ? ol.out.order : nullptr;
    float *v = reinterpret_cast<float *>(ws + ol.bytes);
    const auto add = [&](auto nf, auto gb, auto given, int blocks, const void *from, int parts) {
        constexpr int NF = decltype(nf)::value, GB = decltype(gb)::value;
        constexpr bool kParts = !decltype(given)::value;
        const dim3 grid(up(s.T, 16), up(s.N, 16 * NF * kAddWaves * blocks));
        if (s.r <= 32)
            add_kernel<DT, NF, GB, 1, kParts><<<grid, 64 * kAddWaves, 0, st>>>(
                s, blocks, parts, from, ids, order, b, scale, v, out);
        else
            add_kernel<DT, NF, GB, 2, kParts><<<grid, 64 * kAddWaves, 0, st>>>(
                s, blocks, parts, from, ids, order, b, scale, v, out);
        return hipGetLastError();
    };
    const std::integral_constant<int, 1> c1;
    const std::integral_constant<int, 2> c2;
    const std::integral_constant<int, 4> c4;
    hipError_t e;
    if (few_rows) {
        float *parts = reinterpret_cast<float *>(ws + v_bytes(sh));
        const int tn = up(s.N, few_columns(sh)), splits = few_splits(sh);
        const auto few = [&](auto stream, auto shrink) {
            using S = decltype(stream);
            using F = decltype(shrink);
            // the order's and the shrink's workgroups come last and find the
            // CUs that the parts leave, the latter at most four tasks each
            const int tasks = s.T * up(s.r, F::kBN), other = tn * splits + (order != nullptr);
            const int shrinks =
                std::min(tasks, std::max(device_cu_count() - other, up(tasks, 4)));
            few_kernel<DT, S, F><<<other + shrinks, S::kThreads, 0, st>>>(
                s, tn, splits, x, w, ids, a, v, parts, ol.out.order);
        };
        if (s.T <= 16)
            few(Stream<16, 64, 1, 2, 8, 15, 128>{}, FewStream{});
        else if (s.T <= 32)
            few(Stream<32, 64, 2, 1, 6, 15, 128>{}, FewStream{});
        else if (s.T <= 64)
            few(Stream<64, 64, 2, 1, 6, 12, 128>{}, FewStream{});
        else if (few_columns(sh) == 64)
            few(Stream<128, 64, 2, 1, 4, 9, 128>{}, FewStream{});
        else
            few(Stream<128, 128, 2, 2, 4, 5, 128>{}, FewStream8{});
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        // few rows: many short wavefronts, four adapters' B in flight (128 fp16 rows
        // of 7,168 x 7,168 with 64 adapters of rank 64 72 us, eight 79)
        return add(c2, c4, std::false_type{}, 1, parts, splits);
    }
    if (!ordered) {
        shrink_few_kernel<DT>
            <<<std::min(s.T * up(s.r, FewStream::kBN), 2 * device_cu_count()),
               FewStream::kThreads, 0, st>>>(s, x, ids, a, v);
        e = hipGetLastError();
    } else {
        e = shrink_many<DT>(s, x, ids, ol.out, a, v, st);
    }
    if (e != hipSuccess)
        return e;
    if (!w)
        // two blocks of columns a wavefront read v once, where that leaves
        // enough of them: 100 rows 18.5 us with two, 15.1 with one; 4,097 rows
        // 40.3 and 43.0
        return add(c4, c1, std::true_type{}, s.T > kFewRows ? 2 : 1, base, 0);
    float *parts = reinterpret_cast<float *>(ws + v_bytes(sh));
    const ProjectArgs p{x, w, order, b, scale, v, out, parts};
    const int cus = device_cu_count();
    // 256 x 256 tiles from one a CU on: each value moved from the L2 enters twice
    // the products of 128 x 128 (4,096 x 4,096 x 4,096 141 against 167 us, 8,191 x
    // 7,168 x 7,168 704 against 886); without the halves 768 there, and 278 where
    // with them 251 at 4,352 x 5,120 x 5,120
    const int tm = up(s.T, 256), tn = up(s.N, 256), left = tm * tn % cus;
    const int sm = up(s.T, 128), sn = up(s.N, 128), splits = small_splits(sh);
    if (splits > 1) {
        project_small_kernel<DT, 2, true>
            <<<sm * sn * splits, 256, 0, st>>>(s, sm, sn, splits, p);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        return add(c4, c1, std::false_type{}, 1, parts, splits);
    }
    if (tm * tn >= cus) {
        const int halves = 2 * left <= cus ? left : 0;
        project_large_kernel<DT>
            <<<tm * tn + halves, 512, 0, st>>>(s, tm, tn, tm * tn - halves, p);
    } else if (small_deep(sh)) {
        project_small_kernel<DT, 4, false><<<sm * sn, 256, 0, st>>>(s, sm, sn, 1, p);
    } else {
        project_small_kernel<DT, 2, false><<<sm * sn, 256, 0, st>>>(s, sm, sn, 1, p);
    }
    return hipGetLastError();
}

} // namespace

size_t adapter_workspace_bytes(const moe_adapter_shape &s)
{
    return v_bytes(s) + parts_bytes(s);
}

hipError_t launch_adapter_project(const moe_adapter_shape &s, int dtype, const void *x,
                                  const void *w, const void *base, const int32_t *ids,
                                  const void *a, const void *b, const float *scale, void *out,
                                  void *ws, hipStream_t st)
{
    uint8_t *p = static_cast<uint8_t *>(ws);
    if (dtype == MOE_DT_BF16)
        return adapter_of_type<MOE_DT_BF16>(s, x, w, base, ids, a, b, scale, out, p, st);
    return adapter_of_type<MOE_DT_F16>(s, x, w, base, ids, a, b, scale, out, p, st);
}

} // namespace moe
