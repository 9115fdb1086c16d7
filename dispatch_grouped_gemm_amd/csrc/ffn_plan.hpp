// How the dense feed-forward block's products are cut: which tiles, in how many
// parts of K, and the workspace that takes.  Host code alone, of sizes alone.
#pragma once

#include <math.h>
#include <stddef.h>

#include <algorithm>

namespace moe {

constexpr int kMostParts = 8;

inline long tiles_up(long n, long by) { return (n + by - 1) / by; }

constexpr int kTileCus = 256; // workgroups that fill an MI355X; the workspace goes by it

// How a product of M x N over K is cut.
enum TileKind { kHuge, kWide, kEven, kFlat, kSmall, kFew, kTall, kSlim, kTileKinds };

struct Cut {
    TileKind kind;
    int splits;
    float us; // what that is expected to take
};

// Tiles of a kind down and across: shifts, or a division by a constant.
constexpr int kTileRows[] = {8, 7, 7, 6, 6, 5, 0, 0}; // log2; the last two have 192
constexpr int kTileCols[] = {8, 8, 7, 7, 6, 6, 8, 7}; // log2

inline long tiles_down(TileKind k, long M)
{
    if (k == kTall || k == kSlim)
        return (M + 191) / 192;
    return (M + (1l << kTileRows[k]) - 1) >> kTileRows[k];
}
inline long tiles_across(TileKind k, long N)
{
    return (N + (1l << kTileCols[k]) - 1) >> kTileCols[k];
}

// How many smaller tiles the 256 x 256 ones of the last round become each, 0
// where there is no round before it or it keeps more than half the CUs busy.
inline int huge_rest(long tiles)
{
    const long left = tiles % kTileCus;
    return tiles < kTileCus || left == 0 || 2 * left > kTileCus ? 0
           : 4 * left > kTileCus                               ? 2
                                                               : 4;
}

// Microseconds of a product.  A CU takes its tiles one after the other: a round
// costs its steps of 64 k and what stands before and behind them.  The steps of
// the largest tiles are bound by the matrix instructions, at clocks that fall as
// more of the CUs are busy; those of the others by what a CU draws from the L2,
// about 30 bytes a clock.  The second operand comes from memory at 4.5 TB/s at
// best.  Parts cost their planes and a launch.  Measured (us, in a row of calls, by
// the kinds in their order; the sums over 51 products of 200 to 8,192 rows of three
// blocks are within 0.1% of those of the fastest tiles):
//   8,192 x 4,096 pairs over 7,168    344  391  524  666            371  444
//   4,096 x 4,608 pairs over 5,120    151  183  193  234            167  195
//   8,192 x 7,168 over 2,048          196  224  286  353            204  240
//   4,096 x 5,120 over 2,304           79   92   96  126             83  100
//   4,096 x 2,304 over 5,120 (down)    99  118  108  131             84  106
//         the same with dh's epilogue  145  143  155  185            123  130
//   2,048 x 5,120 over 2,304           48   57   54   65             43   49
//   1,021 x 4,608 pairs over 5,120     92   53   71   77             75   49
//   1,021 x 2,816 pairs over 2,304     47   27   19   25             37   23
//   1,021 x 2,304 over 1,408           31   18   12   17   20   25   24   16
//     128 x 7,168 over 2,048                    23    18   13   17
//      90 x 1,344 over 544                      11     9  6.5  5.8
inline float product_cost(TileKind kind, int splits, long M, long N, long K)
{
    constexpr float step[] = {0.85f, 0.52f, 0.45f, 0.36f, 0.26f, 0.21f, 0.67f, 0.5f};
    constexpr float more[] = {0.60f, 0.31f, 0.09f, 0.0f, 0.0f, 0.0f, 0.45f, 0.2f}; // all busy
    constexpr float once[] = {7.0f, 5.0f, 3.0f, 2.8f, 2.6f, 2.6f, 6.0f, 4.0f};
    long groups = tiles_down(kind, M) * tiles_across(kind, N) * splits;
    const int all = (int)((K + 63) >> 6), steps = splits == 1 ? all : (all + splits - 1) / splits;
    float us = 0.0f;
    if (kind == kHuge && huge_rest(groups)) {
        const TileKind k = huge_rest(groups) == 2 ? kWide : kEven;
        us = steps * (step[k] + 0.8f * more[k]) + once[k];
        groups -= groups % kTileCus;
    }
    // rounds times the share of CUs that are busy in them is groups / kTileCus
    const float rounds = (float)((groups + kTileCus - 1) / kTileCus);
    us += rounds * (steps * step[kind] + once[kind]) +
          groups * (1.0f / kTileCus) * steps * more[kind];
    us = std::max(us, (2e-6f / 4.5f) * N * K + 2.0f);
    if (splits > 1)
        us += 4.0f + (8e-6f / 5.0f) * splits * M * N;
    return us;
}

// The numbers of parts that tiles of a kind may go in.  Pairs need a tile's columns of
// both halves in a wavefront, which the two smallest tiles lack, unless a join forms them.
constexpr long kMostPlanes = 1l << 25; // float32 sums in all parts

inline int fewest_parts(int kind, bool pairs)
{
    return pairs && (kind == kSmall || kind == kFew) ? 2 : 1;
}
inline int most_parts(int kind, long K)
{
    return kind < kEven || kind >= kTall
               ? 1
               : std::max(1, std::min(kMostParts, (int)((K + 63) >> 6) / 4));
}

// The cheapest cut.
inline Cut product_cut(long M, long N, long K, bool pairs)
{
    Cut best{kHuge, 1, product_cost(kHuge, 1, M, N, K)};
    for (int k = kWide; k < kTileKinds; ++k)
        for (int s = fewest_parts(k, pairs); s <= most_parts(k, K); ++s) {
            if (s > 1 && s * M * N > kMostPlanes)
                break;
            const float c = product_cost((TileKind)k, s, M, N, K);
            if (c < best.us)
                best = Cut{(TileKind)k, s, c};
        }
    return best;
}

// No fewer than the parts that product_cut chooses for any of the M to M + 31 rows that
// have the same tiles (M - 1 a multiple of 32): what a cut costs then rises with the
// rows by its planes, so that more parts beat fewer for some of them only where they do for
// M itself, but for the rounding of the costs.
inline int parts_from(long M, long N, long K, bool pairs)
{
    int most = 1;
    float best = 0.0f;
    for (int s = 1; s <= kMostParts; ++s) {
        float us = INFINITY;
        for (int k = kHuge; k < kTileKinds; ++k)
            if (s >= fewest_parts(k, pairs) && s <= most_parts(k, K))
                us = std::min(us, product_cost((TileKind)k, s, M, N, K));
        if (s == 1 || us <= best * 1.0001f)
            most = s;
        best = s == 1 ? us : std::min(best, us);
    }
    return most;
}

// A product's sizes beside its rows.
struct ProductSides {
    long N, K;
    bool pairs;
};

// The most bytes that a call of 1 to T rows needs: parts come and go with the rows, so
// the call of most rows is not the one that needs most.  need(M): those of M rows.
template <int P, typename F>
size_t most_bytes(long T, const ProductSides (&sides)[P], F need)
{
    size_t most = need(T);
    long end = 0; // (two parts of more rows would be past kMostPlanes)
    for (const ProductSides &p : sides)
        end = std::max(end, kMostPlanes / 2 / p.N);
    end = std::min(end, T);
    for (long lo = 1; lo <= end; lo += 32) {
        const long hi = std::min(lo + 31, end);
        // with as many parts for all of them the last rows need most; up to 64 rows the
        // kernels of few rows may take a product's place
        bool alike = lo > 64;
        for (const ProductSides &p : sides)
            alike = alike && parts_from(lo, p.N, p.K, p.pairs) ==
                                 product_cut(hi, p.N, p.K, p.pairs).splits;
        for (long M = alike ? hi : lo; M <= hi; ++M)
            most = std::max(most, need(M));
    }
    return most;
}

inline size_t product_parts_bytes(const Cut &c, long M, long N)
{
    return c.splits > 1 ? (size_t)c.splits * M * N * sizeof(float) : 0;
}

// Whether few rows by 32 of N weight rows a workgroup beat the tiles: each draws
// its rows of x and of the weight at some 72 KB a us, so they need to be many and
// the rows few (14 x 1,216 gate and up rows over 6,304, 38 workgroups: 11 us, by
// tiles with K in parts 8; 4,608 rows over 5,120 12 and 15).
inline int few_blocks(long T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

inline bool few_rows_pay(long T, long N, long K, const Cut &c)
{
    const float memory = (2e-6f / 4.5f) * N * K;
    const float drawn = (2e-3f / 72.0f) * (16 * few_blocks(T) + 32) * K;
    const long rounds = (N / 32 + kTileCus - 1) / kTileCus;
    return T <= 64 && std::max(rounds * drawn, memory) + 2.5f <= c.us;
}

// When the last of up to three jobs of n[j] workgroups that take d[j] each, in
// their order, is through on 32 CUs: an XCD's, which gets every eighth one.
inline float finish(const int *n, const float *d, int jobs)
{
    struct {
        float t; // CUs that are free from then on
        int cus;
    } level[4] = {{0.0f, 32}};
    int levels = 1;
    float end = 0.0f;
    for (int j = 0; j < jobs; ++j)
        for (int left = n[j]; left > 0;) {
            int i = 0;
            for (int k = 1; k < levels; ++k)
                if (level[k].t < level[i].t)
                    i = k;
            const float t = level[i].t + d[j];
            end = std::max(end, t);
            if (left >= level[i].cus) {
                left -= level[i].cus;
                level[i].t = t;
            } else { // the job's last: once a job
                level[i].cus -= left;
                level[levels++] = {t, left};
                left = 0;
            }
        }
    return end;
}

// C [M, N] over K, one of the three gradients' products.
struct Sides {
    long M, N, K;
};

// The tiles of each gradient, the first `along` of them dx: those whose schedule
// ends first, the smallest of such, by what a tile takes with all CUs busy (steps of
// 64 k, and once).  dx may go in any of the five kinds, the weights' gradients in 256 x
// 256, 128 x 256 and 128 x 128.  Measured, all 45 choices at 17 sizes (us; one kind for
// all jobs but a last 128 x 256 beside 256 x 256, and as chosen; in the mean 1.2% behind
// the fastest, one kind 11%):
//      64 rows, 5,120 by 2,304    41   32 (dx 64 x 128, 256 x 256, 128 x 256)
//     700 rows, 5,120 by 2,304    94   81 (128 x 256, 256 x 256, 128 x 256)
//   1,500 rows, 2,304 by 1,408    57   50 (192 x 256, then 128 x 256)
//   2,048 rows, 5,120 by 2,304   196  189 (192 x 256, then 256 x 256)
//   8,192 rows, 1,024 by   512    74   59 (256 x 256, then 128 x 128)
//   8,192 rows, 7,168 by 2,048   923  923 (256 x 256, the last 128 x 256)
inline void choose_tiles(const Sides *p, int jobs, int along, TileKind *kind)
{
    constexpr TileKind kinds[] = {kHuge, kTall, kWide, kEven, kFlat};
    constexpr float step[] = {1.22f, 0.99f, 0.74f, 0.43f, 0.32f};
    constexpr float once[2][5] = {{9.1f, 0.0f, 4.6f, 4.0f, 0.0f}, {7.9f, 2.8f, 4.0f, 3.7f, 0.8f}};
    const auto can = [&](int j, int q) {
        return j < jobs ? j < along || (kinds[q] != kTall && kinds[q] != kFlat) : q == 0;
    };
    int n[3][5] = {};
    float d[3][5] = {}, best = 0.0f;
    for (int j = 0; j < jobs; ++j)
        for (int q = 0; q < 5; ++q) {
            const long tiles = tiles_down(kinds[q], p[j].M) * tiles_across(kinds[q], p[j].N);
            n[j][q] = (int)((tiles + 7) / 8);
            d[j][q] = ((p[j].K + 63) >> 6) * step[q] + once[j < along][q];
        }
    // long calls: what the schedule's end costs is small beside the largest tiles' rate
    const bool rounds = n[0][0] + n[1][0] + n[2][0] > 32 * 32;
    for (int a = 0; a < 5; ++a)
        for (int b = 0; b < 5; ++b)
            for (int c = 0; c < 5; ++c) {
                if (!can(0, a) || !can(1, b) || !can(2, c))
                    continue;
                const int q[3] = {a, b, c}, ns[3] = {n[0][a], n[1][b], n[2][c]};
                const float ds[3] = {d[0][a], d[1][b], d[2][c]};
                if (best > 0.0f && (rounds || ns[0] * ds[0] + ns[1] * ds[1] + ns[2] * ds[2] >= 32 * best))
                    continue;
                const float us = rounds ? 1.0f : finish(ns, ds, jobs);
                if (best == 0.0f || us <= best) {
                    best = us;
                    for (int j = 0; j < jobs; ++j)
                        kind[j] = kinds[q[j]];
                }
            }
    if (rounds && along < jobs)
        kind[jobs - 1] = kWide;
}

} // namespace moe
