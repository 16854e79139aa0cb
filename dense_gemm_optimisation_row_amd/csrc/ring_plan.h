// What a product on the rings is estimated to take, by which its tile and the
// split of its sum are chosen.  Host code.  Internal header.
#pragma once

#include "linear.h"

namespace dgor {

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

inline long long tiles(const Product &p, int tm, int tn)
{
    return (long long)ceil_div(p.M, tm) * ceil_div(p.N, p.gated ? tn / 2 : tn) * p.nbatch;
}

// Time of a product on a ring's tile with its sum in `parts`.  Up to `share`
// workgroups of the tile run on a compute unit at once.  A round of at most one
// a unit takes ends + alone for each 32 k, a full one ends_full + full each.
// Parts are written in FP32 and joined by another launch.  Microseconds, fitted
// to 16 to 4096 workgroups of each tile and sums of 256 to 4096 (BF16, K x N).
// Over 184 products of every tile, layout and split they are 0.89 to 1.20 of the
// times measured for four in five, 0.60 to 1.70 for all (short gated sums take less
// than estimated, long ones of few columns more); which is chosen hangs on
// their order alone.  Full rates of the fit: 1470, 1280, 1180, 890 and 570
// TFLOP/s.  An activation of exponentials adds what its outputs take on the
// vector ALUs: 9 us for 256 x 256 (GELU, 4096 x 8192 outputs of 4096: 222 us,
// 204 without).
struct RingCost {
    RingTile tile;
    int share;
    double ends, alone, ends_full, full;
    double halves;   // times as long a stage whose loads take half lines
};
constexpr RingCost kRings[] = {
    {kRing256, 1, 14.5, 0.73, 14.5, 0.73, 1.0},
    {kRing256x128, 1, 9.8, 0.42, 9.8, 0.42, 1.3},
    {kRing128, 2, 6.8, 0.295, 7.5, 0.455, 1.17},
    {kRing128x64, 2, 4.8, 0.243, 6.2, 0.33, 1.12},
    {kRing64, 2, 4.0, 0.158, 4.2, 0.243, 1.08},
};
constexpr int kRingTiles = sizeof(kRings) / sizeof(kRings[0]);
constexpr double kJoinLaunch = 4.5, kJoinBytes = 8e6;   // and a microsecond's bytes
struct RingTimes {
    double alone, full, join;   // a round of one tile a unit, a full one, joining the parts
};
inline RingTimes times(const Product &p, const RingCost &c, int parts)
{
    // half lines: B as N x K, and each of two matrices' 32 columns
    const bool halves = p.trans_b || (p.gated && ring_tile_n(c.tile) == 64);
    const double stages = 2.0 * product_stages(p) / parts * (halves ? c.halves : 1.0);
    // an activation's time for a workgroup's outputs
    const double act = p.e.act > GEMM_ACT_RELU && parts == 1
                           ? 9.0 * ring_tile_m(c.tile) * ring_tile_n(c.tile) / (p.gated ? 131072 : 65536)
                           : 0.0;
    return {c.ends + stages * c.alone + act, c.ends_full + stages * c.full + act * c.share,
            parts > 1 ? kJoinLaunch + 8.0 * parts * (p.gated ? 2 : p.nbatch) * p.M * p.N / kJoinBytes : 0.0};
}
inline double microseconds(const Product &p, const RingCost &c, long long n, int parts)   // n tiles
{
    const unsigned long long groups = (unsigned long long)n * parts;
    const unsigned long long rounds = groups / (256u * c.share), rest = groups % (256u * c.share);
    const RingTimes t = times(p, c, parts);
    return rounds * t.full + (rest == 0 ? 0.0 : rest <= 256 ? t.alone : t.full) + t.join;
}

}  // namespace dgor
