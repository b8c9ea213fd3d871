// ecf8x_tiles.h -- which workgroup of a product takes which tile, and how long a
// part of its reduction.
//
// A product has so many tiles of BM tokens by BN columns.  As many as fill every
// compute unit some whole number of times are done whole; those that are left,
// which would leave most units without one, are cut along the reduction into
// shares, whose sums go to the workspace and are joined in order.  Few tiles are
// all of them left ones.  (4096 x 13824 x 5120, input gradient: 320 tiles of
// 256 x 256 on 256 compute units.  All of them in three shares 530 us, the 64 that
// are left in four 455.  The product, 864 tiles: all whole 513, 96 in two 478.
// Both by the step times of then; now 445 and 452.)
#ifndef ECF8X_TILES_H
#define ECF8X_TILES_H

#include "ecf8x_common.h"

namespace ecf8x {

struct Tiling {
    int bm, bn;                 // a tile
    int tiles_m, tiles_n;
    int whole, rest;            // tiles done whole, and in shares: the first and the last of their order
    int shares;                 // of each of the rest; 1: there are none
    int length;                 // of a share
};

// A workgroup's tile and share.
struct Part {
    int tm, tn, share;
    int at;                     // of [share][rest] where it leaves sums; -1: a whole tile
};

// The tiles' order: columns of eight tiles down the tokens, so that a die's cache sees the same rows of both operands again.
__host__ __device__ __forceinline__ void tile_at(const Tiling& T, int tile, int& tm, int& tn)
{
    const int band = tile / (8 * T.tiles_n), left = T.tiles_m - band * 8, rows = left < 8 ? left : 8, in_band = tile - band * 8 * T.tiles_n;
    tm = band * 8 + in_band % rows;
    tn = in_band / rows;
}

// Workgroups go to the eight dies in turn; each die gets a run of tiles.
__host__ __device__ __forceinline__ Part part_of(const Tiling& T, int group)
{
    Part p{0, 0, 0, -1};
    int count = T.whole, id = group;
    if (group >= T.whole) {
        count = T.rest;
        p.share = (group - T.whole) / count;
        id = group - T.whole - p.share * count;
    }
    if (count % 8 == 0) id = id % 8 * (count / 8) + id / 8;
    if (group >= T.whole) {
        p.at = p.share * T.rest + id;
        id += T.whole;
    }
    tile_at(T, id, p.tm, p.tn);
    return p;
}

inline uint32_t groups_of(const Tiling& T) { return (uint32_t)T.whole + (uint32_t)T.rest * T.shares; }

inline uint64_t sums_of(const Tiling& T) { return round_up(4ull * T.shares * T.rest * T.bm * T.bn, 256); }

// Microseconds of a step of a workgroup: of one alone on its compute unit and of two side by side (0: no LDS for a second).
struct Cost {
    int bm, bn;
    double one, two;
};

// The tiles, and the shares of those that are left, with the least time by the table: whole rounds of the compute units,
// the last one's part, and for shares the traffic of their sums and the launch that joins them.  step: length of a step;
// unit: what a share's length is a multiple of; least: its least length; small: the tile whose rows may be mostly padding.
inline Tiling tiling_of(const Cost* costs, int count, uint64_t tokens, uint64_t cols, uint64_t length, int step, int unit, int least, int small)
{
    Tiling best{};
    double shortest = -1.0;
    for (int i = 0; i < count; ++i) {
        const Cost& c = costs[i];
        if (c.bm > small && (uint64_t)c.bm / 2 >= tokens) continue;
        const uint64_t down = (tokens + c.bm - 1) / c.bm, across = (cols + c.bn - 1) / c.bn, tiles = down * across, slots = c.two > 0.0 ? 512 : 256;
        const double full = c.two > 0.0 ? c.two : c.one;
        const auto rounds = [&](uint64_t groups) {
            const uint64_t last = groups % slots;
            return groups / slots * full + (last == 0 ? 0.0 : last <= 256 ? c.one : full);
        };
        for (int s = 1; s <= 16 && (s == 1 || length / s >= (uint64_t)least); ++s)
            for (uint64_t whole = s == 1 ? tiles : 0;; whole = tiles / slots * slots) {
                const uint64_t rest = tiles - whole, steps = (length + step - 1) / step, share_steps = ((length + s - 1) / s + step - 1) / step;
                double us = rounds(whole) * steps + rounds(rest * s) * share_steps;
                if (rest) us += 4.0 + 8.0 * s * (rest == tiles ? (double)tokens * cols : (double)rest * c.bm * c.bn) / 5e6;
                if (shortest < 0.0 || us < shortest) {
                    shortest = us;
                    best = Tiling{c.bm, c.bn, (int)down, (int)across, (int)whole, (int)rest, s, (int)round_up((length + s - 1) / s, unit)};
                }
                if (s == 1 || whole == tiles / slots * slots || tiles % slots == 0) break;
            }
    }
    return best;
}

// Sums the shares of the tiles that were left, in order, adds the bias and rounds.
template <int TYPE>
__global__ __launch_bounds__(256) void join_tiles_kernel(const float* sums, Tiling T, int64_t tokens, int cols, const uint16_t* bias, uint16_t* out,
                                                         int64_t ld)
{
    const int lines = T.tiles_m > 1 ? T.bm : (int)tokens, quads = T.bn / 4, each = lines * quads;     // of a tile
    const uint32_t groups = (uint32_t)(each + 255) / 256, tile = blockIdx.x / groups;
    const int inside = (int)(blockIdx.x - tile * groups) * 256 + threadIdx.x, row = inside / quads, quad = inside - row * quads;
    if (inside >= each) return;
    int tm, tn;
    tile_at(T, T.whole + (int)tile, tm, tn);
    const int64_t t = (int64_t)tm * T.bm + row;
    const int c = tn * T.bn + 4 * quad;
    if (t >= tokens || c >= cols) return;
    const float* at = sums + (int64_t)tile * T.bm * T.bn + 4 * inside;
    const int64_t plane = (int64_t)T.rest * T.bm * T.bn;
    f32x4 s{0, 0, 0, 0};
    for (int p = 0; p < T.shares; p += 8) {                   // eight loads in flight, added in order
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(at + min(p + j, T.shares - 1) * plane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p + j < T.shares) s += v[j];
    }
    if (bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) s[j] += load1<TYPE>(bias + c + j);
    }
    store4<TYPE>(out + t * ld + c, s, cols - c);
}

template <int TYPE>
int join_tiles(const float* sums, const Tiling& T, int64_t tokens, int cols, const uint16_t* bias, uint16_t* out, int64_t ld, hipStream_t st)
{
    const uint32_t lines = T.tiles_m > 1 ? T.bm : (uint32_t)tokens;
    join_tiles_kernel<TYPE><<<T.rest * ((lines * T.bn / 4 + 255) / 256), 256, 0, st>>>(sums, T, tokens, cols, bias, out, ld);
    return launch_status();
}

}  // namespace ecf8x

#endif
