// expert_choice.h -- which kernel an experts' product takes, from what the host
// knows before the launch.  Plain C++: the rule is tested without a GPU.
#pragma once

#include <stdint.h>

namespace moe {

// The groups of a product, one per local expert that has rows.
struct ExpertLoad {
    int64_t rows_max;  // most rows that all of them can hold
    int64_t group_max; // most rows that one can hold
    int64_t slots;     // most groups there can be, whatever they were padded to: a launch that
                       // takes one slot per group must have as many
    int64_t groups;    // the same, groups padded to multiples of P
    int64_t rows_mean; // rows of one of that many, pad rows (computed like any other) among them
};

// T tokens of k slots over E experts, EL of them local, groups padded to
// multiples of P; R rows, exact in eager mode; worst: the most rows that any
// routing makes.  A token has a row per expert at most.
inline ExpertLoad expert_load(int64_t T, int64_t k, int64_t E, int64_t EL, int64_t P, int64_t worst, int64_t R,
                              bool eager)
{
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    ExpertLoad l;
    l.rows_max = least(R, worst); // whatever capacity the caller chose
    l.group_max = least(up(T, P) * P, l.rows_max);
    l.slots = least(least(EL, T * least(k, EL)), l.rows_max);
    if (l.slots < 1)
        l.slots = 1;
    l.groups = eager ? least(l.slots, up(l.rows_max, P)) : l.slots;
    if (l.groups < 1)
        l.groups = 1;
    // sync-free: uniform routing
    l.rows_mean = eager ? up(l.rows_max, l.groups) : up(up(T * k, E), P) * P;
    return l;
}

enum class ExpertKernel { rows, ring, tile };

constexpr int kCus = 256;      // MI355X
constexpr int kTileCols = 256; // weight rows of a tile
constexpr int kRingRows = 32;  // rows of a tile of the ring kernel

// N output columns (gated: of each half).  Times are medians in us, E experts
// with r rows each (on average, under random routing, where T tokens are named).
inline ExpertKernel choose_expert_kernel(const ExpertLoad &l, int K, int N, bool gated)
{
    const int cols = gated ? kTileCols / 2 : kTileCols;
    const int64_t tiles = l.groups * ((static_cast<int64_t>(N) + cols - 1) / cols);
    // Products that are over before the others have listed their tiles: no
    // group can be more than two passes of 16 rows, and the work is small.
    // K = 2048, N = 4096 (rows / ring): E = 1: r = 1 5.4 / 13.7, r = 32 9.8 / 14.2,
    // r = 64 20.0 / 14.6; E = 4, r = 16: 9.8 / 14.9; E = 16: r = 1 25.9 / 26.2,
    // r = 16 33.9 / 26.6.  N = 512, E = 64: r = 8 14.6 / 15.6, r = 16 16.3 / 15.6.
    // (Gated, K = 2048, N = 768: E = 1, r = 1 21.0 / 14.6, E = 64 46 / 40: the
    // ring always.)
    // Groups padded to P, top-8 of 128, K = 768, N = 2048: T = 1: P = 16 6.3 / 9.0, P = 32
    // 14 / 9.5; T = 3: P = 4 10.0 / 10.2, P = 8 12.4 / 10.8; T = 5: P = 4 15.2 / 16.7 (the ring
    // by this rule); T = 8, P = 16 22.7 / 19.
    if (!gated && l.group_max <= 32 && tiles * l.rows_mean <= 4 * kCus)
        return ExpertKernel::rows;
    // Tiles of 32 rows while the weights' bytes bound the product, or while
    // taller ones would leave CUs without work.  K = 2048, N = 4096 (ring / tile):
    // E = 64: r = 64 127 / 131, r = 128 207 / 147; E = 1, r = 512 17.1 / 31.6;
    // E = 4: r = 256 28.2 / 32.2, r = 512 50.3 / 35.1.  N = 512: E = 16, r = 512 29.2 / 32.7; E = 64:
    // r = 128 29.4 / 32.6, r = 256 54.4 / 44.6.  (The tile kernel sends two steps
    // ahead: K >= 256.)
    // Random routing, where groups around r = 64 partly need a third ring tile:
    // E = 64, T = 512 (r = 64), K = 2048: N = 512 26.1 / 22.3, 2048 75.6 / 70.7, 4096
    // 143 / 128; T = 384 16.5 / 21.9, 67.9 / 67.3, 126 / 126; T = 1024 at N = 512
    // 36.9 / 26.6, the side that this rule does not take.
    // Gated, K = 2048, random routing on E = 64: N = 768: T = 384 51.8 / 62.7, 512 62.1 /
    // 64.0, 768 86.5 / 68.8; N = 2048: 384 123 / 127, 512 149 / 126, 768 191 / 147; N =
    // 256: 384 19.9 / 22.8, 1024 42.7 / 29.2, 2048 65.2 / 39.4.  N = 768, E = 1: r = 1024 16.0 /
    // 33.5; E = 4: r = 256 16.1 / 33.4, r = 512 27.4 / 34.4; E = 16: r = 64 16.3 / 23.4, r = 128
    // 27.8 / 28.0, r = 256 50.6 / 36.2 (E4M3 outputs; bf16 within 7 %, at N = 256 up to
    // 16 % less).
    // Groups padded to 128 of 128 experts, K = 768, N = 2048: T = 16 78.9 / 52.1, 64 106 /
    // 69.7, 256 108 / 68.0, 1024 110 / 70.1; K = 2048, N = 4096, T = 1024 423 / 277; gated K =
    // 2048, N = 768: T = 256 167 / 105.  Padded to 16, T = 256: 48.4 / 56.5, gated 74.1 / 93.2.
    const int64_t ring_tiles = tiles * ((l.rows_mean + kRingRows - 1) / kRingRows);
    if (K < 256 || l.rows_mean <= 64 || ring_tiles <= 2 * kCus)
        return ExpertKernel::ring;
    return ExpertKernel::tile;
}

}  // namespace moe
