// layer_choice.h -- which form a layer for a few tokens takes, and what that asks of its workspace and its
// grid, from what the host knows.  Plain C++: tested without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kLayerMaxSlots = 1024;  // T * k at most
constexpr int kLayerMaxWidth = 65536; // H and I at most
enum { kLayerBf16 = 0, kLayerFp8 = 1, kLayerMxfp4 = 2 }; // the weights' format

// Whether every slot is on its own: up to 16 of them, or 7 (E4M3 5, MXFP4 4) for 8 experts.
// Together / on its own, us: top-8 of 128, H = 2048, I = 768: bf16 T = 8 107 / 93, T = 12 143 / 134, T = 14 149 / 155, T =
// 16 161 / 174; E4M3 T = 8 57.9 / 53.3, T = 10 61.8 / 63.7, T = 12 71.5 / 74.2; MXFP4 T = 4 30.4 / 24.7, T = 7 39.7 / 37.0,
// T = 8 41.6 / 40.8, T = 10 44.9 / 48.6.  Top-2 of 32, H = 4096, I = 1024: T = 10 bf16 84.5 / 81.3, E4M3 51.6 /
// 45.4, MXFP4 35.0 / 42.6; T = 14 110 / 107, 66.2 / 59.4, 44.0 / 55.3.
// 16 slots: top-2 of 8, H = I = 2048 bf16 53.0 / 53.7, E4M3 30.4 / 30.0, MXFP4 26.2 / 24.7; top-4 of 4, H = 4096, I = 1024
// 40.8 / 46.3, 31.2 / 25.5, 24.3 / 21.7; top-2 of 32, H = 4096, I = 1024 72.6 / 66.8, 46.0 / 39.2, 32.1 / 36.0; of one
// expert, H = I = 2048 30.7 / 26.3, 27.0 / 22.6, 24.3 / 27.9.
inline bool layer_singles(int64_t slots, int64_t E, int fmt)
{
    return slots <= 16 || 8 * slots <= (fmt == kLayerBf16 ? 7 : fmt == kLayerFp8 ? 5 : 4) * E;
}

// The most items that `slots` slots of EL experts make: one per expert in use, and
// one more for every 16 slots beyond its first.
inline int64_t layer_items(int64_t slots, int64_t EL)
{
    const int64_t groups = slots < EL ? slots : EL;
    return groups + (slots - groups) / 16;
}

// Bytes of the workspace, whatever the weights' format: h (4 bytes a value), then the slots' fp32 outputs where
// any format lets slots share weights; more than none for no tokens.
inline size_t layer_ws_bytes(int64_t slots, int64_t E, int64_t H, int64_t I)
{
    const bool own = layer_singles(slots, E, kLayerBf16) && layer_singles(slots, E, kLayerFp8) &&
                     layer_singles(slots, E, kLayerMxfp4);
    return 16 + static_cast<size_t>(slots) * I * 4 + (own ? 0 : static_cast<size_t>(slots) * H * 4);
}

}  // namespace moe
