// layer_choice.h -- which form a layer for a few tokens takes, and what that asks of its workspace and its
// grid, from what the host knows.  Plain C++: tested without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kLayerMaxSlots = 1024;  // T * k at most
constexpr int kLayerMaxWidth = 65536; // H and I at most
enum { kLayerBf16 = 0, kLayerFp8 = 1, kLayerMxfp4 = 2 }; // the weights' format

// Whether every slot is on its own: up to 16 of them, or 7 (E4M3 5, MXFP4 3) for 8 experts.
// Together / on its own, us: top-8 of 128, H = 2048, I = 768: bf16 T = 8 115 / 93, T = 12 142 / 134,
// T = 16 161 / 169; E4M3 T = 8 54.9 / 52.3, T = 10 60.8 / 62.6, T = 12 69.9 / 73.7; MXFP4 T = 4 27.3 /
// 22.4, T = 8 36.7 / 37.9, T = 10 39.9 / 45.1.  Top-2 of 32, H = 4096, I = 1024: bf16 T = 10 86.9 / 82.0, T =
// 14 111 / 108; E4M3 42.2 / 40.9, 53.1 / 54.1; MXFP4 T = 10 29.0 / 37.0.  Top-2 of 8, H = I = 2048,
// T = 8: 39.3 / 47.9, 29.1 / 25.9, 21.7 / 23.7.
inline bool layer_singles(int64_t slots, int64_t E, int fmt)
{
    return slots <= 16 || 8 * slots <= (fmt == kLayerBf16 ? 7 : fmt == kLayerFp8 ? 5 : 3) * E;
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
