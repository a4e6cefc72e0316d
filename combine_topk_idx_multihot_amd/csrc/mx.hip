// mx.hip -- quantization to MXFP4 (mx.h) and back, for weights and for rows.
//
// Both are bound by HBM: 2 or 4 bytes of a value and 17/32 of its code and scale.  A
// lane takes 16 bytes of values, 8 bf16 or 4 fp32, so that loads and stores of a wave
// are consecutive in memory; a block of 32 is four or eight lanes, its largest
// magnitude two or three DPP moves.  (With 8 fp32 per lane, in two loads 32 bytes
// apart, the way back wrote half lines: 126 instead of 85 us at 32768 x 4096.)
// 32768 x 4096 values, there and back: fp32 102 and 85 us (6.0 and 7.2 TB/s, codes from
// the Infinity Cache), bf16 53 and 48; 131072 x 4096 bf16 228 and 230 us (6.0 and 5.9 TB/s).
#include "moe_internal.h"
#include "mx.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMxThreads = 256;
constexpr int kMxPieces = 4; // runs of 64 lanes' values per wave

// Values of a lane.
template <bool F32>
constexpr int kMxValues = F32 ? 4 : 8;

template <bool F32>
__global__ void __launch_bounds__(kMxThreads) k_quantize_mx(MxArgs a)
{
    constexpr int N = kMxValues<F32>;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * (kMxThreads / kWave) + threadIdx.x / kWave;
    const int64_t c0 = wave * (kMxPieces * kWave) + lane; // runs of N values
    u32x4 v[kMxPieces];
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (c < a.runs)
            v[i] = __builtin_nontemporal_load(static_cast<const u32x4 *>(a.values) + c);
    }
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        const bool in = c < a.runs; // the same for the lanes of a block
        float x[8] = {};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = __uint_as_float(F32 ? v[i][j & 3] : j & 1 ? v[i][j >> 1] & 0xFFFF0000u : v[i][j >> 1] << 16);
            m = max(m, mag_bits(x[j]));
        }
        m = max_of_quad(m);
        if (F32) // of the two quads of a block: lane 7 - i of each 8 (row_half_mirror)
            m = max(m, static_cast<uint32_t>(
                           __builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x141, 0xF, 0xF, true)));
        const uint32_t b = mx_scale(m);
        const uint32_t q = mx_pack8(x, b);
        // the scales of the blocks of 16 lanes as one word (before the branch: it needs every lane)
        const uint32_t some = F32 ? __shfl(b, 0, 16) | __shfl(b, 8, 16) << 8 : gather_bytes(b);
        if (!in)
            continue;
        constexpr int kBlocks = 16 * N / kMxBlock; // of 16 lanes
        const bool all = (c | 15) < a.runs;
        if (F32)
            reinterpret_cast<uint16_t *>(a.codes)[c] = static_cast<uint16_t>(q);
        else
            reinterpret_cast<uint32_t *>(a.codes)[c] = q;
        if (all && (lane & 15) == 0) {
            if (F32)
                reinterpret_cast<uint16_t *>(a.scales)[c >> 4] = static_cast<uint16_t>(some);
            else
                reinterpret_cast<uint32_t *>(a.scales)[c >> 4] = some;
        } else if (!all && (lane & (16 / kBlocks - 1)) == 0) {
            a.scales[c * N / kMxBlock] = static_cast<uint8_t>(b);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMxThreads) k_dequantize_mx(MxArgs a)
{
    constexpr int N = kMxValues<F32>;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * (kMxThreads / kWave) + threadIdx.x / kWave;
    const int64_t c0 = wave * (kMxPieces * kWave) + lane;
    uint32_t q[kMxPieces], b[kMxPieces];
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        q[i] = b[i] = 0;
        if (c < a.runs) {
            q[i] = F32 ? reinterpret_cast<const uint16_t *>(a.codes)[c] : reinterpret_cast<const uint32_t *>(a.codes)[c];
            b[i] = a.scales[c * N / kMxBlock];
        }
    }
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        if (c >= a.runs)
            return;
        const float s = mx_scale_operand(b[i]);
        if (F32) {
            const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 0);
            const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 1);
            __builtin_nontemporal_store(f32x4{lo[0], lo[1], hi[0], hi[1]}, static_cast<f32x4 *>(a.out) + c);
        } else {
            u32x4 y;
            y[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 0));
            y[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 1));
            y[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 2));
            y[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 3));
            __builtin_nontemporal_store(y, static_cast<u32x4 *>(a.out) + c);
        }
    }
}

static hipError_t launch_mx(void (*k)(MxArgs), const MxArgs &a, hipStream_t s)
{
    constexpr int64_t kPerBlock = kMxThreads * kMxPieces;
    const int64_t nb = (a.runs + kPerBlock - 1) / kPerBlock;
    if (nb > 0xFFFFFFFFll / kMxThreads)
        return hipErrorInvalidConfiguration;
    launch(k, dim3(static_cast<unsigned>(nb)), dim3(kMxThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_quantize_mx(const MxArgs &a, bool f32, hipStream_t s)
{
    return launch_mx(f32 ? k_quantize_mx<true> : k_quantize_mx<false>, a, s);
}

hipError_t launch_dequantize_mx(const MxArgs &a, bool f32, hipStream_t s)
{
    return launch_mx(f32 ? k_dequantize_mx<true> : k_dequantize_mx<false>, a, s);
}

}  // namespace moe
