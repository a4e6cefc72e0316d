// mx.hip -- quantization to MXFP4 (mx.h) and back, for weights and for rows.
//
// Both are bound by HBM: 2 or 4 bytes of a value and 17/32 of its code and scale.
// A lane takes 8 consecutive values, so that loads and stores of a wave are
// consecutive in memory; a block of 32 is four lanes, its largest magnitude two
// DPP moves.
#include "moe_internal.h"
#include "mx.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMxThreads = 256;
constexpr int kMxPieces = 4; // pieces of 64 lanes x 8 values per wave

__device__ __forceinline__ void unpack_bf16(const u32x4 &v, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(v[j] << 16);
        x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMxThreads) k_quantize_mx(MxArgs a)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * (kMxThreads / kWave) + threadIdx.x / kWave;
    const int64_t c0 = wave * (kMxPieces * kWave) + lane;
    u32x4 v[kMxPieces][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        const u32x4 *p = static_cast<const u32x4 *>(a.values) + (F32 ? 2 * c : c);
        if (c < a.chunks) {
            v[i][0] = __builtin_nontemporal_load(p);
            if (F32)
                v[i][F32] = __builtin_nontemporal_load(p + 1);
        }
    }
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        const bool in = c < a.chunks; // the same for the four lanes of a block
        float x[8];
        if (F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = in ? __uint_as_float(v[i][(j >> 2) & F32][j & 3]) : 0.f;
        } else {
            unpack_bf16(v[i][0], x);
        }
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, mag_bits(x[j]));
        const uint32_t b = mx_scale(max_of_quad(in ? m : 0u));
        const uint32_t q = mx_pack8(x, b);
        const uint32_t four = gather_bytes(b); // (before the branch: it needs every lane)
        if (!in)
            continue;
        reinterpret_cast<uint32_t *>(a.codes)[c] = q;
        // four blocks' scales as one word where all of them are there
        const int64_t first = c & ~static_cast<int64_t>(15);
        if (first + 16 <= a.chunks) {
            if ((lane & 15) == 0)
                reinterpret_cast<uint32_t *>(a.scales)[c >> 4] = four;
        } else if ((lane & 3) == 0) {
            a.scales[c >> 2] = static_cast<uint8_t>(b);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMxThreads) k_dequantize_mx(MxArgs a)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * (kMxThreads / kWave) + threadIdx.x / kWave;
    const int64_t c0 = wave * (kMxPieces * kWave) + lane;
    uint32_t q[kMxPieces], b[kMxPieces];
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        if (c < a.chunks) {
            q[i] = reinterpret_cast<const uint32_t *>(a.codes)[c];
            b[i] = a.scales[c >> 2];
        }
    }
#pragma unroll
    for (int i = 0; i < kMxPieces; ++i) {
        const int64_t c = c0 + i * kWave;
        if (c >= a.chunks)
            return;
        const float s = mx_scale_operand(b[i]);
        if (F32) {
            f32x4 y[2];
#define MOE_MX_PAIR(j)                                                              \
    {                                                                               \
        const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, j);        \
        y[(j) >> 1][((j) & 1) * 2] = p[0];                                          \
        y[(j) >> 1][((j) & 1) * 2 + 1] = p[1];                                      \
    }
            MOE_MX_PAIR(0)
            MOE_MX_PAIR(1)
            MOE_MX_PAIR(2)
            MOE_MX_PAIR(3)
#undef MOE_MX_PAIR
            f32x4 *o = static_cast<f32x4 *>(a.out) + 2 * c;
            o[0] = y[0];
            o[1] = y[1];
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
    const int64_t nb = (a.chunks + kPerBlock - 1) / kPerBlock;
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
