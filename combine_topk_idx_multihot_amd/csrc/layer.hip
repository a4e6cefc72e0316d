// layer.hip -- a whole MoE layer for a few tokens, in two kernels.
//
//   h[s]   = silu(W1g[e] x[t]) * (W1u[e] x[t])          for every slot s = (t, j), e its expert
//   out[t] = sum over t's local slots of w[s] * W2[e] h[s]
// No rows are laid out: k_layer_up writes h (bf16, one row per slot) to the
// workspace, k_layer_down multiplies it and sums a token's slots in its own LDS.
// The weights of the experts in use are what has to be read; tokens and h are
// small and come from the L2.  Weights are widened to bf16 in registers (E4M3 and
// E2M1 codes are exact there, an E8M0 scale too) and multiplied with bf16 tokens
// by the bf16 matrix instructions, in fp32: those have four times the rate that
// the weights' bytes need, and tokens that are not quantized cost nothing here.
// The fp32 scale of a block of E4M3 weights enters after the products of its
// columns.  h is rounded to bf16 as the experts of a bf16 layer would; everything
// else stays in fp32 until out.
//
// Both kernels come in two forms.  With few slots every slot is on its own (an
// expert that two tokens share is read twice, the second time from the L2): a
// workgroup needs to know one id only.  With more, slots of the same expert share
// its weights, up to 16 of them per instruction; the list of experts in use is
// made by one workgroup of k_layer_up for k_layer_down.
#include "moe_internal.h"
#include "mx.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kAhead = 8; // loads of weights that a lane has in flight

__device__ __forceinline__ uint32_t two_bf16(float x, float y)
{
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Columns that the 16 bytes of a lane hold; a step is the four chunks of the
// lanes of a row.
template <int FMT>
constexpr int kChunkCols = FMT == kLayerBf16 ? 8 : FMT == kLayerFp8 ? 16 : 32;

// Columns 8 j .. 8 j + 7 of a lane's chunk in bf16; `scale`: the block's (MXFP4).
template <int FMT>
__device__ __forceinline__ bf16x8 eight(const u32x4 &v, int j, float scale)
{
    u32x4 r;
    if constexpr (FMT == kLayerBf16) {
        r = v;
    } else if constexpr (FMT == kLayerFp8) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j], 1.0f, false));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j], 1.0f, true));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j + 1], 1.0f, false));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * j + 1], 1.0f, true));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[j], scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[j], scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[j], scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[j], scale, 3));
    }
    return __builtin_bit_cast(bf16x8, r);
}

// A run of 16 weight rows as one operand: lane l has row l % 16, and a quarter of
// each step's columns.
struct WeightRows {
    const uint8_t *w;     // this lane's row, at its quarter
    const uint8_t *scale; // MXFP4: the row's scales; E4M3: those of the block of rows that
                          // this lane's results belong to
};

// acc[j] += rows j of weights * b^T over steps first, first + stride, ...: b holds
// 16 rows of bf16, lane l the row l % 16, `x` at its quarter of the first step.
// acc[j][i]: weight row 4 (l / 16) + i, row l % 16 of b.
template <int FMT, int W>
__device__ __forceinline__ void products(const WeightRows (&rows)[W], const uint16_t *__restrict__ x, int first,
                                         int stride, int steps, f32x4 (&acc)[W])
{
    constexpr int C = kChunkCols<FMT>;
    constexpr int U = kAhead / W;
    const int quarter = (threadIdx.x & (kWave - 1)) >> 4;
    for (int s0 = first; s0 < steps; s0 += stride * U) {
        u32x4 v[U][W];
        uint32_t sc[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = min(s0 + u * stride, steps - 1); // (beyond the last step: unused)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                v[u][j] = *reinterpret_cast<const u32x4 *>(rows[j].w + static_cast<int64_t>(s) * 64);
                if constexpr (FMT == kLayerMxfp4) // the scales of the row's four blocks
                    sc[u][j] = *reinterpret_cast<const uint32_t *>(rows[j].scale + s * 4);
                else if constexpr (FMT == kLayerFp8)
                    sc[u][j] = *reinterpret_cast<const uint32_t *>(rows[j].scale + (s >> 1) * 4);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * stride;
            if (s >= steps)
                break;
            bf16x8 b[C / 8];
#pragma unroll
            for (int i = 0; i < C / 8; ++i)
                b[i] = *reinterpret_cast<const bf16x8 *>(x + s * (4 * C) + i * 8);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                f32x4 q = FMT == kLayerFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[j];
                const float scale = FMT == kLayerMxfp4 ? mx_scale_operand((sc[u][j] >> (quarter * 8)) & 255u) : 1.0f;
#pragma unroll
                for (int i = 0; i < C / 8; ++i)
                    q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(eight<FMT>(v[u][j], i, scale), b[i], q, 0, 0, 0);
                if constexpr (FMT == kLayerFp8) {
                    const float f = __uint_as_float(sc[u][j]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j][i] = fmaf(q[i], f, acc[j][i]);
                } else {
                    acc[j] = q;
                }
            }
        }
    }
}

// Bytes of a row of n columns.
template <int FMT>
__device__ __forceinline__ int64_t row_bytes(int n)
{
    return FMT == kLayerBf16 ? static_cast<int64_t>(n) * 2 : FMT == kLayerFp8 ? n : n >> 1;
}

// Weight row `row` of expert e of [EL, n, K] for this lane, whose results belong to
// row `mine` (E4M3 scales are of 128 rows).
template <int FMT>
__device__ __forceinline__ WeightRows weight_rows(const void *w, const void *scale, int e, int n, int K, int row,
                                                  int mine)
{
    const int quarter = (threadIdx.x & (kWave - 1)) >> 4;
    WeightRows r;
    r.w = static_cast<const uint8_t *>(w) + (static_cast<int64_t>(e) * n + row) * row_bytes<FMT>(K) + quarter * 16;
    r.scale = nullptr;
    if constexpr (FMT == kLayerMxfp4)
        r.scale = static_cast<const uint8_t *>(scale) + (static_cast<int64_t>(e) * n + row) * (K >> 5);
    else if constexpr (FMT == kLayerFp8)
        r.scale = static_cast<const uint8_t *>(scale) +
                  (static_cast<int64_t>(e) * ((n + 127) >> 7) + (mine >> 7)) * (K >> 7) * 4;
    return r;
}

// The local expert of slot s, -1 if it has none here.
__device__ __forceinline__ int slot_expert(const LayerArgs &a, int s)
{
    const int64_t id = a.idx_i64 ? static_cast<const int64_t *>(a.idx)[s] : static_cast<const int32_t *>(a.idx)[s];
    const int64_t e = id - a.lb;
    return e >= 0 && e < a.EL && id < a.E ? static_cast<int>(e) : -1;
}

__device__ __forceinline__ float layer_gated(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// The flags of the ids, by one workgroup.
__device__ void write_flags(const LayerArgs &a)
{
    __shared__ int flags;
    if (threadIdx.x == 0)
        flags = 0;
    __syncthreads();
    const auto id = [&](int s) {
        return a.idx_i64 ? static_cast<const int64_t *>(a.idx)[s]
                         : static_cast<int64_t>(static_cast<const int32_t *>(a.idx)[s]);
    };
    for (int s = threadIdx.x; s < a.slots; s += blockDim.x) {
        const int64_t mine = id(s);
        int f = mine < -1 || mine >= a.E ? 1 : 0;
        if (mine >= 0 && mine < a.E)
            for (int o = s - s % a.k; o < s; ++o)
                if (id(o) == mine)
                    f |= 2;
        if (f)
            atomicOr(&flags, f);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        *a.flags = flags;
}

// The partial sums of the waves of a workgroup, in the order of the waves, in wave 0.
template <int WAVES, int W>
__device__ __forceinline__ void add_waves(f32x4 (&acc)[W], f32x4 (*part)[W][kWave])
{
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    if (wave > 0) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            part[wave - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int p = 0; p < WAVES - 1; ++p)
                acc[j] += part[p][j][lane];
    }
}

// ---------------------------------------------------------------------------
// every slot on its own
// ---------------------------------------------------------------------------
// A workgroup has one slot and 8 columns of h: the operand's rows are 8 gate rows
// and the 8 up rows, the waves take every fourth step.  Grid: [slots][I / 8], and
// one workgroup more for the flags where they are wanted.
template <int FMT>
__global__ void __launch_bounds__(kUpWaves * kWave) k_layer_up_slots(LayerArgs a)
{
    __shared__ f32x4 part[kUpWaves - 1][1][kWave];
    const int tiles = a.I >> 3;
    const int s = blockIdx.x / tiles, n0 = (blockIdx.x - s * tiles) * 8;
    if (s == a.slots) {
        write_flags(a);
        return;
    }
    const int e = __builtin_amdgcn_readfirstlane(slot_expert(a, s));
    if (e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    const WeightRows rows[1] = {weight_rows<FMT>(a.w1, a.w1_scale, e, 2 * a.I, a.H,
                                                 l16 < 8 ? n0 + l16 : a.I + n0 + l16 - 8,
                                                 quarter < 2 ? n0 : a.I + n0)};
    const uint16_t *x = a.x + static_cast<int64_t>(s / a.k) * a.H + quarter * kChunkCols<FMT>;
    f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    products<FMT, 1>(rows, x, wave, kUpWaves, a.H / (4 * kChunkCols<FMT>), acc);
    add_waves<kUpWaves, 1>(acc, part);
    if (wave != 0)
        return;
    // gate rows in the lower half of the lanes, up rows in the upper half
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = layer_gated(acc[0][i], __shfl_xor(acc[0][i], 32));
    if (l16 == 0 && quarter < 2)
        *reinterpret_cast<u32x2 *>(a.h + static_cast<int64_t>(s) * a.I + n0 + quarter * 4) =
            u32x2{two_bf16(h[0], h[1]), two_bf16(h[2], h[3])};
}

// out[t, n] of a workgroup's columns from y[part][slot][column] in LDS: fp32, in
// ascending slot order, the first term's product rounded, each further term one fma.
template <int COLS>
__device__ __forceinline__ void sum_slots(const LayerArgs &a, const float *y, int parts, int n0)
{
    for (int i = threadIdx.x; i < a.T * (COLS / 2); i += kDownWaves * kWave) {
        const int t = i / (COLS / 2), c = (i - t * (COLS / 2)) * 2;
        float s0 = 0.f, s1 = 0.f;
        bool first = true;
        for (int j = 0; j < a.k; ++j) {
            const int s = t * a.k + j;
            if (slot_expert(a, s) < 0)
                continue;
            const float w = a.topk_w[s];
            float v0 = y[s * COLS + c], v1 = y[s * COLS + c + 1];
            for (int p = 1; p < parts; ++p) {
                v0 += y[(p * a.slots + s) * COLS + c];
                v1 += y[(p * a.slots + s) * COLS + c + 1];
            }
            s0 = first ? v0 * w : fmaf(v0, w, s0);
            s1 = first ? v1 * w : fmaf(v1, w, s1);
            first = false;
        }
        *reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(t) * a.H + n0 + c) = two_bf16(s0, s1);
    }
}

// A workgroup has 8 columns of out and all slots, two at a time: the operand's rows
// are 8 weight rows of the first one's expert and 8 of the second one's, columns 0
// and 1 of the other operand their rows of h.  Where there are fewer pairs than
// waves, several waves share one (a.parts of them).
template <int FMT>
__global__ void __launch_bounds__(kDownWaves * kWave) k_layer_down_slots(LayerArgs a)
{
    extern __shared__ float y[]; // [parts][slots][8]
    const int n0 = blockIdx.x * 8;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    const int steps = a.I / (4 * kChunkCols<FMT>);
    const int part = wave % a.parts;
    for (int p = wave / a.parts; 2 * p < a.slots; p += kDownWaves / a.parts) {
        const int s0 = 2 * p, s1 = min(s0 + 1, a.slots - 1);
        int e0 = __builtin_amdgcn_readfirstlane(slot_expert(a, s0));
        int e1 = __builtin_amdgcn_readfirstlane(slot_expert(a, s1));
        if (e0 < 0 && e1 < 0)
            continue;
        // (a slot without an expert here: the other one in its place)
        const int h0 = e0 < 0 ? s1 : s0, h1 = e1 < 0 ? s0 : s1;
        e0 = e0 < 0 ? e1 : e0;
        e1 = e1 < 0 ? e0 : e1;
        const int row = n0 + (l16 & 7);
        WeightRows rows[1] = {weight_rows<FMT>(a.w2, a.w2_scale, l16 < 8 ? e0 : e1, a.H, a.I, row, n0)};
        if constexpr (FMT == kLayerFp8)
            rows[0].scale = weight_rows<FMT>(a.w2, a.w2_scale, quarter < 2 ? e0 : e1, a.H, a.I, row, n0).scale;
        const uint16_t *h = a.h + static_cast<int64_t>(l16 == 0 ? h0 : h1) * a.I + quarter * kChunkCols<FMT>;
        f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
        products<FMT, 1>(rows, h, part, a.parts, steps, acc);
        // rows 0 .. 7 of column 0, rows 8 .. 15 of column 1
        if (l16 == quarter >> 1) {
            const int s = quarter < 2 ? s0 : s1;
            if (quarter < 2 || s1 > s0)
                *reinterpret_cast<f32x4 *>(y + (part * a.slots + s) * 8 + (quarter & 1) * 4) = acc[0];
        }
    }
    __syncthreads();
    sum_slots<8>(a, y, a.parts, n0);
}

// ---------------------------------------------------------------------------
// slots of an expert together
// ---------------------------------------------------------------------------
// What k_layer_down reads, made by one workgroup of k_layer_up: per expert in use
// and 16 of its slots an item {expert, first of its slots in the list, how many},
// and the slots expert by expert.  One wave; an expert's slots in ascending order.
__device__ void make_plan(const LayerArgs &a)
{
    __shared__ int32_t count[kMaxLocal], begin[kMaxLocal];
    const int lane = threadIdx.x & (kWave - 1);
    for (int e = threadIdx.x; e < a.EL; e += blockDim.x)
        count[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.slots; s += blockDim.x) {
        const int e = slot_expert(a, s);
        if (e >= 0)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        int slots = 0, items = 0;
        for (int base = 0; base < a.EL; base += kWave) {
            const int e = base + lane;
            const int n = e < a.EL ? count[e] : 0, m = (n + 15) >> 4;
            int in = n, im = m;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const int un = __shfl_up(in, o), um = __shfl_up(im, o);
                if (lane >= o) {
                    in += un;
                    im += um;
                }
            }
            if (e < a.EL)
                begin[e] = slots + in - n;
            for (int i = 0; i < m; ++i)
                a.plan->items[items + im - m + i] =
                    make_int4(e, slots + in - n + 16 * i, min(16, n - 16 * i), 0);
            slots += __shfl(in, kWave - 1);
            items += __shfl(im, kWave - 1);
        }
        if (lane == 0)
            a.plan->count = items;
    }
    __syncthreads();
    // every slot's place: its expert's first, and the earlier slots of that expert
    for (int s = threadIdx.x; s < a.slots; s += blockDim.x) {
        const int e = slot_expert(a, s);
        if (e < 0)
            continue;
        // (any order will do: a slot's results do not depend on its place)
        a.plan->list[atomicAdd(&begin[e], 1)] = s;
    }
}

// A workgroup has 16 columns of h for one expert: 16 gate rows and the 16 up rows,
// the waves every fourth step, 16 of the expert's slots at a time.  Expert
// workgroup i: expert i, or (fewer slots than experts) the expert of slot i where
// no earlier slot has it.  Grid: [experts or slots][I / 16], and one more for the
// plan.
template <int FMT>
__global__ void __launch_bounds__(kUpWaves * kWave) k_layer_up_experts(LayerArgs a)
{
    __shared__ f32x4 part[kUpWaves - 1][2][kWave];
    __shared__ int32_t list[kLayerMaxSlots];
    const int tiles = a.I >> 4;
    const int i0 = blockIdx.x / tiles, n0 = (blockIdx.x - i0 * tiles) * 16;
    const bool by_slot = a.slots < a.EL;
    if (i0 == (by_slot ? a.slots : a.EL)) {
        make_plan(a);
        if (a.flags)
            write_flags(a);
        return;
    }
    const int e = __builtin_amdgcn_readfirstlane(by_slot ? slot_expert(a, i0) : i0);
    if (e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    int n = 0;
    for (int base = 0; base < a.slots; base += kWave) {
        const int s = base + lane;
        const uint64_t m = __ballot(s < a.slots && slot_expert(a, s) == e);
        if (by_slot && n == 0 && m && base + __builtin_ctzll(m) < i0)
            return; // an earlier slot's workgroups have this expert
        if (wave == 0 && (m >> lane & 1))
            list[n + __popcll(m & ((1ull << lane) - 1))] = s;
        n += __popcll(m);
    }
    if (n == 0)
        return;
    __syncthreads();
    const WeightRows rows[2] = {weight_rows<FMT>(a.w1, a.w1_scale, e, 2 * a.I, a.H, n0 + l16, n0),
                                weight_rows<FMT>(a.w1, a.w1_scale, e, 2 * a.I, a.H, a.I + n0 + l16, a.I + n0)};
    for (int p = 0; p < n; p += 16) {
        const int s = list[min(p + l16, n - 1)];
        const uint16_t *x = a.x + static_cast<int64_t>(s / a.k) * a.H + quarter * kChunkCols<FMT>;
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        products<FMT, 2>(rows, x, wave, kUpWaves, a.H / (4 * kChunkCols<FMT>), acc);
        add_waves<kUpWaves, 2>(acc, part);
        if (wave == 0 && p + l16 < n) {
            float h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[i] = layer_gated(acc[0][i], acc[1][i]);
            *reinterpret_cast<u32x2 *>(a.h + static_cast<int64_t>(s) * a.I + n0 + quarter * 4) =
                u32x2{two_bf16(h[0], h[1]), two_bf16(h[2], h[3])};
        }
        if (p + 16 < n)
            __syncthreads(); // the sums are read: room for the next slots'
    }
}

// A workgroup has 16 columns of out; its waves take the plan's items in turn.
template <int FMT>
__global__ void __launch_bounds__(kDownWaves * kWave) k_layer_down_experts(LayerArgs a)
{
    extern __shared__ float y[]; // [slots][16]
    const int n0 = blockIdx.x * 16;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    const int items = a.plan->count;
    for (int i = wave; i < items; i += kDownWaves) {
        const int4 it = a.plan->items[i];
        const int e = __builtin_amdgcn_readfirstlane(it.x);
        const int s = a.plan->list[it.y + min(l16, it.z - 1)];
        const WeightRows rows[1] = {weight_rows<FMT>(a.w2, a.w2_scale, e, a.H, a.I, n0 + l16, n0)};
        const uint16_t *h = a.h + static_cast<int64_t>(s) * a.I + quarter * kChunkCols<FMT>;
        f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
        products<FMT, 1>(rows, h, 0, 1, a.I / (4 * kChunkCols<FMT>), acc);
        if (l16 < it.z)
            *reinterpret_cast<f32x4 *>(y + s * 16 + quarter * 4) = acc[0];
    }
    __syncthreads();
    sum_slots<16>(a, y, 1, n0);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
template <int FMT>
static hipError_t launch_layer_of(const LayerArgs &a0, hipStream_t s)
{
    LayerArgs a = a0;
    const dim3 up(kUpWaves * kWave), down(kDownWaves * kWave);
    if (a.slots <= kLayerSingleSlots) {
        const int pairs = (a.slots + 1) / 2;
        a.parts = 1;
        while (a.parts * 2 * pairs <= kDownWaves)
            a.parts *= 2;
        launch(k_layer_up_slots<FMT>, dim3(a.slots * (a.I / 8) + (a.flags ? 1 : 0)), up, 0, s, a);
        launch(k_layer_down_slots<FMT>, dim3(a.H / 8), down, a.parts * a.slots * 8 * sizeof(float), s, a);
    } else {
        const int64_t groups = a.slots < a.EL ? a.slots : a.EL;
        launch(k_layer_up_experts<FMT>, dim3(static_cast<unsigned>(groups * (a.I / 16) + 1)), up, 0, s, a);
        launch(k_layer_down_experts<FMT>, dim3(a.H / 16), down, a.slots * 16 * sizeof(float), s, a);
    }
    return hipGetLastError();
}

hipError_t launch_layer(const LayerArgs &a, int fmt, hipStream_t s)
{
    switch (fmt) {
    case kLayerBf16: return launch_layer_of<kLayerBf16>(a, s);
    case kLayerFp8: return launch_layer_of<kLayerFp8>(a, s);
    default: return launch_layer_of<kLayerMxfp4>(a, s);
    }
}

}  // namespace moe
