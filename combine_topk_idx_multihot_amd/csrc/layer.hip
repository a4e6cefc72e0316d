// layer.hip -- a whole MoE layer for a few tokens, in two kernels or three.
//
//   h[s]   = silu(W1g[e] x[t]) * (W1u[e] x[t])          for every slot s = (t, j), e its expert
//   out[t] = sum over t's local slots of w[s] * W2[e] h[s]
// No rows are laid out: the first kernel writes h to the
// workspace, the second one multiplies it and sums a token's slots (where slots
// share weights a third one does).
// The weights of the experts in use are what has to be read; tokens and h are
// small and come from the L2.  Weights are widened to bf16 in registers (E4M3 and
// E2M1 codes are exact there, an E8M0 scale too) and multiplied with bf16 tokens
// in fp32; the fp32 scale of a block of E4M3 weights enters after the products of
// its columns.  Tokens that are not quantized cost nothing here: the rates of the
// units are several times what the weights' bytes need.  Everything stays in fp32 until out, but h
// where slots share weights, which is an operand of the matrix instructions: two bf16 terms, its rounding and the
// rest, about 16 bits in all (the outputs' error against 64 bits is the final rounding's then, 0.0017 relative; with
// one term 0.0024).
//
// There are two forms.  With few slots every slot is on its own (an
// expert that two tokens share is read twice, the second time from the L2): a wave
// keeps its share of the token in registers and passes whole rows of weights by it.
// With more, slots of the same expert share its weights in the matrix
// instructions, up to 16 of them; a third kernel adds up a token's slots.  (These sums by the
// last workgroup of a column tile to arrive took 288 us instead of 26 at 32 tokens, H = 2048, I =
// 768, 128 experts: what one XCD wrote has to leave its L2 at every workgroup's end.)
#include "expert_tiles.h"
#include "mx.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kLayerWaves = 4;

// Columns that 16 bytes of weights hold: a chunk.
template <int FMT>
constexpr int kChunkCols = FMT == kLayerBf16 ? 8 : FMT == kLayerFp8 ? 16 : 32;

// Columns 8 j .. 8 j + 7 of a chunk in bf16; `scale`: the block's (MXFP4).
template <int FMT>
__device__ __forceinline__ u32x4 eight(const u32x4 &v, int j, float scale)
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
    return r;
}

// Bytes of a row of n columns.
template <int FMT>
__device__ __forceinline__ int64_t row_bytes(int n)
{
    return FMT == kLayerBf16 ? static_cast<int64_t>(n) * 2 : FMT == kLayerFp8 ? n : n >> 1;
}

// Row `row` of expert e of weights [EL, n, K], and its scales: MXFP4 a byte per 32
// columns, E4M3 an fp32 per 128.
template <int FMT>
__device__ __forceinline__ const uint8_t *weight_row(const void *w, int e, int n, int K, int row)
{
    return static_cast<const uint8_t *>(w) + (static_cast<int64_t>(e) * n + row) * row_bytes<FMT>(K);
}
template <int FMT>
__device__ __forceinline__ const uint8_t *scale_row(const void *scale, int e, int n, int K, int row)
{
    const uint8_t *p = static_cast<const uint8_t *>(scale);
    if constexpr (FMT == kLayerMxfp4)
        p += (static_cast<int64_t>(e) * n + row) * (K >> 5);
    else if constexpr (FMT == kLayerFp8)
        p += (static_cast<int64_t>(e) * ((n + 127) >> 7) + (row >> 7)) * (K >> 7) * 4;
    return p;
}

// What the rounding of x and y to `top` leaves (nothing of an infinity), in bf16 itself.
__device__ __forceinline__ uint32_t rest_bf16(float x, float y, uint32_t top)
{
    x -= __uint_as_float(top << 16);
    y -= __uint_as_float(top & 0xFFFF0000u);
    return pack_bf16(fabsf(x) < INFINITY ? x : 0.f, fabsf(y) < INFINITY ? y : 0.f);
}

// The local expert of slot s, -1 if it has none here.
__device__ __forceinline__ int slot_expert(const LayerArgs &a, int s)
{
    // both widths without a branch, so that loads of several ids go out together
    const int32_t *p = static_cast<const int32_t *>(a.idx) + (static_cast<int64_t>(s) << a.idx_i64);
    const int id = p[0], high = p[a.idx_i64];
    const bool whole = !a.idx_i64 || high == 0; // (the ids that matter are not negative)
    // (without a sign: an id below lb, however far, becomes one above every expert)
    const uint32_t e = static_cast<uint32_t>(id) - static_cast<uint32_t>(a.lb);
    return whole && e < static_cast<uint32_t>(a.EL) ? static_cast<int>(e) : -1;
}

// The flags of the ids, by one workgroup; `flags`: a word of its LDS.
__device__ void write_flags(const LayerArgs &a, int *flags)
{
    if (threadIdx.x == 0)
        *flags = 0;
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
            atomicOr(flags, f);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        *a.flags = *flags;
}

// ---------------------------------------------------------------------------
// every slot on its own
// ---------------------------------------------------------------------------
// Rows of weights pass by a wave 64 chunks (1 KB) at a time, lane l the chunk l of
// them, so that a load is as wide as loads get; the same columns of the token stay
// in registers for all rows of the wave.  Two products per instruction, rows
// interleaved.  (With the matrix instructions, whose lanes have 16 rows of weights
// and 4 chunks of columns, a chunk of MXFP4 needs four loads of the token beside
// its own: one token, H = 4096, I = 1024 14.5 us for the first kernel.)
// The two kernels, us (bytes): one token, top-8 of 128, E4M3, H = 2048, I = 768 6.4 (25 MB)
// and 5.7 (13 MB), MXFP4, H = 4096, I = 1024 8.4 (36 MB) and 7.1 (18 MB): latency counts
// as much as HBM.  5 tokens, top-6 of 64, half of them local, bf16 15.2 (70 MB) and 9.6 (35 MB).
// h is fp32, in the order in which the second kernel's lanes take it (row after row, lanes 128 bytes apart with
// MXFP4: top-8 of 128, whole layer, T = 1, H = 4096, I = 1024 20.6 us instead of 16.9, T = 6, H = 2048, I = 768 40.0
// instead of 32.5).

// The sum over the wave's lanes, in lane 63: in rows of 16 lanes, then across them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<0x111>(v); // row_shr:1, 2, 4, 8
    v = dpp_add<0x112>(v);
    v = dpp_add<0x114>(v);
    v = dpp_add<0x118>(v);
    v = dpp_add<0x142>(v); // row_bcast:15, 31
    return dpp_add<0x143>(v);
}

// A chunk's products with its columns of the token, added to acc (E4M3: under the
// block's scale).
template <int FMT>
__device__ __forceinline__ float chunk_dot(const u32x4 &w, uint32_t scale, const u32x4 (&x)[kChunkCols<FMT> / 8],
                                           float acc)
{
    float q = FMT == kLayerFp8 ? 0.f : acc;
    const float s = FMT == kLayerMxfp4 ? mx_scale_operand(scale) : 1.0f;
#pragma unroll
    for (int j = 0; j < kChunkCols<FMT> / 8; ++j) {
        const u32x4 v = eight<FMT>(w, j, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (copies: this compiler takes the first element for any in a bit cast of one)
            const uint32_t a = v[i], b = x[j][i];
            q = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), q, false);
        }
    }
    return FMT == kLayerFp8 ? fmaf(q, __uint_as_float(scale), acc) : q;
}

// The same with columns of h, in fp32.
template <int FMT>
__device__ __forceinline__ float chunk_dot32(const u32x4 &w, uint32_t scale, const f32x4 (&h)[kChunkCols<FMT> / 4],
                                             float acc)
{
    float q = FMT == kLayerFp8 ? 0.f : acc;
    const float s = FMT == kLayerMxfp4 ? mx_scale_operand(scale) : 1.0f;
#pragma unroll
    for (int j = 0; j < kChunkCols<FMT> / 2; ++j) {
        f32x2 v;
        if constexpr (FMT == kLayerBf16) {
            v[0] = __uint_as_float(w[j] << 16);
            v[1] = __uint_as_float(w[j] & 0xFFFF0000u);
        } else if constexpr (FMT == kLayerFp8) {
            v = j & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[j >> 1], 1.0f, true)
                      : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[j >> 1], 1.0f, false);
        } else {
            const uint32_t word = w[j >> 2];
            v = (j & 3) == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 0)
                : (j & 3) == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 1)
                : (j & 3) == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 2)
                               : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, s, 3);
        }
        q = fmaf(v[0], h[j >> 1][2 * (j & 1)], q);
        q = fmaf(v[1], h[j >> 1][2 * (j & 1) + 1], q);
    }
    return FMT == kLayerFp8 ? fmaf(q, __uint_as_float(scale), acc) : q;
}

// The scale that chunk c of a row goes with.
template <int FMT>
__device__ __forceinline__ uint32_t chunk_scale(const uint8_t *scales, int c)
{
    if constexpr (FMT == kLayerMxfp4)
        return scales[c];
    else if constexpr (FMT == kLayerFp8)
        return reinterpret_cast<const uint32_t *>(scales)[c >> 3];
    return 0;
}

// Where a slot's row of h has quad i of the columns that chunk c of a row of W2 is multiplied with:
// lanes have consecutive chunks, and read consecutive quads.
template <int FMT>
__device__ __forceinline__ int h_quad(int I, int c, int i)
{
    return (i * (I / kChunkCols<FMT>) + c) * 4;
}

// A wave has one slot and N columns of h, N gate rows and N up rows.  Grid: [slots]
// [I / (4 N)], and one workgroup more for the flags where they are wanted.
template <int FMT>
__global__ void __launch_bounds__(kLayerWaves * kWave) k_layer_up_slots(LayerArgs a)
{
    constexpr int N = kLayerUpCols, U = kLayerUpAhead, C = kChunkCols<FMT>;
    const int tiles = a.I / (kLayerWaves * N);
    const int s = blockIdx.x / tiles;
    __shared__ int flags;
    if (s == a.slots) {
        write_flags(a, &flags);
        return;
    }
    const int e = __builtin_amdgcn_readfirstlane(slot_expert(a, s));
    if (e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int n0 = ((blockIdx.x - s * tiles) * kLayerWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave)) * N;
    const uint16_t *x = a.x + static_cast<int64_t>(s / a.k) * a.H;
    const int64_t stride = row_bytes<FMT>(a.H);
    const uint8_t *wg = weight_row<FMT>(a.w1, e, 2 * a.I, a.H, n0), *wu = wg + a.I * stride;
    const uint8_t *sg = scale_row<FMT>(a.w1_scale, e, 2 * a.I, a.H, n0);
    const uint8_t *su = scale_row<FMT>(a.w1_scale, e, 2 * a.I, a.H, a.I + n0);
    // (N divides 128: E4M3 scales are the same for all of the wave's columns)
    const int scale_stride = FMT == kLayerMxfp4 ? a.H >> 5 : 0;
    float acc[2 * N];
#pragma unroll
    for (int i = 0; i < 2 * N; ++i)
        acc[i] = 0.f;
    const int chunks = a.H / C;
    for (int c0 = lane; c0 < chunks + lane; c0 += U * kWave) {
        u32x4 v[U][2 * N], xv[U][C / 8];
        uint32_t sc[U][2 * N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = min(c0 + u * kWave, chunks - 1); // (beyond the row: left out below)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[u][i] = *reinterpret_cast<const u32x4 *>(wg + i * stride + c * 16);
                v[u][N + i] = *reinterpret_cast<const u32x4 *>(wu + i * stride + c * 16);
                sc[u][i] = chunk_scale<FMT>(sg + i * scale_stride, c);
                sc[u][N + i] = chunk_scale<FMT>(su + i * scale_stride, c);
            }
#pragma unroll
            for (int j = 0; j < C / 8; ++j)
                xv[u][j] = *reinterpret_cast<const u32x4 *>(x + c * C + j * 8);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = c0 + u * kWave < chunks;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) {
                const float q = chunk_dot<FMT>(v[u][i], sc[u][i], xv[u], acc[i]);
                acc[i] = in ? q : acc[i];
            }
        }
    }
    float h[N];
#pragma unroll
    for (int i = 0; i < 2 * N; ++i)
        acc[i] = wave_sum(acc[i]);
#pragma unroll
    for (int i = 0; i < N; ++i)
        h[i] = gated(acc[i], acc[N + i]);
    if (lane == kWave - 1) {
        static_assert(N == 2, "columns of one quad");
        float *o = reinterpret_cast<float *>(a.h) + static_cast<int64_t>(s) * a.I;
        *reinterpret_cast<f32x2 *>(o + h_quad<FMT>(a.I, n0 / C, n0 % C >> 2) + (n0 & 3)) = f32x2{h[0], h[1]};
    }
}

// A wave has one token and N columns of out: the rows of its slots' experts one
// behind the other, 64 chunks at a time.  A lane's products of a chunk are
// multiplied with its slot's weight and added up; the lanes' sums last.  Grid: [T]
// [H / (4 N)].
template <int FMT>
__global__ void __launch_bounds__(kLayerWaves * kWave) k_layer_down_slots(LayerArgs a)
{
    constexpr int N = kLayerDownCols, U = kLayerDownAhead, C = kChunkCols<FMT>;
    const int tiles = a.H / (kLayerWaves * N);
    const int t = blockIdx.x / tiles;
    const int lane = threadIdx.x & (kWave - 1);
    const int n0 = ((blockIdx.x - t * tiles) * kLayerWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave)) * N;
    // the token's local slots, one per lane (k <= 64), the first ones first
    const int mine = lane < a.k ? slot_expert(a, t * a.k + lane) : -1;
    uint64_t local = __ballot(mine >= 0);
    const int count = __popcll(local);
    const float w = mine >= 0 ? a.topk_w[t * a.k + lane] : 0.f;
    // lane i: the i-th local slot
    int from = 0;
    for (int i = 0; i < count; ++i) {
        const int b = __builtin_ctzll(local);
        local &= local - 1;
        from = lane == i ? b : from;
    }
    const int expert = __shfl(mine, from);
    const float weight = __shfl(w, from);
    const int per = a.I / C; // chunks of a row
    const int total = count * per;
    const int64_t stride = row_bytes<FMT>(a.I);
    const int scale_stride = FMT == kLayerMxfp4 ? a.I >> 5 : 0;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = 0.f;
    for (int base = 0; base < total; base += U * kWave) {
        u32x4 v[U][N];
        f32x4 hv[U][C / 4];
        uint32_t sc[U][N];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = min(base + u * kWave + lane, total - 1); // (beyond the last: left out below)
            const int j = at / per, c = at - j * per;
            const int e = __shfl(expert, j), slot = t * a.k + __shfl(from, j);
            f[u] = __shfl(weight, j);
            const uint8_t *wr = weight_row<FMT>(a.w2, e, a.H, a.I, n0) + c * 16;
            const uint8_t *sr = scale_row<FMT>(a.w2_scale, e, a.H, a.I, n0);
            const float *h = reinterpret_cast<const float *>(a.h) + static_cast<int64_t>(slot) * a.I;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[u][i] = *reinterpret_cast<const u32x4 *>(wr + i * stride);
                sc[u][i] = chunk_scale<FMT>(sr + i * scale_stride, c);
            }
#pragma unroll
            for (int i = 0; i < C / 4; ++i)
                hv[u][i] = *reinterpret_cast<const f32x4 *>(h + h_quad<FMT>(a.I, c, i));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = base + u * kWave + lane < total;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float q = chunk_dot32<FMT>(v[u][i], sc[u][i], hv[u], 0.f);
                acc[i] = in ? fmaf(q, f[u], acc[i]) : acc[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = wave_sum(acc[i]);
    if (lane == kWave - 1) {
        uint32_t *o = reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(t) * a.H + n0);
#pragma unroll
        for (int i = 0; i < N; i += 2)
            o[i / 2] = pack_bf16(acc[i], acc[i + 1]);
    }
}

// ---------------------------------------------------------------------------
// slots of an expert together
// ---------------------------------------------------------------------------
// Weights are one operand of the 16x16x32 bf16 instructions, 16 rows each, 16 slots the
// other; a lane has row l % 16 of both and a quarter of the columns of four chunks.
// Weights come through LDS, whole lines at a time, and so do the tokens (or rows of h):
// workgroups walk a list of tiles of one expert, up to 16 of its slots and 128 weight rows (64 gate and
// 64 up rows, or 128 rows of W2); their steps of 128 bytes of each row (64 where MXFP4 goes with two
// terms of h) go through a ring of three or four stages, all but one of them, across tiles, on their way at any time.  A wave
// has 32 weight rows for all columns: two runs of 16, in the first kernel gate and up rows
// of the same columns of h.
// (Weights from HBM to registers, a load taking 64 bytes of 16 rows, whose address units were busy
// 72 % of the cycles with MXFP4: with one term of h, top-8 of 128, H = 2048, I = 768, 32 tokens MXFP4 86 us instead
// of 63, E4M3 123 / 109, bf16 206 / 218; 128 tokens 142 / 99, 181 / 139, 274 / 256; top-2 of 8, H =
// I = 2048, 256 tokens 85 / 53, 104 / 68, 169 / 87.)
//
// Bound by HBM, the second kernel by the bytes on their way: 32 tokens with MXFP4 weights 41.2 and 29.3 us (186 and
// 95 MB: 4.5 and 3.2 TB/s), and 4.9 us for the sums.
//
// A stage: 128 weight rows, their scales (MXFP4 a byte per 32 columns; E4M3 each wave's two, of
// its runs' blocks), and 16 rows of bf16: tokens, or rows of h, once for each term.  Where the tile has no slots for
// a wave's rows it brings none: what the stage holds there enters only results that are dropped (all 16
// always: 64.7 us instead of 62.9 at 32 tokens, MXFP4).
//
// The second kernel multiplies both terms of h with the weights that it has widened.  Top-8 of 128, H = 2048, I = 768, whole
// layer, one term / two: MXFP4 T = 8 39.7 / 41.6, T = 32 68.6 / 72.9, T = 128 99.7 / 104.6; E4M3 T = 32 106.8 / 107.0,
// T = 128 134 / 137; bf16 T = 32 215 / 212.  MXFP4, T = 32, 64, 128 (73.7, 86.1, 106.2 here): steps of 128 bytes, whose
// 1 KB per slot leaves room for two stages, 73.0, 84.3, 103.8, with a last half step to treat apart; tiles of 256 rows
// and three stages 75.3, 83.5, 98.8, but top-2 of 8, H = I = 2048, T = 64 37.5 instead of 33.5; eight waves that share
// three stages of 128 bytes, one workgroup per CU, 75.5, 86.0, 108.2.
template <int FMT, bool UP>
struct LayerRing {
    static constexpr int kPlanes = UP ? 1 : 2; // of rows of bf16: tokens, or h's two terms
    static constexpr int kStages = UP ? (FMT == kLayerBf16 ? 4 : 3) : (FMT == kLayerMxfp4 ? 4 : 3);
    static constexpr int kChunks = !UP && FMT == kLayerMxfp4 ? 4 : 8; // of 16 bytes, of a weight row in a step
    static constexpr int kCols = kChunks * kChunkCols<FMT>; // columns of a step
    static constexpr int kWRows = 64 / kChunks;       // weight rows that a load of a wave brings
    static constexpr int kWLoads = 32 / kWRows;       // loads of a wave for its 32
    static constexpr int kXBytes = 2 * kCols;         // a row of bf16 in a step
    static constexpr int kXRows = 1024 / kXBytes;     // such rows that a load of a wave brings
    static constexpr int kXLoads = kXRows < 4 ? 4 / kXRows : 1; // loads of a wave for a plane of them
    static constexpr uint32_t kSW = 128 * 16 * kChunks; // in a stage: weight rows, their scales,
    static constexpr uint32_t kX = kSW + (FMT == kLayerBf16 ? 0 : kLayerWaves * 256); // planes of 16 rows of bf16
    static constexpr uint32_t kPlane = 16 * kXBytes;
    static constexpr uint32_t kStage = kX + kPlanes * kPlane;
    static constexpr int kLoads = kWLoads + (FMT != kLayerBf16); // loads of a wave per step, but for rows of bf16
    // where row r of bf16 keeps its chunk c, and which chunk is at place c (rows in whose way
    // 16 others lie on the same banks); the same of weight rows
    __device__ static __forceinline__ int place(int r, int c) { return kXBytes < 256 ? place_of(r, c) : c ^ (r & 15); }
    __device__ static __forceinline__ int wplace(int r, int c) { return kChunks == 8 ? place_of(r, c) : c ^ ((r >> 2) & 3); }
    static constexpr uint32_t kExpert = kStages * kStage;           // the slots' experts, 16 bits each
    static constexpr uint32_t kItem = kExpert + kLayerMaxSlots * 2; // items: expert * 64 + pass, 16 bits
    static constexpr uint32_t kCount = kItem + kLayerMaxSlots * 2;  // how many
    static constexpr uint32_t kList = kCount + 16;                  // [wave][16] slots of a tile, 16 bits
    static constexpr uint32_t kBytes = kList + kLayerWaves * 16 * 2;
    static_assert(2 * (kBytes + 512) <= 160 * 1024, "two workgroups per CU");
    static_assert(kStages * kStage >= kMaxLocal * 4, "the counters lie in the stages");
    static_assert(kLayerMaxSlots <= 16 * 64 && kMaxLocal <= 1024, "16 bits for an item");
};
typedef __attribute__((address_space(3))) uint16_t *lds_half;
typedef const __attribute__((address_space(3))) u32x2 *lds_pair;
typedef const __attribute__((address_space(3))) uint32_t *lds_word;

// The slots' experts, and per expert in use and 16 of its slots an item, experts in order.
template <typename L>
__device__ __forceinline__ void ring_tables(const LayerArgs &a)
{
    const int lane = threadIdx.x & (kWave - 1);
    for (int e = threadIdx.x; e < a.EL; e += blockDim.x)
        *lds_at<lds_int>(e * 4) = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.slots; s += blockDim.x) {
        const int e = slot_expert(a, s);
        *lds_at<lds_half>(L::kExpert + s * 2) = static_cast<uint16_t>(e); // (none: 65535)
        if (e >= 0)
            __hip_atomic_fetch_add(lds_at<lds_int>(e * 4), 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        int items = 0;
        for (int base = 0; base < a.EL; base += kWave) {
            const int e = base + lane;
            const int m = e < a.EL ? (*lds_at<lds_int>(e * 4) + 15) >> 4 : 0;
            int in = m;
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) {
                const int u = __shfl_up(in, o);
                if (lane >= o)
                    in += u;
            }
            for (int i = 0; i < m; ++i)
                *lds_at<lds_half>(L::kItem + (items + in - m + i) * 2) = static_cast<uint16_t>(e * 64 + i);
            items += __shfl(in, kWave - 1);
        }
        if (lane == 0)
            *lds_at<lds_int>(L::kCount) = items;
    }
    __syncthreads(); // (the counters are read: room for the stages)
}

// The slots of an item, in ascending order, to this wave's list; how many.
template <typename L>
__device__ __forceinline__ int ring_slots(const LayerArgs &a, int item)
{
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t list = L::kList + uniform(threadIdx.x / kWave) * 32;
    const int e = item >> 6, first = (item & 63) * 16;
    int n = 0;
    for (int base = 0; base < a.slots && n < first + 16; base += kWave) {
        const int s = base + lane;
        const bool in = s < a.slots && *lds_at<lds_half>(L::kExpert + s * 2) == e;
        const uint64_t m = __ballot(in);
        const int rank = n + __popcll(m & ((1ull << lane) - 1)) - first;
        if (in && rank >= 0 && rank < 16)
            *lds_at<lds_half>(list + rank * 2) = static_cast<uint16_t>(s);
        n += __popcll(m);
    }
    __builtin_amdgcn_wave_barrier(); // (a wave's LDS accesses are in order)
    return min(16, n - first);
}

template <int FMT, bool UP>
__global__ void __launch_bounds__(kLayerWaves * kWave) k_layer_ring(LayerArgs a)
{
    typedef LayerRing<FMT, UP> L;
    constexpr int C = kChunkCols<FMT>;
    extern __shared__ uint8_t ring_lds[]; // from 0, and the kernel's only LDS
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    // (the compiler does not see the loads to LDS: the array's address escapes)
    asm volatile("" : : "v"(ring_lds) : "memory");
    if (UP && a.flags && blockIdx.x == gridDim.x - 1) {
        write_flags(a, reinterpret_cast<int *>(ring_lds));
        return;
    }
    ring_tables<L>(a);
    const int K = UP ? a.H : a.I, N = UP ? 2 * a.I : a.H; // columns and rows of an expert's weights
    const int ntn = UP ? a.I / 64 : a.H / 128;
    const int tiles = uniform(*lds_at<lds_int>(L::kCount)) * ntn;
    const int stride = gridDim.x - (UP && a.flags ? 1 : 0);
    const int steps = K / L::kCols; // (a whole number: H is a multiple of 256, I of 128)
    const uint32_t row_stride = static_cast<uint32_t>(row_bytes<FMT>(K)), row_blocks = K >> 5;
    const uint8_t *const weights = static_cast<const uint8_t *>(UP ? a.w1 : a.w2);
    const uint8_t *const scales = static_cast<const uint8_t *>(UP ? a.w1_scale : a.w2_scale);
    const uint8_t *const rows = reinterpret_cast<const uint8_t *>(UP ? a.x : a.h);

    // ---- loads: the tile and step to send for, and where it goes
    int to = blockIdx.x - stride, to_b = steps, to_stage = 0;
    uint32_t woff[L::kWLoads], wrow = 0;
    const uint8_t *wbase = nullptr, *swbase = nullptr, *xrow[L::kXLoads] = {};
    bool with_x = true; // the newest loads have rows of bf16 among them
    const int64_t to_rest = static_cast<int64_t>(a.slots) * K * 2;
    const auto send = [&]() {
        if (to >= tiles)
            return;
        if (to_b == steps) {
            to += stride;
            if (to >= tiles)
                return;
            to_b = 0;
            const int which = to / ntn, ni = to - which * ntn;
            const int item = uniform(*lds_at<lds_half>(L::kItem + which * 2));
            const int n = ring_slots<L>(a, item);
            const int64_t first = static_cast<int64_t>(item >> 6) * N +
                                  (UP ? ni * 64 + (wave >= 2 ? a.I : 0) + (wave & 1) * 32 : ni * 128 + wave * 32);
            wbase = weights + first * row_stride;
            if constexpr (FMT == kLayerMxfp4) {
                swbase = scales + first * row_blocks;
                // (a row's one or two words; of one, the upper lanes' are copies)
                wrow = L::kChunks == 8 ? (lane >> 1) * row_blocks + (lane & 1) * 4 : (lane & 31) * row_blocks;
            } else if constexpr (FMT == kLayerFp8) { // (a run's rows lie in one block) lane j: run j % 2
                const int row = UP ? (lane & 1) * a.I + ni * 64 : ni * 128;
                swbase = scale_row<FMT>(scales, item >> 6, N, K, row);
            }
#pragma unroll
            for (int i = 0; i < L::kWLoads; ++i) {
                const int r = i * L::kWRows + lane / L::kChunks;
                woff[i] = r * row_stride + L::wplace(r, lane & (L::kChunks - 1)) * 16;
            }
            with_x = wave * L::kXLoads * L::kXRows < n;
#pragma unroll
            for (int i = 0; i < L::kXLoads; ++i) {
                const int r = (wave * L::kXLoads + i) * L::kXRows + lane * 16 / L::kXBytes;
                const int s = *lds_at<lds_half>(L::kList + wave * 32 + min(r, n - 1) * 2);
                xrow[i] = rows + static_cast<int64_t>(UP ? s / a.k : s) * K * 2;
            }
        }
        const uint32_t at = uniform(to_stage) * L::kStage;
#pragma unroll
        for (int i = 0; i < L::kWLoads; ++i)
            lds_load16(at + (wave * L::kWLoads + i) * 1024, wbase + to_b * (16 * L::kChunks) + woff[i]);
        if constexpr (FMT == kLayerMxfp4)
            lds_load4(at + L::kSW + wave * 256, swbase + to_b * L::kChunks + wrow);
        else if constexpr (FMT == kLayerFp8)
            lds_load4(at + L::kSW + wave * 256, swbase + to_b * 4);
#pragma unroll
        for (int i = 0; i < L::kXLoads; ++i) {
            if (!with_x)
                break;
            const int r = (wave * L::kXLoads + i) * L::kXRows + lane * 16 / L::kXBytes;
            const int c = L::place(r, lane & (L::kXBytes / 16 - 1));
#pragma unroll
            for (int p = 0; p < L::kPlanes; ++p)
                lds_load16(at + L::kX + p * L::kPlane + (wave * L::kXLoads + i) * 1024,
                           xrow[i] + p * to_rest + to_b * L::kXBytes + c * 16);
        }
        ++to_b;
        to_stage = to_stage + 1 == L::kStages ? 0 : to_stage + 1;
    };
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i)
        send();

    // ---- products
    int stage = 0;
    for (int t = blockIdx.x; t < tiles; t += stride) {
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        for (int b = 0; b < steps; ++b) {
            // this step's loads are there: the next step's are newer
            if (to >= tiles)
                step_barrier<0>();
            else if (with_x)
                step_barrier<(L::kStages - 2) * L::kLoads + L::kXLoads * L::kPlanes>(); // (of steps but the newest: at least)
            else
                step_barrier<(L::kStages - 2) * L::kLoads>();
            send(); // over the stage before, which every wave is done with
            const uint32_t at = stage * L::kStage;
            int mine[2];
            u32x2 sc[2];
            f32x4 sum[2]; // E4M3: of this step, whose columns have one scale
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mine[j] = UP ? j * 64 + wave * 16 + l16 : wave * 32 + j * 16 + l16;
                sc[j] = u32x2{0u, 0u};
                if constexpr (FMT == kLayerMxfp4 && L::kChunks == 8)
                    sc[j] = *lds_at<lds_pair>(at + L::kSW + mine[j] * 8);
                else if constexpr (FMT == kLayerMxfp4)
                    sc[j][0] = *lds_at<lds_word>(at + L::kSW + wave * 256 + (j * 16 + l16) * 4);
                sum[j] = FMT == kLayerFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[j];
            }
#pragma unroll
            for (int u = 0; u < L::kChunks / 4; ++u) { // four chunks of a row
                u32x4 x[L::kPlanes][C / 8];
#pragma unroll
                for (int p = 0; p < L::kPlanes; ++p)
#pragma unroll
                    for (int i = 0; i < C / 8; ++i)
                        x[p][i] = *lds_at<lds_chunk>(at + L::kX + p * L::kPlane + l16 * L::kXBytes +
                                                     L::place(l16, (u * 4 + quarter) * (C / 8) + i) * 16);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const u32x4 w = *lds_at<lds_chunk>(at + mine[j] * (16 * L::kChunks) +
                                                       L::wplace(mine[j], u * 4 + quarter) * 16);
                    const uint32_t word = sc[j][u];
                    const float f = mx_scale_operand((word >> (quarter * 8)) & 255u);
#pragma unroll
                    for (int i = 0; i < C / 8; ++i) {
                        const bf16x8 v = __builtin_bit_cast(bf16x8, eight<FMT>(w, i, f));
#pragma unroll
                        for (int p = 0; p < L::kPlanes; ++p)
                            sum[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, x[p][i]),
                                                                             sum[j], 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (FMT == kLayerFp8) {
                    const float f = *lds_at<lds_float>(at + L::kSW + wave * 256 + j * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j][i] = fmaf(sum[j][i], f, acc[j][i]);
                } else {
                    acc[j] = sum[j];
                }
            }
            stage = stage + 1 == L::kStages ? 0 : stage + 1;
        }
        // acc[j][i]: weight row 4 quarter + i of run j, slot l16 of the tile
        const int which = t / ntn, ni = t - which * ntn;
        const int n = ring_slots<L>(a, uniform(*lds_at<lds_half>(L::kItem + which * 2)));
        if (l16 < n) {
            const int64_t s = *lds_at<lds_half>(L::kList + wave * 32 + l16 * 2);
            if constexpr (UP) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = gated(acc[0][i], acc[1][i]);
                uint16_t *o = a.h + s * a.I + ni * 64 + wave * 16 + quarter * 4;
                const u32x2 top = {pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
                *reinterpret_cast<u32x2 *>(o) = top;
                *reinterpret_cast<u32x2 *>(o + static_cast<int64_t>(a.slots) * a.I) =
                    u32x2{rest_bf16(h[0], h[1], top[0]), rest_bf16(h[2], h[3], top[1])};
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<f32x4 *>(a.y + s * a.H + ni * 128 + wave * 32 + j * 16 + quarter * 4) = acc[j];
            }
        }
    }
    // no load to LDS may be left when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// ---------------------------------------------------------------------------
// out[t, n] from the slots' rows, in ascending slot order: the first term's product
// rounded, each further term one fma.  A thread has four columns of a token.
__global__ void __launch_bounds__(kLayerWaves * kWave) k_layer_sum(LayerArgs a)
{
    const int quads = a.H >> 2;
    const int i = blockIdx.x * (kLayerWaves * kWave) + threadIdx.x;
    const int t = i / quads, n = (i - t * quads) * 4; // (H is a multiple of 256: a wave has one token)
    if (t >= a.T)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int mine = lane < a.k ? slot_expert(a, t * a.k + lane) : -1;
    const float w = mine >= 0 ? a.topk_w[t * a.k + lane] : 0.f;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    bool first = true;
    uint64_t local = __ballot(mine >= 0);
    const float *y = a.y + static_cast<int64_t>(t) * a.k * a.H + n;
    while (local) {
        constexpr int kBatch = 8;
        f32x4 v[kBatch];
        int slot[kBatch];
        int count = 0;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            slot[b] = local ? __builtin_ctzll(local) : slot[0]; // (no more: the first one again, unused)
            count += local != 0;
            local &= local - 1;
            v[b] = *reinterpret_cast<const f32x4 *>(y + static_cast<int64_t>(slot[b]) * a.H);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), slot[b]));
            if (b < count) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sum[q] = first ? v[b][q] * f : fmaf(v[b][q], f, sum[q]);
                first = false;
            }
        }
    }
    *reinterpret_cast<u32x2 *>(a.out + static_cast<int64_t>(t) * a.H + n) =
        u32x2{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
template <int FMT>
static hipError_t launch_layer_of(const LayerArgs &a, hipStream_t s)
{
    const dim3 blk(kLayerWaves * kWave);
    if (layer_singles(a.slots, a.E, FMT)) {
        launch(k_layer_up_slots<FMT>, dim3(a.slots * (a.I / (kLayerWaves * kLayerUpCols)) + (a.flags ? 1 : 0)), blk, 0,
               s, a);
        launch(k_layer_down_slots<FMT>, dim3(a.T * (a.H / (kLayerWaves * kLayerDownCols))), blk, 0, s, a);
        return hipGetLastError();
    }
    const int64_t items = layer_items(a.slots, a.EL);
    const int64_t up = items * (a.I / 64), down = items * (a.H / 128), most = 2 * kCus;
    launch(k_layer_ring<FMT, true>, dim3(static_cast<unsigned>(up < most ? up : most) + (a.flags ? 1 : 0)), blk,
           LayerRing<FMT, true>::kBytes, s, a);
    launch(k_layer_ring<FMT, false>, dim3(static_cast<unsigned>(down < most ? down : most)), blk,
           LayerRing<FMT, false>::kBytes, s, a);
    launch(k_layer_sum, dim3((a.T * (a.H / 4) + kLayerWaves * kWave - 1) / (kLayerWaves * kWave)), blk, 0, s, a);
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
