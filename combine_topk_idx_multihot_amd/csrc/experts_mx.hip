// experts_mx.hip -- the experts' products on MXFP4 rows of the expanded layout.
//
// Rows and weights are E2M1 codes, two a byte, with one E8M0 scale per 32
// columns (mx.h).  Row r of local expert e's group:
//   y[r,n] = sum over blocks b of 32 columns of
//            2^(sa[r,b] + sw[e,n,b] - 254) * (sum over k in b of a[r,k] * w[e,n,k])
// The f8f6f4 matrix instructions take both scales as operands, one byte per lane
// and 32 columns, so a product's accumulators run through all of K: nothing is
// left for the vector units.  Measured with chosen operands: the 4-bit products
// and their sums are exact within an instruction as far as 24 bits hold them, and
// an instruction's result is within 2^-22 of the sum of the magnitudes that enter
// it (the accumulator's among them), which is fp32 addition in some order.  A
// scale of 255 makes every result that it enters NaN, with codes of 0 too.
// Products are taken as w * a^T, as in experts.hip: a lane of an accumulator then
// holds one token row and runs of four consecutive output columns.
#include "expert_tiles.h"
#include "mx.h"

#include <type_traits>

namespace moe {

constexpr int kFp4 = 4; // the instructions' number for E2M1

__device__ __forceinline__ i32x8 widen(const u32x4 &v)
{
    return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
                 0, 0, 0, 0};
}

// silu(g) * u, with the reciprocal instruction (off by one step at most) for the
// division: a tile of 256 x 128 values takes 1.9 us less (of 24), and h is rounded to 8 or
// 2 bits next.
__device__ __forceinline__ float mx_gated(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// c + a * b^T over 128 columns: a and b hold 16 rows each, lane l the row l % 16
// and a block of 32 columns, sa and sb that block's scale in the lowest byte.
__device__ __forceinline__ f32x4 mfma_mx128(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, 0,
                                                            static_cast<int>(sa), 0, static_cast<int>(sb));
}

// The same over 64 columns of 32 rows each, lane l the row l % 32; the scales in
// byte B.
template <int B>
__device__ __forceinline__ f32x16 mfma_mx64(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb, const f32x16 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, kFp4, kFp4, B,
                                                           static_cast<int>(sa), B, static_cast<int>(sb));
}

// 8 values h (consecutive columns after the exchange below) to codes: the lane
// holds columns 4 u .. 4 u + 3 (lo) and 8 + 4 u .. (hi) of 16, u = lane / 32.
// Afterwards columns 8 u .. 8 u + 7.
__device__ __forceinline__ uint32_t mx_pack_eights(const f32x4 &lo, const f32x4 &hi, uint32_t b)
{
    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    const uint32_t q = mx_pack8(x, b);
    uint32_t first = q & 0xFFFFu, last = q >> 16;
    whole_eights(first, last);
    return first | (last << 16);
}

// ---------------------------------------------------------------------------
// Products of a few tokens: a workgroup takes 32 output columns (gated: 32 gate
// and the 32 up columns, one block of outputs) of one expert that has rows, its
// waves every kSplit-th step of 128 columns, from HBM to registers; the waves'
// sums are added in the order of the waves through LDS.  16 rows at a time; more
// rows read the weights again, from L2.
// Top-8 of 128, one token, K = 768, N = 2048: 5.4 us, 6.7 MB, so launch, a first load and
// the stores are what it takes.
// ---------------------------------------------------------------------------
constexpr int kMxSplit = 4;
constexpr int kMxCols = 32;
constexpr int kMxAhead = 4; // steps whose loads a wave has in flight

template <bool GATED, bool MX>
__global__ void __launch_bounds__(kMxSplit * kWave) k_expert_mx_rows(MxExpertArgs a)
{
    constexpr int W = GATED ? 4 : 2; // runs of 16 weight rows
    __shared__ f32x4 part[kMxSplit - 1][W][kWave];
    flag_mismatch(a);
    const int slot = blockIdx.x / a.ntn, ni = blockIdx.x - slot * a.ntn;
    const int e = uniform(a.load.slots < a.EL ? nonempty_expert(a, slot) : slot);
    if (e < 0)
        return;
    const int64_t r0 = group_begin(a, e), r1 = group_begin(a, e + 1);
    if (r1 <= r0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    const int steps = a.K >> 7;
    const int row_bytes = a.K >> 1, row_blocks = a.K >> 5;
    const int n0 = ni * kMxCols;
    const uint8_t *__restrict__ w[W];
    const uint8_t *__restrict__ sw[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const int64_t row = GATED ? static_cast<int64_t>(e) * 2 * a.N + (j >> 1) * a.N + n0 + (j & 1) * 16 + l16
                                  : static_cast<int64_t>(e) * a.N + min(n0 + j * 16 + l16, a.N - 1);
        w[j] = a.w + row * row_bytes + quarter * 16;
        sw[j] = a.sw + row * row_blocks;
    }
    for (int64_t r = r0; r < r1; r += 16) {
        const int rows = static_cast<int>(min<int64_t>(16, r1 - r));
        const int64_t mine = r + min(l16, rows - 1);
        const uint8_t *__restrict__ x = a.a + mine * row_bytes + quarter * 16;
        const uint8_t *__restrict__ sx = a.sa + mine * row_blocks;
        f32x4 acc[W];
#pragma unroll
        for (int j = 0; j < W; ++j)
            acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int b0 = wave; b0 < steps; b0 += kMxSplit * kMxAhead) {
            u32x4 wf[kMxAhead][W], xf[kMxAhead];
            uint32_t ws[kMxAhead][W], xs[kMxAhead];
#pragma unroll
            for (int i = 0; i < kMxAhead; ++i) {
                const int b = min(b0 + i * kMxSplit, steps - 1); // (beyond the last step: unused)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    wf[i][j] = *reinterpret_cast<const u32x4 *>(w[j] + b * 64);
                    ws[i][j] = *reinterpret_cast<const uint32_t *>(sw[j] + b * 4);
                }
                xf[i] = *reinterpret_cast<const u32x4 *>(x + b * 64);
                xs[i] = *reinterpret_cast<const uint32_t *>(sx + b * 4);
            }
#pragma unroll
            for (int i = 0; i < kMxAhead; ++i) {
                if (b0 + i * kMxSplit < steps) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        acc[j] = mfma_mx128(wf[i][j], ws[i][j] >> (quarter * 8), xf[i], xs[i] >> (quarter * 8), acc[j]);
                }
            }
        }
        if (wave > 0) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                part[wave - 1][j][lane] = acc[j];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int p = 0; p < kMxSplit - 1; ++p)
                    acc[j] += part[p][j][lane];
            }
            // acc[j][i]: row r + l16, column n0 + 16 j + 4 quarter + i
            if constexpr (GATED) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[j][i] = mx_gated(acc[j][i], acc[j + 2][i]);
            }
            uint32_t b = 0;
            if constexpr (MX) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m = max(m, mag_bits(acc[j][i]));
                m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
                m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
                b = mx_scale(m);
                const float v[8] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3], acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
                const uint32_t q = mx_pack8(v, b);
                if (l16 < rows) {
                    uint16_t *o = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(a.out) + (r + l16) * (a.N >> 1) +
                                                               (n0 >> 1));
                    o[quarter] = static_cast<uint16_t>(q);
                    o[4 + quarter] = static_cast<uint16_t>(q >> 16);
                    if (quarter == 0)
                        a.out_scale[(r + l16) * (a.N >> 5) + ni] = static_cast<uint8_t>(b);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const u32x2 v = {pack_bf16(acc[j][0], acc[j][1]), pack_bf16(acc[j][2], acc[j][3])};
                    const int n = n0 + j * 16 + quarter * 4;
                    if (l16 < rows && n < a.N)
                        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + (r + l16) * a.N + n) = v;
                }
            }
        }
        if (r + 16 < r1)
            __syncthreads(); // the sums are read: room for the next rows'
    }
}

// ---------------------------------------------------------------------------
// Products with up to a few dozen rows per expert: the weights, read once, are
// all that counts.  Workgroups of four waves walk a list of tiles of 32 rows by
// 128 weight rows (gated: 64 gate and 64 up rows); their steps of 256 columns go
// through a ring of three stages in LDS, two steps, across tiles, on their way at
// any time.  A wave has 32 weight rows (gated: 16 gate and the 16 up rows of the
// same columns).
//
// A stage: 128 weight rows and 32 rows of 128 bytes (swizzled, place_of), then
// their scales, 8 bytes a row.  In a step the instruction i = 0 .. 3 takes chunk
// 4 (l / 32) + i of lane l's row, so that the four scales of a lane are one
// aligned word.  Where K is no multiple of 256 the last step has half as many
// columns: its upper chunks repeat the lower ones, and the lanes that use them take
// scales of 2^-127 on both sides: products below 2^-240, which vanish in fp32.
// Bound by HBM: gated with MXFP4 outputs, 333 tokens, 32 of 128 experts, K = 2048, N = 768 12.9
// us, 55 MB read (4.3 TB/s), matrix units busy 5 % of the cycles.
// ---------------------------------------------------------------------------
struct MxRingLds {
    static constexpr int kRows = kRingRows;
    static constexpr int kCols = 128; // weight rows
    static constexpr int kStages = 3;
    static constexpr uint32_t kX = kCols * 128;                  // in a stage: weight rows, rows,
    static constexpr uint32_t kSW = kX + kRows * 128;            // scales of the weight rows,
    static constexpr uint32_t kSX = kSW + kCols * 8;             // of the rows
    static constexpr uint32_t kStage = kSX + kRows * 8;
    static constexpr uint32_t kTop = kStages * kStage;           // gated: [wave][row] largest magnitudes
    static constexpr uint32_t kPre = kTop + 4 * kRows * 4;
    static constexpr uint32_t kOff = kPre + (kMaxLocal + 1) * 4;
    static constexpr uint32_t kBytes = kOff + (kMaxLocal + 1) * 4;
    static_assert(2 * (kBytes + 512) <= 160 * 1024, "two workgroups per CU");
};
constexpr int kMxRingWaves = 4;
constexpr int kMxRingLoads = 6; // loads of a wave per step; wave 0 has one more

typedef const __attribute__((address_space(3))) uint32_t *lds_word;

template <bool GATED, bool MX>
__global__ void __launch_bounds__(kMxRingWaves * kWave) k_expert_mx_ring(MxExpertArgs a)
{
    typedef MxRingLds L;
    constexpr int kOut = GATED ? 64 : 128; // output columns
    extern __shared__ uint8_t tile_lds[];  // from 0, and the kernel's only LDS
    flag_mismatch(a);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int l32 = lane & 31, upper = lane >> 5;
    if (wave == 0)
        tile_tables<L::kRows>(a, L::kPre, L::kOff);
    // (the compiler does not see the loads to LDS: the array's address escapes)
    asm volatile("" : : "v"(tile_lds) : "memory");
    __syncthreads();
    const int steps = (a.K + 255) >> 8;
    const bool half = a.K & 255; // the last step has 128 columns
    const uint32_t row_bytes = a.K >> 1, row_blocks = a.K >> 5;

    // ---- loads: the tile and step to send for, and where it goes
    TileList<L::kRows> ahead(a, L::kPre, L::kOff);
    Tile to = {0, 0, 0, 0};
    int to_b = steps, to_stage = 0;
    uint32_t woff[4], xoff = 0, wrow = 0; // rows' byte offsets; this lane's weight row for scales
    uint32_t xrow = 0;
    const uint8_t *wbase = nullptr, *xbase = nullptr, *swbase = nullptr, *sxbase = nullptr;
    const auto send = [&]() {
        if (to.e < 0)
            return;
        if (to_b == steps) {
            to = ahead.next(a);
            if (to.e < 0)
                return;
            to_b = 0;
            // weight row j of the tile: gated, waves 0 and 1 the gate rows, 2 and 3 the up rows
            const int64_t first = static_cast<int64_t>(to.e) * (GATED ? 2 * a.N : a.N) +
                                  static_cast<int64_t>(to.ni) * kOut + (GATED && wave >= 2 ? a.N : 0);
            const int last = GATED ? 63 : a.N - 1 - to.ni * kOut;
            const int base = GATED ? (wave & 1) * 32 : wave * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                woff[i] = min(base + i * 8 + (lane >> 3), last) * row_bytes;
            wrow = min(base + (lane >> 1), last) * row_blocks;
            xoff = min(wave * 8 + (lane >> 3), to.rows - 1) * row_bytes;
            xrow = min(lane >> 1, to.rows - 1) * row_blocks;
            wbase = a.w + first * row_bytes;
            swbase = a.sw + first * row_blocks;
            xbase = a.a + to.r0 * row_bytes;
            sxbase = a.sa + to.r0 * row_blocks;
        }
        const bool cut = half && to_b + 1 == steps;
        const uint32_t at = uniform(to_stage) * L::kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int c = place_of(wave * 32 + i * 8 + (lane >> 3), lane & 7);
            c = cut ? c & 3 : c;
            lds_load16(at + (wave * 4 + i) * 1024, wbase + to_b * 128 + (woff[i] + c * 16));
        }
        int c = place_of(wave * 8 + (lane >> 3), lane & 7);
        c = cut ? c & 3 : c;
        lds_load16(at + L::kX + wave * 1024, xbase + to_b * 128 + (xoff + c * 16));
        const uint32_t word = cut ? 0 : (lane & 1) * 4;
        lds_load4(at + L::kSW + wave * 256, swbase + to_b * 8 + (wrow + word));
        if (wave == 0)
            lds_load4(at + L::kSX, sxbase + to_b * 8 + (xrow + word));
        ++to_b;
        to_stage = to_stage + 1 == L::kStages ? 0 : to_stage + 1;
    };
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i)
        send();

    // ---- products
    TileList<L::kRows> list(a, L::kPre, L::kOff);
    const int mine = GATED ? (l32 < 16 ? wave * 16 + l32 : 64 + wave * 16 + l32 - 16) : wave * 32 + l32;
    int stage = 0;
    for (Tile t = list.next(a); t.e >= 0; t = list.next(a)) {
        f32x16 acc = f32x16{};
        for (int b = 0; b < steps; ++b) {
            // this step's loads are there: the next step's are newer
            if (to.e < 0)
                step_barrier<0>();
            else if (wave == 0)
                step_barrier<(L::kStages - 2) * (kMxRingLoads + 1)>();
            else
                step_barrier<(L::kStages - 2) * kMxRingLoads>();
            send(); // over the stage before, which every wave is done with
            const uint32_t at = stage * L::kStage;
            const bool cut = half && b + 1 == steps;
            u32x4 wf[4], xf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wf[i] = *lds_at<lds_chunk>(at + mine * 128 + place_of(mine, upper * 4 + i) * 16);
                xf[i] = *lds_at<lds_chunk>(at + L::kX + l32 * 128 + place_of(l32, upper * 4 + i) * 16);
            }
            uint32_t ws = *lds_at<lds_word>(at + L::kSW + mine * 8 + upper * 4);
            uint32_t xs = *lds_at<lds_word>(at + L::kSX + l32 * 8 + upper * 4);
            if (cut && upper)
                ws = xs = 0;
            acc = mfma_mx64<0>(wf[0], ws, xf[0], xs, acc);
            acc = mfma_mx64<1>(wf[1], ws, xf[1], xs, acc);
            acc = mfma_mx64<2>(wf[2], ws, xf[2], xs, acc);
            acc = mfma_mx64<3>(wf[3], ws, xf[3], xs, acc);
            stage = stage + 1 == L::kStages ? 0 : stage + 1;
        }
        const int64_t r = t.r0 + l32;
        const bool in = l32 < t.rows;
        if constexpr (!GATED) {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const int n = t.ni * kOut + wave * 32 + g * 8 + upper * 8;
                const u32x4 v = pack_eights(acc, g);
                if (in && n < a.N)
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + r * a.N + n) = v;
            }
            continue;
        }
        // h in place of the gate: the first 8 elements
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = mx_gated(acc[i], acc[8 + i]);
        const int n = t.ni * kOut + wave * 16 + upper * 8;
        if constexpr (MX) {
            // two waves share a block of 32 columns
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max(m, mag_bits(acc[i]));
            m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
            if (upper == 0)
                *lds_at<lds_int>(L::kTop + (wave * L::kRows + l32) * 4) = static_cast<int>(m);
            lds_barrier();
            m = max(m, static_cast<uint32_t>(*lds_at<lds_int>(L::kTop + ((wave ^ 1) * L::kRows + l32) * 4)));
            const uint32_t b = mx_scale(m);
            const uint32_t q = mx_pack_eights(f32x4{acc[0], acc[1], acc[2], acc[3]},
                                              f32x4{acc[4], acc[5], acc[6], acc[7]}, b);
            if (in)
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.out) + r * (a.N >> 1) + (n >> 1)) = q;
            if (in && (wave & 1) == 0 && upper == 0)
                a.out_scale[r * (a.N >> 5) + (n >> 5)] = static_cast<uint8_t>(b);
        } else {
            const u32x4 v = pack_eights(acc, 0);
            if (in)
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + r * a.N + n) = v;
        }
    }
    // no load to LDS may be left when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// ---------------------------------------------------------------------------
// Products with many rows per expert: workgroups of four waves, one per CU and one
// wave per SIMD, each taking tiles of up to 256 rows by 256 weight rows (gated: 128
// gate and 128 up rows) one after the other.  A wave has half of the rows (32 of
// each block of 64) and 128 weight rows: 16 accumulators of 32 x 32, which is what
// its 512 registers hold, and the fewest LDS reads per product.  Rows, weights and
// their scales come through LDS 256 columns (a step) at a time, in two stages: while
// a step is worked on, the next one's data, or the first step's of the next tile, is
// on its way.
//
// Per step and CU 256 32x32x64 instructions (33.6 Mflop), 68 KB into LDS and 132 KB
// out of it.  16384 tokens, top-8 of 128, K = 2048, N = 4096: 793 us, 2.77 PFLOP/s at 1.87 GHz;
// a step takes 4400 cycles, 2100 of them the matrix instructions' own; without its loads
// to LDS it takes 3470, without its LDS reads 4270.  Beside its steps a tile takes about 5 us
// (conversion and stores), as much as two steps.  Gated with MXFP4 outputs, 4096 tokens, N =
// 768: 115 to 125 us, 1.65 to 1.8 PFLOP/s.
// ---------------------------------------------------------------------------
constexpr int kMxTileWaves = 4;
constexpr int kMxTileRows = 256;

struct MxTileLds {
    static constexpr uint32_t kX = kTileCols * 128;  // in a stage: weight rows, rows,
    static constexpr uint32_t kSW = kX + kMxTileRows * 128; // scales of the weight rows,
    static constexpr uint32_t kSX = kSW + kTileCols * 8;    // of the rows
    static constexpr uint32_t kStage = kSX + kMxTileRows * 8;
    static constexpr uint32_t kPre = 2 * kStage;
    static constexpr uint32_t kOff = kPre + (kMaxLocal + 1) * 4;
    static constexpr uint32_t kBytes = kOff + (kMaxLocal + 1) * 4;
    static_assert(kBytes <= 160 * 1024, "LDS of a CU");
};

// Where a wave's loads of a tile come from: 8 rows each, lane l's row l / 8 and the
// chunk that belongs at place l % 8; scales 32 rows each, two words a row.
struct MxAim {
    const uint8_t *w, *x, *sw, *sx;
    uint32_t woff[8], xoff[8]; // byte offsets of rows and chunks
    uint32_t wrow[2], xrow[2]; // of rows' scales
};

template <bool GATED>
__device__ __forceinline__ void mx_aim(const MxExpertArgs &a, const Tile &t, MxAim &m)
{
    constexpr int kOut = GATED ? 128 : kTileCols;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const uint32_t row_bytes = a.K >> 1, row_blocks = a.K >> 5;
    // gated: waves 0 and 1 bring the gate rows, 2 and 3 the up rows
    const int64_t first = static_cast<int64_t>(t.e) * (GATED ? 2 * a.N : a.N) +
                          static_cast<int64_t>(t.ni) * kOut + (GATED && wave >= 2 ? a.N : 0);
    const int base = GATED ? (wave & 1) * 64 : wave * 64;
    const int last = GATED ? 127 : a.N - 1 - t.ni * kOut;
    m.w = a.w + first * row_bytes;
    m.sw = a.sw + first * row_blocks;
    m.x = a.a + t.r0 * row_bytes;
    m.sx = a.sa + t.r0 * row_blocks;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (a row's place depends on its number modulo 16 only)
        m.woff[i] = min(base + i * 8 + (lane >> 3), last) * row_bytes + place_of(i * 8 + (lane >> 3), lane & 7) * 16;
        // load i of the rows: rows 32 i + 8 wave .. + 7, so that fewer blocks of 64 rows take
        // fewer loads
        m.xoff[i] = min(i * 32 + wave * 8 + (lane >> 3), t.rows - 1) * row_bytes +
                    place_of(wave * 8 + (lane >> 3), lane & 7) * 16;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m.wrow[i] = min(base + i * 32 + (lane >> 1), last) * row_blocks;
        m.xrow[i] = min(i * 128 + wave * 32 + (lane >> 1), t.rows - 1) * row_blocks;
    }
}

// Load p (0 .. kMxSends - 1) of step b, for M blocks of 64 rows, to the stage at `at`:
// first the weights' and rows' scales, two each, then weights and rows in turn, eight
// each.  cut: the step has 128 columns, its upper chunks repeat the lower ones.
constexpr int kMxSends = 20;
constexpr int kMxSends0 = 12; // of them in the first round

template <int M>
__device__ __forceinline__ void mx_send(const MxAim &m, int p, int b, bool cut, uint32_t at)
{
    typedef MxTileLds L;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    at = uniform(at);
    if (p < 4) {
        const int i = p >> 1;
        const uint32_t word = cut ? 0 : (lane & 1) * 4;
        if ((p & 1) == 0)
            lds_load4(at + L::kSW + (wave * 2 + i) * 256, m.sw + b * 8 + (m.wrow[i] + word));
        else if (i * 128 < 64 * M) // (of blocks of 128 rows: more than needed where M is odd)
            lds_load4(at + L::kSX + (i * 4 + wave) * 256, m.sx + b * 8 + (m.xrow[i] + word));
        return;
    }
    const int i = (p - 4) >> 1;
    if ((p & 1) == 0) {
        const uint32_t back = cut ? (place_of(i * 8 + (lane >> 3), lane & 7) & 4) * 16 : 0;
        lds_load16(at + (wave * 8 + i) * 1024, m.w + b * 128 + (m.woff[i] - back));
    } else if (i < 2 * M) {
        const uint32_t back = cut ? (place_of(wave * 8 + (lane >> 3), lane & 7) & 4) * 16 : 0;
        lds_load16(at + L::kX + (i * 4 + wave) * 1024, m.x + b * 128 + (m.xoff[i] - back));
    }
}

// One tile with M blocks of 64 rows, whose first step has been sent for; sends for
// the first one of `next` during the last step.  `keep`: vector memory accesses (the
// last tile's stores) newer than that, which may be on their way at the start.
// Returns the same for the next tile.
template <int M, bool GATED, bool MX>
__device__ __forceinline__ int mx_tile_run(const MxExpertArgs &a, const Tile &t, const Tile &next, MxAim &aim,
                                           uint32_t &stage, int keep)
{
    typedef MxTileLds L;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave >> 1, wn = wave & 1;
    const int l32 = lane & 31, upper = lane >> 5;
    const int steps = (a.K + 255) >> 8;
    const bool half = a.K & 255;
    const int xrow = wm * 32 + l32; // + 64 m
    // weight row of run j: plain, 32 j of this wave's 128; gated, runs 0 and 1 gate rows, 2 and 3
    // the up rows of the same columns
    const int wrow = (GATED ? wn * 64 : wn * 128) + l32;
    constexpr int kRun2 = (GATED ? 128 : 64) * 128; // from runs 0 and 1 to 2 and 3
    uint32_t wad[4], xad[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        wad[i] = wrow * 128 + place_of(wrow, upper * 4 + i) * 16;
        xad[i] = L::kX + xrow * 128 + place_of(xrow, upper * 4 + i) * 16;
    }
    const uint32_t wsad = L::kSW + wrow * 8 + upper * 4, xsad = L::kSX + xrow * 8 + upper * 4;
    f32x16 acc[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[m][j] = f32x16{};
    // A step: four rounds of 4 M matrix instructions, one chunk of every row each.  What the
    // next round and the next step need is read and sent for one piece at a time behind the
    // instructions, in exactly this order: a wave is alone on its SIMD, and whatever it issues
    // in a run of its own leaves the matrix unit idle (with all reads and loads of a round ahead
    // of its instructions a step took twice the time).
    // SM: the blocks of rows to send for, at most.
    const auto step = [&](auto smc, int bn, bool cut, bool cut_next) {
        constexpr int SM = decltype(smc)::value;
        // this step's data is there, the other stage is free
        if (keep >= 32)
            step_barrier<32>();
        else if (keep >= 16)
            step_barrier<16>();
        else if (keep >= 8)
            step_barrier<8>();
        else if (keep >= 4)
            step_barrier<4>();
        else
            step_barrier<0>();
        keep = 0;
        const uint32_t at = stage, to = L::kStage - stage;
        uint32_t ws[4], xs[M];
        u32x4 w[2][4], x[2][M];
        const auto read = [&](int k, int i) { // runs of weights, then blocks of rows
            if (i < 4)
                w[k & 1][i] = *lds_at<lds_chunk>(at + wad[k] + (i & 1) * 4096 + (i >> 1) * kRun2);
            else
                x[k & 1][i - 4] = *lds_at<lds_chunk>(at + xad[k] + (i - 4) * 8192);
        };
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ws[j] = *lds_at<lds_word>(at + wsad + (j & 1) * 256 + (j >> 1) * (kRun2 / 16));
#pragma unroll
        for (int m = 0; m < M; ++m)
            xs[m] = *lds_at<lds_word>(at + xsad + m * 512);
        read(0, 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            read(0, i);
#pragma unroll
        for (int i = 5; i < 4 + M; ++i)
            read(0, i);
        if (cut && upper) { // scales of 2^-127 on both sides: products that vanish beside any other
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ws[j] = 0;
#pragma unroll
            for (int m = 0; m < M; ++m)
                xs[m] = 0;
        }
        __builtin_amdgcn_sched_barrier(0);
        const auto round = [&](auto kc) {
            constexpr int k = decltype(kc)::value;
            // the sends early, as the next step waits for them
            constexpr int kReads = k < 3 ? 4 + M : 0, kSends = k == 0 ? kMxSends0 : k == 1 ? kMxSends - kMxSends0 : 0;
            constexpr int kPieces = kReads + kSends > 0 ? kReads + kSends : 1, kSend0 = k == 0 ? 0 : kMxSends0;
#pragma unroll
            for (int q = 0; q < 4 * M; ++q) {
                acc[q / 4][q % 4] = mfma_mx64<k>(w[k & 1][q % 4], ws[q % 4], x[k & 1][q / 4], xs[q / 4],
                                                 acc[q / 4][q % 4]);
#pragma unroll
                for (int p = q * kPieces / (4 * M); p < (q + 1) * kPieces / (4 * M) && p < kReads + kSends; ++p) {
                    // (in turn, as many of each as there are)
                    const int r = p * kReads / kPieces, r1 = (p + 1) * kReads / kPieces;
                    if (r1 > r)
                        read(k + 1, r);
                    else
                        mx_send<SM>(aim, kSend0 + p - r, bn, cut_next, to);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        round(std::integral_constant<int, 0>{});
        round(std::integral_constant<int, 1>{});
        round(std::integral_constant<int, 2>{});
        round(std::integral_constant<int, 3>{});
        stage = to;
    };
    for (int b = 0; b + 1 < steps; ++b)
        step(std::integral_constant<int, M>{}, b + 1, false, half && b + 2 == steps);
    // (without a next tile: this one's last step again, unused)
    if (next.e >= 0)
        mx_aim<GATED>(a, next, aim);
    step(std::integral_constant<int, 4>{}, next.e >= 0 ? 0 : steps - 1, half, half && (next.e < 0 || steps == 1));
    // accumulator element i of a lane: weight row 8 (i / 4) + 4 upper + i % 4
    if constexpr (!GATED) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                // as in k_expert_tile: four lanes trade, so that a store writes whole cache lines
                u32x4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] = pack_eights(acc[m][2 * p + (c >> 1)], (c & 1) * 2);
                trade<1>(v[0], v[1]);
                trade<1>(v[2], v[3]);
                trade<2>(v[0], v[2]);
                trade<2>(v[1], v[3]);
                const int row = 64 * m + (xrow & ~3);
                const int n = t.ni * kTileCols + wn * 128 + p * 64 + (lane & 3) * 16 + upper * 8;
                uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N + n;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row + i < t.rows && n < a.N)
                        *reinterpret_cast<u32x4 *>(o + static_cast<int64_t>(i) * a.N) = v[i];
            }
        }
    } else {
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[m][j][i] = mx_gated(acc[m][j][i], acc[m][j + 2][i]);
            if constexpr (MX) {
                const int row = 64 * m + xrow;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // a block of 32 columns is the 16 values of this lane and of lane ^ 32
                    const f32x16 &h = acc[m][j];
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        top = max(top, mag_bits(h[i]));
                    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
                    const uint32_t sc = mx_scale(top);
                    uint32_t lo = mx_pack_eights(f32x4{h[0], h[1], h[2], h[3]}, f32x4{h[4], h[5], h[6], h[7]}, sc);
                    uint32_t hi = mx_pack_eights(f32x4{h[8], h[9], h[10], h[11]}, f32x4{h[12], h[13], h[14], h[15]}, sc);
                    whole_eights(lo, hi); // 16 columns per lane
                    const int n = t.ni * 128 + wn * 64 + j * 32;
                    if (row < t.rows) {
                        *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + (t.r0 + row) * (a.N >> 1) + (n >> 1) +
                                                   upper * 8) = u32x2{lo, hi};
                        if (upper == 0)
                            a.out_scale[(t.r0 + row) * (a.N >> 5) + (n >> 5)] = static_cast<uint8_t>(sc);
                    }
                }
            } else {
                u32x4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] = pack_eights(acc[m][c >> 1], (c & 1) * 2);
                trade<1>(v[0], v[1]);
                trade<1>(v[2], v[3]);
                trade<2>(v[0], v[2]);
                trade<2>(v[1], v[3]);
                const int row = 64 * m + (xrow & ~3);
                uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N + t.ni * 128 + wn * 64 +
                              (lane & 3) * 16 + upper * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row + i < t.rows)
                        *reinterpret_cast<u32x4 *>(o + static_cast<int64_t>(i) * a.N) = v[i];
            }
        }
    }
    // (the waits above count on every one of a whole tile's stores)
    const bool all = t.rows == 64 * M && (GATED || (t.ni + 1) * kTileCols <= a.N);
    return all ? (GATED ? 4 * M : 8 * M) : 0;
}

template <bool GATED, bool MX>
__global__ void __launch_bounds__(kMxTileWaves * kWave) __attribute__((amdgpu_waves_per_eu(1, 1)))
k_expert_mx_tile(MxExpertArgs a)
{
    typedef MxTileLds L;
    extern __shared__ uint8_t tile_lds[]; // all of it by address, from 0
    flag_mismatch(a);
    if (uniform(threadIdx.x / kWave) == 0)
        tile_tables<kMxTileRows>(a, L::kPre, L::kOff);
    asm volatile("" : : "v"(tile_lds) : "memory"); // (as in k_expert_tile)
    __syncthreads();
    TileList<kMxTileRows> list(a, L::kPre, L::kOff);
    Tile t = list.next(a);
    if (t.e < 0)
        return;
    MxAim aim;
    uint32_t stage = 0;
    int keep = 0;
    mx_aim<GATED>(a, t, aim);
#pragma unroll
    for (int p = 0; p < kMxSends; ++p)
        mx_send<4>(aim, p, 0, a.K < 256, 0);
    while (t.e >= 0) {
        const Tile next = list.next(a);
        switch ((t.rows + 63) >> 6) {
        case 1: keep = mx_tile_run<1, GATED, MX>(a, t, next, aim, stage, keep); break;
        case 2: keep = mx_tile_run<2, GATED, MX>(a, t, next, aim, stage, keep); break;
        case 3: keep = mx_tile_run<3, GATED, MX>(a, t, next, aim, stage, keep); break;
        default: keep = mx_tile_run<4, GATED, MX>(a, t, next, aim, stage, keep); break;
        }
        t = next;
    }
    // no load to LDS may be left when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
static hipError_t launch_mx_rows(MxExpertArgs &a, hipStream_t s)
{
    a.ntn = (a.N + kMxCols - 1) / kMxCols;
    const int64_t nb = a.load.slots * a.ntn;
    if (nb > 0xFFFFFFFFll / (kMxSplit * kWave))
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb)), blk(kMxSplit * kWave);
    if (!a.gated)
        launch(k_expert_mx_rows<false, false>, g, blk, 0, s, a);
    else if (a.out_scale)
        launch(k_expert_mx_rows<true, true>, g, blk, 0, s, a);
    else
        launch(k_expert_mx_rows<true, false>, g, blk, 0, s, a);
    return hipGetLastError();
}

static hipError_t launch_mx_ring(MxExpertArgs &a, hipStream_t s)
{
    const int cols = a.gated ? 64 : 128;
    a.ntn = (a.N + cols - 1) / cols;
    const int64_t nb = tiles_max(a, MxRingLds::kRows);
    if (nb > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb < 2 * kCus ? nb : 2 * kCus)), blk(kMxRingWaves * kWave);
    if (!a.gated)
        launch(k_expert_mx_ring<false, false>, g, blk, MxRingLds::kBytes, s, a);
    else if (a.out_scale)
        launch(k_expert_mx_ring<true, true>, g, blk, MxRingLds::kBytes, s, a);
    else
        launch(k_expert_mx_ring<true, false>, g, blk, MxRingLds::kBytes, s, a);
    return hipGetLastError();
}

static hipError_t launch_mx_tile(MxExpertArgs &a, hipStream_t s)
{
    const int cols = a.gated ? 128 : kTileCols;
    a.ntn = (a.N + cols - 1) / cols;
    const int64_t nb = tiles_max(a, kMxTileRows);
    if (nb > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb < kCus ? nb : kCus)), blk(kMxTileWaves * kWave);
    if (!a.gated)
        launch(k_expert_mx_tile<false, false>, g, blk, MxTileLds::kBytes, s, a);
    else if (a.out_scale)
        launch(k_expert_mx_tile<true, true>, g, blk, MxTileLds::kBytes, s, a);
    else
        launch(k_expert_mx_tile<true, false>, g, blk, MxTileLds::kBytes, s, a);
    return hipGetLastError();
}

hipError_t launch_expert_product_mx(const MxExpertArgs &a0, hipStream_t s)
{
    MxExpertArgs a = a0;
    switch (choose_mx_kernel(a.load, a.N, a.gated != 0)) {
    case ExpertKernel::rows: return launch_mx_rows(a, s);
    case ExpertKernel::ring: return launch_mx_ring(a, s);
    default: return launch_mx_tile(a, s);
    }
}

}  // namespace moe
