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

namespace moe {

constexpr int kFp4 = 4; // the instructions' number for E2M1

__device__ __forceinline__ i32x8 widen(const u32x4 &v)
{
    return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
                 0, 0, 0, 0};
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
                        acc[j][i] = gated(acc[j][i], acc[j + 2][i]);
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
// columns: its upper chunks repeat the lower ones, and the lanes that would use
// them put zeros in place of the weights.
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
            const uint32_t ws = *lds_at<lds_word>(at + L::kSW + mine * 8 + upper * 4);
            const uint32_t xs = *lds_at<lds_word>(at + L::kSX + l32 * 8 + upper * 4);
            if (cut && upper) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    wf[i] = u32x4{0u, 0u, 0u, 0u};
            }
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
            acc[i] = gated(acc[i], acc[8 + i]);
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

hipError_t launch_expert_product_mx(const MxExpertArgs &a0, hipStream_t s)
{
    MxExpertArgs a = a0;
    if (choose_mx_kernel(a.load, a.K, a.N, a.gated != 0) == ExpertKernel::rows)
        return launch_mx_rows(a, s);
    return launch_mx_ring(a, s);
}

}  // namespace moe
