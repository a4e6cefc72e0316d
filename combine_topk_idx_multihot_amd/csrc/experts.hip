// experts.hip -- the experts' products on FP8 rows of the expanded layout.
//
// Rows are E4M3 codes with one fp32 scale per 128 columns (the FP8 dispatch's
// output), weights E4M3 codes [EL,N,K] with one fp32 scale per 128 x 128
// block.  Row r of local expert e's group:
//   y[r,n] = sum over blocks b of 128 columns of
//            sa[r,b] * sw[e, n / 128, b] * (sum over k in b of a[r,k] * w[e,n,k])
// The inner sum is one matrix instruction of depth 128 or two of depth 64
// (gfx950's f8f6f4 forms, whose 8-bit rate is twice that of the older 8-bit
// instructions); the two scales are multiplied in fp32 and the block's sum
// enters the fp32 accumulator by one fma.
// What the 8-bit matrix instructions sum, measured on MI355X with chosen
// operands: products are exact, groups of 8 consecutive columns are aligned to
// the group's largest exponent sum E and cut off below 2^(E-13), and the
// groups are added in fp32.  On normal data that is 1.5e-5 of the result in
// norm (6e-5 on heavy tails), a hundredth of the bf16 output's rounding; the
// older 8-bit instructions do the same, and bf16 instructions on widened
// codes, which are exact to fp32, run at half the rate.  Outputs are therefore
// bf16 (or E4M3), not fp32.  Where it shows: a few outputs round the other way.
// bf16 outputs differ from those of fp32 sums by 2.5e-4 in norm (0.0017 from 64
// bits on either side), values of requantized E4M3 outputs by 6e-4 to 1.6e-3
// (0.0022 - 0.0028 from 64 bits; with fp32 sums 0.0021 - 0.0024).
// Products are taken as w * a^T: a lane of an accumulator then holds one token
// row and runs of four consecutive output columns, so that its row scale is a
// single register and its outputs are stored together.
//
// Three kernels, chosen by choose_expert_kernel: k_expert_rows (a few tokens),
// k_expert_ring (up to dozens of rows per expert) and k_expert_tile.
#include "moe_internal.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 1e-4f;

// Two fp32 values to bf16, nearest-even, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y)
{
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ i32x8 join(const u32x4 &lo, const u32x4 &hi)
{
    i32x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = static_cast<int>(lo[i]);
        v[4 + i] = static_cast<int>(hi[i]);
    }
    return v;
}

// The tile of rows and output columns that a workgroup computes.
struct Tile {
    int e;       // local expert, -1: no tile
    int64_t r0;  // first row
    int rows;    // 1 .. BM
    int ni;      // column tile
};

__device__ __forceinline__ int64_t group_begin(const ExpertArgs &a, int e)
{
    return max<int64_t>(0, min<int64_t>(a.off[e], a.R));
}

__device__ __forceinline__ void flag_mismatch(const ExpertArgs &a)
{
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.eager && a.status[0] != a.R)
        atomicOr(&a.status[1], 4);
}

// silu(g) * u
__device__ __forceinline__ float gated(float g, float u)
{
    return g / (1.0f + __expf(-g)) * u;
}

// Into [-448, 448]; a NaN stays one (and becomes the NaN code).
__device__ __forceinline__ float clamp_e4m3(float y)
{
    return fabsf(y) > kE4M3Max ? copysignf(kE4M3Max, y) : y;
}

// Four E4M3 codes of h * inv, nearest-even.
__device__ __forceinline__ int pack_e4m3(const f32x4 &h, float inv)
{
    const int q = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(h[0] * inv), clamp_e4m3(h[1] * inv), 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(h[2] * inv), clamp_e4m3(h[3] * inv), q, true);
}

// ---------------------------------------------------------------------------
// Products of a few tokens: a workgroup takes 32 output columns of one expert
// that has rows, each of its kSplit waves every kSplit-th step of 128 columns,
// from HBM to registers; the waves' sums are added in the order of the waves
// through LDS.  16 rows at a time; more rows read the weights again, from L2.
// What counts here is the time from the launch to the first and from the last
// load, not their rate: 4.2 MB of weights in K = 512 columns each take 4.6 us,
// where the kernels below, which first list their tiles, take 13.
// ---------------------------------------------------------------------------
constexpr int kSplit = 4;
constexpr int kRowsCols = 32;

// c + a * b^T over 128 columns: a and b hold 16 rows each, lane l the row
// l % 16 and a quarter of its columns (any quarter, the same one in both).
__device__ __forceinline__ f32x4 mfma128(const i32x8 &a, const i32x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// A lane's quarter of 128 columns at p: 16 bytes of each 64-byte half, so that
// the four lanes of a row read 64 bytes together (a load's cost goes with the
// cache lines that it touches).
__device__ __forceinline__ i32x8 load_quarter(const uint8_t *p, int quarter)
{
    return join(*reinterpret_cast<const u32x4 *>(p + quarter * 16),
                *reinterpret_cast<const u32x4 *>(p + 64 + quarter * 16));
}

// The local expert of the s-th group that has rows, -1 if there are not so many.
__device__ __forceinline__ int nonempty_expert(const ExpertArgs &a, int s)
{
    const int lane = threadIdx.x & (kWave - 1);
    for (int base = 0; base < a.EL; base += kWave) {
        const int e = base + lane;
        const bool some = e < a.EL && group_begin(a, e + 1) > group_begin(a, e);
        const uint64_t m = __ballot(some);
        const int n = __popcll(m);
        if (s < n) {
            const int rank = __popcll(m & ((1ull << lane) - 1));
            return base + __builtin_ctzll(__ballot(some && rank == s));
        }
        s -= n;
    }
    return -1;
}

__global__ void __launch_bounds__(kSplit * kWave) k_expert_rows(ExpertArgs a)
{
    __shared__ f32x4 part[kSplit - 1][2][kWave];
    flag_mismatch(a);
    const int slot = blockIdx.x / a.ntn, ni = blockIdx.x - slot * a.ntn;
    // as many slots as experts, or as groups where those are fewer
    const int e = __builtin_amdgcn_readfirstlane(a.load.slots < a.EL ? nonempty_expert(a, slot) : slot);
    if (e < 0)
        return;
    const int64_t r0 = group_begin(a, e), r1 = group_begin(a, e + 1);
    if (r1 <= r0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, quarter = lane >> 4;
    const int KB = a.K >> 7;
    const int n0 = ni * kRowsCols;
    const uint8_t *__restrict__ w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = a.w + (static_cast<int64_t>(e) * a.N + min(n0 + j * 16 + l16, a.N - 1)) * a.K;
    const float *__restrict__ sw = a.sw + (static_cast<int64_t>(e) * a.NB + (n0 >> 7)) * KB;
    for (int64_t r = r0; r < r1; r += 16) {
        const int rows = static_cast<int>(min<int64_t>(16, r1 - r));
        const int64_t mine = r + min(l16, rows - 1);
        const uint8_t *__restrict__ x = a.a + mine * a.K;
        const float *__restrict__ sx = a.sa + mine * KB;
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        for (int b = wave; b < KB; b += kSplit) {
            i32x8 wf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                wf[j] = load_quarter(w[j] + b * 128, quarter);
            const i32x8 xf = load_quarter(x + b * 128, quarter);
            const float f = sx[b] * sw[b];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x4 q = mfma128(wf[j], xf, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = fmaf(q[i], f, acc[j][i]);
            }
        }
        if (wave > 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                part[wave - 1][j][lane] = acc[j];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int p = 0; p < kSplit - 1; ++p)
                    acc[j] += part[p][j][lane];
                const u32x2 v = {pack_bf16(acc[j][0], acc[j][1]), pack_bf16(acc[j][2], acc[j][3])};
                const int n = n0 + j * 16 + quarter * 4;
                if (l16 < rows && n < a.N)
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + (r + l16) * a.N + n) = v;
            }
        }
        if (r + 16 < r1)
            __syncthreads(); // the sums are read: room for the next rows'
    }
}

// ---------------------------------------------------------------------------
// Products with many rows per expert: workgroups of 8 waves, one per CU, each
// taking tiles of up to 256 rows by 256 output columns (gated: 128 gate and 128
// up columns) one after the other.  Rows and weights come through LDS 128
// columns (a step) at a time, in two stages: while a step is worked on, the
// next one's data, or the first step's of the next tile, is on its way.
//
// What bounds it: per step and CU 128 32x32x64 instructions (16.8 Mflop), 64 KB
// into LDS and 192 KB out of it, and 1024 wave fmas that bring the blocks' sums
// under their scales.  At 16384 tokens, top-8 of 128, K = 2048, N = 4096 the
// matrix units are busy for 50 % of the cycles, and the clock settles at 1.6 -
// 1.7 GHz instead of 2.4: the card's power limit, which also makes zeros 15 - 20 %
// faster than random codes.  There 1194 - 1271 us over runs and cards, 1.73 - 1.84
// PFLOP/s (a library's FP8 product without block scales: 2.62 at 8192^3, 3.19 at
// 16384^3), and 1.4 times the bytes that it needs.  4096 tokens, K = 768, N = 2048
// (256 rows per expert, 6 steps a tile): 110 - 115 us, 3.1 - 3.3 TB/s: what a step
// needs is sent in the step before and awaited at its end.  Gated: 4096 tokens, K =
// 2048, N = 768 184 - 191 us, 1.08 - 1.12 PFLOP/s; 16 of 128 experts, 16384 tokens, K
// = 4096, N = 1024 182 - 200 us, 1.38 - 1.51 PFLOP/s.
// At its 256 registers it spills 3 addresses (gated E4M3 12, gated bf16 15).  Before
// a reload is used the compiler waits for every load in flight: at the first
// scales of a tile, before the next tile's scales (gated), before the stores of
// codes (gated E4M3).
// Measured against it and dropped: 16x16x128 instructions (from registers alone
// 4.3 PFLOP/s, 32x32x64 5.0), two barriers per step with the waves in two groups
// (6 - 12 % slower), scales loaded with every step (0.2 - 0.3 us more per step of
// 2.0), tiles dealt by height for equal shares (the 16-expert case 5 % faster, the
// 16384-token one 6 % slower, as tiles of the same weights drift apart).
// ---------------------------------------------------------------------------
constexpr int kTileWaves = 8;
constexpr int kTileRows = 256;
constexpr int kTileBlocks = kTileRows / 64; // blocks of 64 rows, 32 per half of the waves
constexpr int kLoads = 8;                   // loads of a wave per step

// 16 or 4 bytes per lane from each lane's address to LDS, lane l's at `lds` +
// 16 l (4 l).  No register receives anything: the data is there once vmcnt says
// so.  Written as assembly because the compiler, given the builtin, waits for
// every such load before any LDS read that follows, those of the other stage
// among them.  The address is in vector registers and M0 is set here by a
// scalar move: a scalar base that a vector instruction has just written (a
// readfirstlane, a reload of a spilled one) would need five wait states before
// the load, which the compiler does not count for assembly.
__device__ __forceinline__ void lds_load16(uint32_t lds, const uint8_t *from)
{
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off"
                 : "={m0}"(m0)
                 : "s"(lds), "v"(from));
}
__device__ __forceinline__ void lds_load4(uint32_t lds, const void *from)
{
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off"
                 : "={m0}"(m0)
                 : "s"(lds), "v"(from));
}

// This wave's vector memory accesses are done, but for the newest KEEP, and so
// are its LDS accesses and those of every wave of the workgroup.
template <int KEEP>
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(KEEP) : "memory");
}
// The LDS accesses of every wave are done.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// A row of a stage in LDS is 128 bytes, eight 16-byte chunks.  Where row r keeps
// its chunk c, and which chunk is at place c: rows of one parity share their
// banks (64 of 4 bytes make two rows), and 16 consecutive rows read at one chunk
// then lie in different ones.  With r % 8 in place of (r / 2) % 8 conflicts were
// 53 % of the LDS cycles (16384 tokens, K = 2048, N = 4096; now 18 %) and the
// products 1 - 3 % slower.
__device__ __forceinline__ int place_of(int r, int c) { return c ^ ((r >> 1) & 7); }

// LDS of the tile kernel, from address 0: the loads to LDS take plain addresses
// and the two stages are told apart by one address bit.  Dynamic LDS starts
// there only in a kernel without static LDS, so neither this kernel nor the ring
// kernel may have a __shared__ of its own (the tests read that from the built
// code).
struct TileLds {
    static constexpr uint32_t kX = kTileCols * 128;  // in a stage: weight rows, then rows
    static constexpr uint32_t kStage = 65536;        // two stages
    static constexpr uint32_t kS = 2 * kStage;       // two sets of scales of four steps: [row][4],
    static constexpr uint32_t kSW = kTileRows * 16;  // then [weight block][4]
    static constexpr uint32_t kSet = kSW + 256;
    static constexpr uint32_t kAmax = kS + 2 * kSet; // gated: [4][row] largest magnitudes
    static constexpr uint32_t kPre = kAmax + 4 * kTileRows * 4; // [EL+1] tiles before the expert
    static constexpr uint32_t kOff = kPre + (kMaxLocal + 1) * 4; // [EL+1] first row of its group
    static constexpr uint32_t kBytes = kOff + (kMaxLocal + 1) * 4;
    static_assert(kX + kTileRows * 128 <= kStage && kBytes <= 160 * 1024, "LDS of a CU");
};

typedef const __attribute__((address_space(3))) u32x4 *lds_chunk;
typedef __attribute__((address_space(3))) float *lds_float;
typedef __attribute__((address_space(3))) int *lds_int;
template <typename P>
__device__ __forceinline__ P lds_at(uint32_t at)
{
    return reinterpret_cast<P>(static_cast<uintptr_t>(at));
}

// 32 rows of a stage as a matrix operand: lane l row l % 32, columns 64 half +
// 32 (l / 32) .. + 31, chunks c = 4 half + 2 (l / 32) and c + 1.  at[i], i = 2
// half + 0 or 1: the address of such a chunk of the lane's row; `by` bytes
// further on the row wanted.
__device__ __forceinline__ i32x8 read_half(const uint32_t (&at)[4], int half, int by)
{
    const u32x4 lo = *lds_at<lds_chunk>(at[2 * half] + by), hi = *lds_at<lds_chunk>(at[2 * half + 1] + by);
    return join(lo, hi);
}

// A 32 x 32 accumulator's rows of weights are spread over lanes l and l + 32, 4
// of 8 each.  Given those of two groups of 8 (x, then y), the lower lanes get
// all of x's and the upper lanes all of y's, in order: first and last 4.
__device__ __forceinline__ void whole_eights(uint32_t &x, uint32_t &y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}

// Groups g and g + 1 of 8 weight rows of an accumulator as bf16, 8 per lane.
__device__ __forceinline__ u32x4 pack_eights(const f32x16 &v, int g)
{
    uint32_t x0 = pack_bf16(v[4 * g], v[4 * g + 1]), x1 = pack_bf16(v[4 * g + 2], v[4 * g + 3]);
    uint32_t y0 = pack_bf16(v[4 * g + 4], v[4 * g + 5]), y1 = pack_bf16(v[4 * g + 6], v[4 * g + 7]);
    whole_eights(x0, y0);
    whole_eights(x1, y1);
    return u32x4{x0, x1, y0, y1};
}

// The value of lane l ^ X, X = 1 or 2.
template <int X>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v)
{
    constexpr int kPerm = X == 1 ? 0xB1 : 0x4E; // quad_perm 1 0 3 2, 2 3 0 1
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kPerm, 0xF, 0xF, true));
}

// Lanes l and l ^ X each hold x and y: afterwards the lower one has both x, the
// upper one both y, each first the lower lane's.
template <int X>
__device__ __forceinline__ void trade(u32x4 &x, u32x4 &y)
{
    const bool up = threadIdx.x & X;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (both moves before the choice: they need every lane)
        const uint32_t other_x = lane_xor<X>(x[i]), other_y = lane_xor<X>(y[i]);
        x[i] = up ? other_y : x[i];
        y[i] = up ? y[i] : other_x;
    }
}

__device__ __forceinline__ f32x16 mfma64(const i32x8 &a, const i32x8 &b, const f32x16 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A group of g rows is cut into the fewest tiles of up to BM rows, of equal
// height but for rounding up to whole blocks of 64 (or BM).
template <int BM>
__device__ __forceinline__ int row_tiles(int g) { return (g + BM - 1) / BM; }
template <int BM>
__device__ __forceinline__ int tile_height(int g, int mt)
{
    constexpr int kBlock = BM < 64 ? BM : 64;
    return ((g + mt - 1) / mt + kBlock - 1) / kBlock * kBlock;
}

// Tables of the tile list, by wave 0: tiles (row tiles * column tiles) before
// each expert, and the groups' first rows, clamped into [0, R].
template <int BM>
__device__ void tile_tables(const ExpertArgs &a, uint32_t pre, uint32_t off)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.EL + kWave - 1) / kWave;
    const int e0 = min(a.EL, lane * per), e1 = min(a.EL, e0 + per);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int lo = static_cast<int>(group_begin(a, e));
        mine += row_tiles<BM>(max(0, static_cast<int>(group_begin(a, e + 1)) - lo)) * a.ntn;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(incl, o);
        if (lane >= o)
            incl += v;
    }
    int run = incl - mine;
    for (int e = e0; e < e1; ++e) {
        const int lo = static_cast<int>(group_begin(a, e)), hi = static_cast<int>(group_begin(a, e + 1));
        *lds_at<lds_int>(pre + e * 4) = run;
        *lds_at<lds_int>(off + e * 4) = lo;
        run += row_tiles<BM>(max(0, hi - lo)) * a.ntn;
    }
    if (lane == kWave - 1) {
        *lds_at<lds_int>(pre + a.EL * 4) = incl;
        *lds_at<lds_int>(off + a.EL * 4) = static_cast<int>(group_begin(a, a.EL));
    }
}

// Tile number `id` of the list: experts in order, within one the row tiles in
// groups of 8, within a group the column tiles with the row tiles of each side
// by side (they read the same weights, and the next column tile the same rows).
template <int BM>
__device__ __forceinline__ Tile list_tile(const ExpertArgs &a, int id, uint32_t pre, uint32_t off)
{
    const int lane = threadIdx.x & (kWave - 1);
    int e = 0; // experts whose tiles all come before
    for (int x = lane; x < (a.EL + kWave - 1) / kWave * kWave; x += kWave)
        e += __popcll(__ballot(x < a.EL && *lds_at<lds_int>(pre + (x + 1) * 4) <= id));
    e = uniform(e);
    int rest = id - uniform(*lds_at<lds_int>(pre + e * 4));
    const int lo = uniform(*lds_at<lds_int>(off + e * 4));
    const int g = max(1, uniform(*lds_at<lds_int>(off + e * 4 + 4)) - lo);
    const int mt = row_tiles<BM>(g), bm = tile_height<BM>(g, mt);
    const int grp = rest / (8 * a.ntn);
    const int gm = min(8, mt - 8 * grp);
    rest -= grp * 8 * a.ntn;
    const int ni = rest / gm;
    Tile t;
    t.e = e;
    t.ni = ni;
    t.r0 = lo + (8 * grp + rest - ni * gm) * bm;
    t.rows = min(bm, static_cast<int>(lo + g - t.r0));
    return t;
}

// The tiles of this workgroup, in order.  Workgroup j runs on XCD j % 8; every
// XCD takes a run of consecutive tiles, so that its L2 holds what they share,
// dealt over its workgroups in rounds.  A group's tiles may differ in height
// and follow each other in a short rhythm, so the dealing shifts from round to
// round.
template <int BM>
struct TileList {
    int first, count, slot, slots, round;
    uint32_t pre, off;
    __device__ __forceinline__ TileList(const ExpertArgs &a, uint32_t pre_, uint32_t off_) : pre(pre_), off(off_)
    {
        const int total = uniform(*lds_at<lds_int>(pre + a.EL * 4));
        const int chunk = (total + kXcds - 1) / kXcds;
        first = blockIdx.x % kXcds * chunk;
        count = min(chunk, total - first);
        slot = blockIdx.x / kXcds;
        slots = gridDim.x / kXcds;
        round = 0;
    }
    __device__ __forceinline__ Tile next(const ExpertArgs &a)
    {
        const int pos = round * slots + (slot + 5 * round) % slots;
        ++round;
        Tile t = {-1, 0, 0, 0};
        if (pos < count)
            t = list_tile<BM>(a, first + pos, pre, off);
        return t;
    }
};

// What a wave keeps from tile to tile.
struct TileWave {
    // loads of a step of the tile that is being sent for, four of weight rows
    // and four of rows, 8 rows each: where this lane's row l / 8 and the chunk
    // that belongs at place l % 8 are
    uint32_t off[8];
    const uint8_t *wbase, *xbase;
    // LDS: chunks of this lane's row in the stage being worked on, that stage,
    // and the set of scales in use (toggled by kStage, kSet)
    uint32_t xad[4];
    uint32_t stage, set;
};

// Where this lane reads rows (wave * n + i) * 8 + l / 8, i < n, of a tile: n
// loads per wave make 64 n rows.
__device__ __forceinline__ void aim_rows(const ExpertArgs &a, const Tile &t, TileWave &w, int n)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (wave * n + i) * 8 + (lane >> 3);
        w.off[4 + i] = min(r, t.rows - 1) * static_cast<uint32_t>(a.K) + place_of(r, lane & 7) * 16;
    }
}

template <bool GATED>
__device__ __forceinline__ void aim(const ExpertArgs &a, const Tile &t, TileWave &w)
{
    constexpr int kCols = GATED ? 128 : kTileCols; // output columns
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const uint32_t K = a.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = wave * 32 + i * 8 + (lane >> 3);
        w.off[i] = (GATED ? r & 127 : min(r, a.N - 1 - t.ni * kTileCols)) * K + place_of(r, lane & 7) * 16;
    }
    aim_rows(a, t, w, 4);
    w.xbase = a.a + t.r0 * a.K;
    w.wbase = a.w + (static_cast<int64_t>(t.e) * (GATED ? 2 * a.N : a.N) +
                     static_cast<int64_t>(t.ni) * kCols) * a.K;
    if (GATED && wave >= kTileWaves / 2) // the stage's weight rows 128 .. 255: up rows
        w.wbase += static_cast<int64_t>(a.N) * a.K;
}

// Load i of step b of the tile aimed at (weight rows, then rows, n loads of
// them), to the stage at `stage`.
__device__ __forceinline__ void send_load(const TileWave &w, int i, int b, uint32_t stage, int n = 4)
{
    const int wave = uniform(threadIdx.x / kWave);
    lds_load16(uniform(stage) + (i < 4 ? (wave * 4 + i) * 1024 : TileLds::kX + (wave * n + i - 4) * 1024),
               (i < 4 ? w.wbase : w.xbase) + b * 128 + w.off[i]);
}

// Load `part` of the scales of steps 4 c .. 4 c + 3 of tile t: of 16 rows
// (parts 0 - 15) or of the two weight blocks (part 16); none beyond.  Four
// lanes per row: one step's scales of a row are far from the next row's, so a
// load for each step would touch one cache line per lane.
template <bool GATED>
__device__ __forceinline__ void send_scales(const ExpertArgs &a, const Tile &t, int c, int part, uint32_t set)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int KB = a.K >> 7;
    const int col = min(4 * c + (lane & 3), KB - 1);
    set = uniform(set);
    if (part < 16) {
        if (part * 16 < t.rows)
            lds_load4(TileLds::kS + set + part * 256,
                      a.sa + t.r0 * KB +
                          (static_cast<uint32_t>(min(part * 16 + (lane >> 2), t.rows - 1)) * KB + col));
    } else if (part == 16) {
        const int nb = GATED ? t.ni : t.ni * 2;
        const uint32_t other = GATED ? a.N >> 7 : min(nb + 1, a.NB - 1) - nb;
        lds_load4(TileLds::kS + set + TileLds::kSW,
                  a.sw + (static_cast<int64_t>(t.e) * a.NB + nb) * KB + ((lane >> 2) ? other * KB + col : col));
    }
}

// One tile with M blocks of 64 rows (a wave's 32 rows of each: waves 0 - 3 the
// first, waves 4 - 7 the second), whose first step and scales have been sent for; sends for
// the first ones of `next` during the last step.  `keep`: vector memory
// accesses newer than those that may be in flight at the start.  Returns the
// same for the next tile.
template <int M, bool GATED, bool FP8>
__device__ __forceinline__ int tile_run(const ExpertArgs &a, const Tile &t, const Tile &next, TileWave &w,
                                        int keep)
{
    typedef TileLds L;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave >> 2, wn = wave & 3;
    const int l32 = lane & 31, upper = lane >> 5;
    const int KB = a.K >> 7;
    const int xrow = wm * 32 + l32;               // + 64 m
    constexpr int kW1 = (GATED ? 128 : 32) * 128; // from the first 32 weight rows to the others
    f32x16 acc[M][2], q[2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[m][j] = f32x16{};
    q[1] = f32x16{}; // the products of the last block of the step before
    float f1 = 0.f;
    // Here: step 0's loads, then (kLoads) step 1's, then the last tile's
    // stores may be on the way.
    if (keep >= 16)
        asm volatile("s_waitcnt vmcnt(24) lgkmcnt(0)\n\ts_barrier" : : : "memory");
    else if (keep >= 8)
        asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" : : : "memory");
    else if (keep >= 4)
        asm volatile("s_waitcnt vmcnt(12) lgkmcnt(0)\n\ts_barrier" : : : "memory");
    else
        asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" : : : "memory");
    // Step b; with `send`, the loads (n of rows) of step `sb` of the tile aimed
    // at go out behind the first two matrix instructions: at the step's start
    // they would hold up its LDS reads, later they would arrive late.  Everything is pinned in this order: the first
    // operands are read first; while the matrix unit works on a block, the
    // products of the block before enter the accumulators, and the next
    // block's rows are read as soon as the last instruction that uses the
    // registers is out.
    const auto step = [&](int b, bool send, int sb, int n) {
        const uint32_t to = w.stage ^ L::kStage;
        const uint32_t wd = ((wn * (GATED ? 32 : 64) - wm * 32) * 128) - L::kX; // from a row's chunk to a weight row's
        uint32_t wad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            wad[i] = w.xad[i] + wd;
        const uint32_t sat = L::kS + w.set + (b & 3) * 4;
        const uint32_t swat = sat + L::kSW + (GATED ? 0 : (wn >> 1) * 16);
        i32x8 wf[2][2], xa, xb;
        wf[0][0] = read_half(wad, 0, 0);
        xa = read_half(w.xad, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        wf[0][1] = read_half(wad, 1, 0);
        xb = read_half(w.xad, 1, 0);
        __builtin_amdgcn_sched_barrier(0);
        wf[1][0] = read_half(wad, 0, kW1);
        wf[1][1] = read_half(wad, 1, kW1);
        const float s0 = *lds_at<lds_float>(swat);
        const float s1 = GATED ? *lds_at<lds_float>(swat + 16) : s0;
        float s = *lds_at<lds_float>(sat + xrow * 16);
        __builtin_amdgcn_sched_barrier(0);
        int unit = 0;
        const auto loads = [&]() {
            if (unit < 2 && send) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (unit * 4 + i < 4 + n)
                        send_load(w, unit * 4 + i, sb, to, n);
            }
            ++unit;
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x16 &into = j ? acc[m][0] : acc[(m + M - 1) % M][1];
                const float f = f1;
                q[j] = mfma64(wf[j][0], xa, f32x16{});
                __builtin_amdgcn_sched_barrier(0);
                if (j && m + 1 < M)
                    xa = read_half(w.xad, 0, (m + 1) * 8192);
                loads();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    into[i] = fmaf(q[1 - j][i], f, into[i]);
                __builtin_amdgcn_sched_barrier(0);
                q[j] = mfma64(wf[j][1], xb, q[j]);
                __builtin_amdgcn_sched_barrier(0);
                f1 = s * (GATED && j ? s1 : s0);
                if (j && m + 1 < M) {
                    xb = read_half(w.xad, 1, (m + 1) * 8192);
                    s = *lds_at<lds_float>(sat + (xrow + 64 * (m + 1)) * 16);
                }
                loads();
#pragma unroll
                for (int i = 8; i < 16; ++i)
                    into[i] = fmaf(q[1 - j][i], f, into[i]);
                // the sums are due here, not where a later branch first needs them
                asm volatile("" : "+v"(into));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        w.stage ^= L::kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w.xad[i] ^= L::kStage;
    };
    const auto scales = [&](int b) {
        if ((b | 3) + 1 < KB)
            send_scales<GATED>(a, t, (b >> 2) + 1, (b & 3) * 8 + wave, w.set ^ L::kSet);
        if ((b & 3) == 3)
            w.set ^= L::kSet;
    };
    aim_rows(a, t, w, M);
    step(0, false, 0, 0);
    // step 1 is needed next: everything but the stores
    if (keep >= 16)
        step_barrier<16>();
    else if (keep >= 8)
        step_barrier<8>();
    else if (keep >= 4)
        step_barrier<4>();
    else
        step_barrier<0>();
    scales(0);
    for (int b = 1; b + 1 < KB; ++b) {
        step(b, true, b + 1, M);
        scales(b);
        step_barrier<0>();
    }
    // (without a next tile its loads are this one's last step's again, unused)
    const int n0 = next.e >= 0 ? 0 : KB - 1, n1 = next.e >= 0 ? 1 : KB - 1;
    if (next.e >= 0)
        aim<GATED>(a, next, w);
    else
        aim_rows(a, t, w, 4);
    step(KB - 1, true, n0, 4);
    if (next.e >= 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            send_scales<GATED>(a, next, 0, i * 8 + wave, w.set ^ L::kSet);
    }
    w.set ^= L::kSet;
    lds_barrier(); // the last step's stage is free
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        send_load(w, i, n1, w.stage ^ L::kStage);
    // The next tile's waits count this one's stores as newer than these loads,
    // which name no memory themselves: here no store may be moved ahead of them
    // (and, by the clobber of the waits, none behind the next tile's start).
    asm volatile("" : : : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[M - 1][1][i] = fmaf(q[1][i], f1, acc[M - 1][1][i]);
    // accumulator element i of a lane: weight row 8 (i / 4) + 4 upper + i % 4
    const bool whole = t.rows == 64 * M && (GATED || (t.ni + 1) * kTileCols <= a.N);
    if (!GATED) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            // v[c]: columns 16 c + 8 upper .. + 7 of this lane's row; traded in
            // groups of four lanes, v[i] is of row i of the four and columns 16
            // (lane % 4) + 8 upper, so that a store writes whole cache lines
            u32x4 v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = pack_eights(acc[m][c >> 1], (c & 1) * 2);
            trade<1>(v[0], v[1]);
            trade<1>(v[2], v[3]);
            trade<2>(v[0], v[2]);
            trade<2>(v[1], v[3]);
            const int row = 64 * m + (xrow & ~3);
            const int n = t.ni * kTileCols + wn * 64 + (lane & 3) * 16 + upper * 8;
            uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N + n;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (row + i < t.rows && n < a.N)
                    *reinterpret_cast<u32x4 *>(o + static_cast<int64_t>(i) * a.N) = v[i];
        }
        return whole ? 4 * M : 0;
    }
    // h in place of the gate
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[m][0][i] = gated(acc[m][0][i], acc[m][1][i]);
    // largest magnitude of each row over the four waves that share it
    if (FP8) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v = fmaxf(v, fabsf(acc[m][0][i]));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (upper == 0)
                *lds_at<lds_float>(L::kAmax + (wn * kTileRows + 64 * m + xrow) * 4) = v;
        }
        lds_barrier();
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (FP8) {
            const int row = 64 * m + xrow;
            const int64_t r = t.r0 + row;
            float v = kAmaxFloor;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v = fmaxf(v, *lds_at<lds_float>(L::kAmax + (i * kTileRows + row) * 4));
            const float inv = __fdiv_rn(kE4M3Max, v);
            uint32_t c[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                c[g] = pack_e4m3(f32x4{acc[m][0][4 * g], acc[m][0][4 * g + 1], acc[m][0][4 * g + 2],
                                       acc[m][0][4 * g + 3]}, inv);
            // columns 16 upper .. + 15: eights of columns, then pairs of those
            whole_eights(c[0], c[1]);
            whole_eights(c[2], c[3]);
            whole_eights(c[0], c[2]);
            whole_eights(c[1], c[3]);
            if (row < t.rows)
                *reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(a.out) + r * a.N + t.ni * 128 + wn * 32 +
                                           upper * 16) = u32x4{c[0], c[1], c[2], c[3]};
            if (wn == 0 && upper == 0 && row < t.rows)
                a.out_scale[r * (a.N >> 7) + t.ni] = __fdiv_rn(v, kE4M3Max);
        } else {
            // (as above, in groups of two lanes: a wave has 64 bytes of a row)
            u32x4 v[2] = {pack_eights(acc[m][0], 0), pack_eights(acc[m][0], 2)};
            trade<1>(v[0], v[1]);
            const int row = 64 * m + (xrow & ~1);
            uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N + t.ni * 128 + wn * 32 +
                          (lane & 1) * 16 + upper * 8;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (row + i < t.rows)
                    *reinterpret_cast<u32x4 *>(o + static_cast<int64_t>(i) * a.N) = v[i];
        }
    }
    return whole ? (FP8 ? M : 2 * M) : 0;
}

template <bool GATED, bool FP8>
__global__ void __launch_bounds__(kTileWaves * kWave) k_expert_tile(ExpertArgs a)
{
    typedef TileLds L;
    extern __shared__ uint8_t tile_lds[]; // all of it by address, from 0
    flag_mismatch(a);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    if (wave == 0)
        tile_tables<kTileRows>(a, L::kPre, L::kOff);
    // the compiler sees LDS reads and writes but not the loads to LDS, nor
    // what the assembly above does: the array's address escapes here
    asm volatile("" : : "v"(tile_lds) : "memory");
    __syncthreads();
    TileList<kTileRows> list(a, L::kPre, L::kOff);
    Tile t = list.next(a);
    if (t.e < 0)
        return;
    TileWave w;
    w.stage = 0;
    w.set = 0;
    const int l32 = lane & 31, upper = lane >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t place = place_of(l32, (i >> 1) * 4 + upper * 2 + (i & 1)) * 16;
        w.xad[i] = L::kX + ((wave >> 2) * 32 + l32) * 128 + place;
    }
    aim<GATED>(a, t, w);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        send_load(w, i, 0, 0);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        send_scales<GATED>(a, t, 0, i * 8 + wave, 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        send_load(w, i, 1, L::kStage);
    int keep = 0;
    while (t.e >= 0) {
        const Tile next = list.next(a);
        switch ((t.rows + 63) >> 6) {
        case 1: keep = tile_run<1, GATED, FP8>(a, t, next, w, keep); break;
        case 2: keep = tile_run<2, GATED, FP8>(a, t, next, w, keep); break;
        case 3: keep = tile_run<3, GATED, FP8>(a, t, next, w, keep); break;
        default: keep = tile_run<4, GATED, FP8>(a, t, next, w, keep); break;
        }
        t = next;
    }
    // no load to LDS may be left when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
}

// ---------------------------------------------------------------------------
// Products with up to a few dozen rows per expert: the weights, read once, are
// all that counts.  Workgroups of 8 waves walk a list of tiles of 32 rows by
// 256 weight rows (gated: 128 gate and 128 up rows) as above, but their steps
// go through a ring of four stages in LDS: three steps, across tiles, are on
// their way at any time.  A wave has 32 weight rows (gated: 16 gate and the 16
// up rows of the same columns).
// With tiles for every CU the rate is HBM's: 256 tokens, top-8 of 128, K = 768,
// N = 2048 42 - 45 us, 4.7 - 5.1 TB/s; gated, 333 tokens on 32 experts, K = 2048, N = 768
// 19.7 - 23 us, 4.5 - 5.2 TB/s.  With fewer, a CU's own: 0.6 us per step of 36 KB, whatever
// the order of its loads and LDS reads, and also where idle CUs had read the
// weights into the L2 before it.  One token, gated, 48 tiles of 16 steps: 16 - 18 us
// (from HBM to registers, 16 waves per 128 columns: 20 - 22 us); for E4M3 outputs a group of 128
// columns shares one scale, so fewer columns per tile are no choice there.
// ---------------------------------------------------------------------------
struct RingLds {
    static constexpr int kRows = kRingRows;
    static constexpr int kStages = 4, kSets = 4;
    static constexpr uint32_t kX = kTileCols * 128;              // in a stage
    static constexpr uint32_t kStage = kX + kRows * 128;
    static constexpr uint32_t kS = kStages * kStage;             // sets of scales of four steps: [row][4],
    static constexpr uint32_t kSW = kRows * 16;                  // then [weight block][4]
    static constexpr uint32_t kSet = kSW + 256;
    static constexpr uint32_t kAmax = kS + kSets * kSet;         // gated: [wave][row]
    static constexpr uint32_t kPre = kAmax + kTileWaves * kRows * 4;
    static constexpr uint32_t kOff = kPre + (kMaxLocal + 1) * 4;
    static constexpr uint32_t kBytes = kOff + (kMaxLocal + 1) * 4;
    static_assert(kBytes <= 160 * 1024, "LDS of a CU");
};
constexpr int kRingLoads = 5; // loads of a wave per step, scales aside

template <bool GATED, bool FP8>
__global__ void __launch_bounds__(kTileWaves * kWave) k_expert_ring(ExpertArgs a)
{
    typedef RingLds L;
    constexpr int kCols = GATED ? 128 : kTileCols; // output columns
    extern __shared__ uint8_t tile_lds[]; // from 0, and the kernel's only LDS
    flag_mismatch(a);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const int l32 = lane & 31, upper = lane >> 5;
    if (wave == 0)
        tile_tables<L::kRows>(a, L::kPre, L::kOff);
    asm volatile("" : : "v"(tile_lds) : "memory"); // (as in the tile kernel)
    __syncthreads();
    const int KB = a.K >> 7;
    const uint32_t K = a.K;

    // ---- loads: the tile and step to send for, and where it goes
    TileList<L::kRows> ahead(a, L::kPre, L::kOff);
    Tile to = {0, 0, 0, 0};
    int to_b = KB, to_stage = 0, to_set = L::kSets - 1;
    uint32_t woff[4], xoff = 0;
    const uint8_t *wbase = nullptr, *xbase = nullptr;
    const auto send = [&]() {
        if (to.e < 0)
            return;
        if (to_b == KB) {
            to = ahead.next(a);
            if (to.e < 0)
                return;
            to_b = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = wave * 32 + i * 8 + (lane >> 3);
                woff[i] = (GATED ? r & 127 : min(r, a.N - 1 - to.ni * kTileCols)) * K +
                          place_of(r, lane & 7) * 16;
            }
            const int r = (wave & 3) * 8 + (lane >> 3);
            xoff = min(r, to.rows - 1) * K + place_of(r, lane & 7) * 16;
            xbase = a.a + to.r0 * a.K;
            wbase = a.w + (static_cast<int64_t>(to.e) * (GATED ? 2 * a.N : a.N) +
                           static_cast<int64_t>(to.ni) * kCols) * a.K;
            if (GATED && wave >= kTileWaves / 2) // up rows
                wbase += static_cast<int64_t>(a.N) * a.K;
        }
        const uint32_t at = uniform(to_stage) * L::kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds_load16(at + (wave * 4 + i) * 1024, wbase + to_b * 128 + woff[i]);
        // two waves bring each 8 rows, so that all count the same loads
        lds_load16(at + L::kX + (wave & 3) * 1024, xbase + to_b * 128 + xoff);
        if ((to_b & 3) == 0) { // with a set's first step its scales: waves 0, 1 the rows', 2 the weights'
            to_set = (to_set + 1) & (L::kSets - 1);
            const uint32_t set = L::kS + uniform(to_set) * L::kSet;
            const int col = min(to_b + (lane & 3), KB - 1);
            if (wave < 2) {
                const uint32_t row = min(wave * 16 + (lane >> 2), to.rows - 1);
                lds_load4(set + wave * 256, a.sa + to.r0 * KB + row * KB + col);
            } else if (wave == 2) {
                const int nb = GATED ? to.ni : to.ni * 2;
                const uint32_t other = GATED ? a.N >> 7 : min(nb + 1, a.NB - 1) - nb;
                lds_load4(set + L::kSW, a.sw + (static_cast<int64_t>(to.e) * a.NB + nb) * KB +
                                            ((lane >> 2) ? other * KB + col : col));
            }
        }
        ++to_b;
        to_stage = (to_stage + 1) & (L::kStages - 1);
    };
#pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i)
        send();

    // ---- products
    TileList<L::kRows> list(a, L::kPre, L::kOff);
    const int wrow = GATED ? (l32 < 16 ? wave * 16 + l32 : 128 + wave * 16 + l32 - 16) : wave * 32 + l32;
    int stage = 0, set = L::kSets - 1;
    for (Tile t = list.next(a); t.e >= 0; t = list.next(a)) {
        f32x16 acc = f32x16{};
        for (int b = 0; b < KB; ++b) {
            // this step's loads are there: at least the next two steps' are newer
            if (to.e >= 0)
                step_barrier<(L::kStages - 2) * kRingLoads>();
            else
                step_barrier<0>();
            send(); // over the stage before, which every wave is done with
            if ((b & 3) == 0)
                set = (set + 1) & (L::kSets - 1);
            const uint32_t at = stage * L::kStage, sat = L::kS + set * L::kSet + (b & 3) * 4;
            uint32_t xad[4], wad[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = (i >> 1) * 4 + upper * 2 + (i & 1);
                xad[i] = at + L::kX + l32 * 128 + place_of(l32, c) * 16;
                wad[i] = at + wrow * 128 + place_of(wrow, c) * 16;
            }
            f32x16 q = mfma64(read_half(wad, 0, 0), read_half(xad, 0, 0), f32x16{});
            q = mfma64(read_half(wad, 1, 0), read_half(xad, 1, 0), q);
            const uint32_t swat = sat + L::kSW + (GATED ? 0 : (wave >> 2) * 16);
            const float s = *lds_at<lds_float>(sat + l32 * 16);
            const float f0 = s * *lds_at<lds_float>(swat);
            const float f1 = GATED ? s * *lds_at<lds_float>(swat + 16) : f0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[i] = fmaf(q[i], i < 8 ? f0 : f1, acc[i]);
            stage = (stage + 1) & (L::kStages - 1);
        }
        const int64_t r = t.r0 + l32;
        const bool in = l32 < t.rows;
        if (!GATED) {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const int n = t.ni * kTileCols + wave * 32 + g * 8 + upper * 8;
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
        const int n = t.ni * 128 + wave * 16 + upper * 8;
        if (FP8) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v = fmaxf(v, fabsf(acc[i]));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (upper == 0)
                *lds_at<lds_float>(L::kAmax + (wave * L::kRows + l32) * 4) = v;
            lds_barrier();
            v = kAmaxFloor;
#pragma unroll
            for (int i = 0; i < kTileWaves; ++i)
                v = fmaxf(v, *lds_at<lds_float>(L::kAmax + (i * L::kRows + l32) * 4));
            const float inv = __fdiv_rn(kE4M3Max, v);
            uint32_t c0 = pack_e4m3(f32x4{acc[0], acc[1], acc[2], acc[3]}, inv);
            uint32_t c1 = pack_e4m3(f32x4{acc[4], acc[5], acc[6], acc[7]}, inv);
            whole_eights(c0, c1);
            if (in)
                *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + r * a.N + n) = u32x2{c0, c1};
            if (in && wave == 0 && upper == 0)
                a.out_scale[r * (a.N >> 7) + t.ni] = __fdiv_rn(v, kE4M3Max);
        } else {
            const u32x4 v = pack_eights(acc, 0);
            if (in)
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + r * a.N + n) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// The most tiles that `rows` rows in EL groups can make.
static int64_t tiles_max(const ExpertArgs &a, int bm)
{
    const int64_t groups = a.load.rows_max < a.EL ? a.load.rows_max : a.EL;
    const int64_t n = (a.load.rows_max / bm + groups) * a.ntn;
    return (n + kXcds - 1) / kXcds * kXcds;
}

// One slot per possible group: a slot per local expert, as a sync-free call's
// padded worst case would have it, cost 7 us at one token (K = 2048, N = 4096,
// 128 experts: 20.5 against 13.4 us).
static hipError_t launch_rows(ExpertArgs &a, hipStream_t s)
{
    a.ntn = (a.N + kRowsCols - 1) / kRowsCols;
    const int64_t nb = a.load.slots * a.ntn;
    if (nb > 0xFFFFFFFFll / (kSplit * kWave))
        return hipErrorInvalidConfiguration;
    launch(k_expert_rows, dim3(static_cast<unsigned>(nb)), dim3(kSplit * kWave), 0, s, a);
    return hipGetLastError();
}

static hipError_t launch_tile(ExpertArgs &a, hipStream_t s)
{
    const int cols = a.gated ? 128 : kTileCols;
    a.ntn = (a.N + cols - 1) / cols;
    const int64_t nb = tiles_max(a, kTileRows);
    if (nb > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb < kCus ? nb : kCus)), blk(kTileWaves * kWave);
    if (!a.gated)
        launch(k_expert_tile<false, false>, g, blk, TileLds::kBytes, s, a);
    else if (a.out_scale)
        launch(k_expert_tile<true, true>, g, blk, TileLds::kBytes, s, a);
    else
        launch(k_expert_tile<true, false>, g, blk, TileLds::kBytes, s, a);
    return hipGetLastError();
}

static hipError_t launch_ring(ExpertArgs &a, hipStream_t s)
{
    const int cols = a.gated ? 128 : kTileCols;
    a.ntn = (a.N + cols - 1) / cols;
    const int64_t nb = tiles_max(a, RingLds::kRows);
    if (nb > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb < kCus ? nb : kCus)), blk(kTileWaves * kWave);
    if (!a.gated)
        launch(k_expert_ring<false, false>, g, blk, RingLds::kBytes, s, a);
    else if (a.out_scale)
        launch(k_expert_ring<true, true>, g, blk, RingLds::kBytes, s, a);
    else
        launch(k_expert_ring<true, false>, g, blk, RingLds::kBytes, s, a);
    return hipGetLastError();
}

hipError_t launch_expert_product(const ExpertArgs &a0, hipStream_t s)
{
    ExpertArgs a = a0;
    switch (choose_expert_kernel(a.load, a.K, a.N, a.gated != 0)) {
    case ExpertKernel::rows: return launch_rows(a, s);
    case ExpertKernel::ring: return launch_ring(a, s);
    default: return launch_tile(a, s);
    }
}

}  // namespace moe
