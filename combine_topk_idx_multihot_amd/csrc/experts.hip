// experts.hip -- the experts' products on FP8 rows of the expanded layout.
//
// Rows are E4M3 codes with one fp32 scale per 128 columns (the FP8 dispatch's
// output), weights E4M3 codes [EL,N,K] with one fp32 scale per 128 x 128
// block.  Row r of local expert e's group:
//   y[r,n] = sum over blocks b of 128 columns of
//            sa[r,b] * sw[e, n / 128, b] * (sum over k in b of a[r,k] * w[e,n,k])
// The inner sum is one matrix instruction of depth 128 (gfx950's f8f6f4 form,
// whose 8-bit rate is twice that of the older 8-bit instructions); the two
// scales are multiplied in fp32 and the block's sum enters the fp32
// accumulator by one fma.
// What the 8-bit matrix instructions sum, measured on MI355X with chosen
// operands: products are exact, groups of 8 consecutive columns are aligned to
// the group's largest exponent sum E and cut off below 2^(E-13), and the
// groups are added in fp32.  On normal data that is 1.5e-5 of the result in
// norm (6e-5 on heavy tails), a hundredth of the bf16 output's rounding; the
// older 8-bit instructions do the same, and bf16 instructions on widened
// codes, which are exact to fp32, run at half the rate.  Outputs are therefore
// bf16 (or E4M3), not fp32.
// Products are taken as w * a^T: the accumulator of a 16 x 16 tile then holds,
// per lane, one token row and four consecutive output columns, so that a
// lane's row scale is a single register and its outputs are stored together.
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

// c + a * b^T over 128 columns: a and b hold 16 rows each, lane l the row
// l % 16 and a quarter of its columns (any quarter, the same one in both).
__device__ __forceinline__ f32x4 mfma128(const i32x8 &a, const i32x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
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

// A lane's quarter of 128 columns at p: 16 bytes of each 64-byte half, so
// that the four lanes of a row read whole 64-byte runs.
__device__ __forceinline__ i32x8 load_quarter(const uint8_t *p, int quarter)
{
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(p + quarter * 16);
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(p + 64 + quarter * 16);
    return join(lo, hi);
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

// Tile number `id` of the list: experts in order, within one the row tiles in
// groups of 8, within a group the column tiles with the row tiles of each side
// by side (they read the same weights, and the next column tile the same rows).  The
// group sizes are on the device only, so the grid covers the most tiles that
// R rows can make and workgroups past the real count find none.  Consecutive
// workgroups run on different XCDs; each XCD takes a run of consecutive tiles
// of its own, so that its L2 holds what they share.  Every wave computes this
// by itself: a lane sums the tiles of EL / 64 experts, a wave scan follows.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ExpertArgs &a, int64_t bid)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.EL + kWave - 1) / kWave;
    const int e0 = min(a.EL, lane * per), e1 = min(a.EL, e0 + per);
    int64_t mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int64_t lo = group_begin(a, e), hi = max(lo, group_begin(a, e + 1));
        mine += (hi - lo + BM - 1) / BM;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int64_t v = __shfl_up(incl, o);
        if (lane >= o)
            incl += v;
    }
    const int64_t total = __shfl(incl, kWave - 1) * a.ntn;
    Tile t = {-1, 0, 0, 0};
    const int64_t chunk = (total + kXcds - 1) / kXcds;
    const int64_t pos = bid / kXcds;
    const int64_t id = (bid % kXcds) * chunk + pos;
    if (pos >= chunk || id >= total)
        return t;
    const uint64_t m = __ballot(incl * a.ntn > id);
    const int src = __builtin_ctzll(m); // total > id: some lane holds it
    int64_t rest = id - __shfl(incl - mine, src) * a.ntn;
    int e = min(a.EL, src * per);
    const int eend = min(a.EL, e + per);
    for (; e < eend; ++e) {
        const int64_t lo = group_begin(a, e), hi = max(lo, group_begin(a, e + 1));
        const int64_t mt = (hi - lo + BM - 1) / BM;
        if (rest < mt * a.ntn) {
            const int64_t grp = rest / (8 * a.ntn);
            const int64_t gm = min<int64_t>(8, mt - 8 * grp);
            rest -= grp * 8 * a.ntn;
            const int64_t ni = rest / gm;
            t.e = e;
            t.ni = static_cast<int>(ni);
            t.r0 = lo + (8 * grp + rest - ni * gm) * BM;
            t.rows = static_cast<int>(min<int64_t>(BM, hi - t.r0));
            break;
        }
        rest -= mt * a.ntn;
    }
    return t;
}

// The tile in scalar registers: it is the same in every lane, which the
// compiler cannot see (R, and so a row, fits 31 bits).
template <int BM>
__device__ __forceinline__ Tile uniform_tile(const ExpertArgs &a)
{
    Tile t = find_tile<BM>(a, blockIdx.x);
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.ni = __builtin_amdgcn_readfirstlane(t.ni);
    t.r0 = __builtin_amdgcn_readfirstlane(static_cast<int>(t.r0));
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    return t;
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
// product, one wave per 16 output columns and 16 * MT rows
// ---------------------------------------------------------------------------
constexpr int kProdWaves = 4;

template <int MT>
__global__ void __launch_bounds__(kProdWaves * kWave) k_expert_gemm(ExpertArgs a)
{
    flag_mismatch(a);
    const Tile t = uniform_tile<16 * MT>(a);
    if (t.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = (t.ni * kProdWaves + wave) * 16;
    if (n0 >= a.N)
        return;
    const int l16 = lane & 15, quarter = lane >> 4;
    const int KB = a.K >> 7;
    const uint8_t *__restrict__ w =
        a.w + (static_cast<int64_t>(t.e) * a.N + min(n0 + l16, a.N - 1)) * a.K;
    const float *__restrict__ sw =
        a.sw + (static_cast<int64_t>(t.e) * a.NB + (n0 >> 7)) * KB;
    const uint8_t *x[MT];
    const float *sx[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t r = t.r0 + min(m * 16 + l16, t.rows - 1);
        x[m] = a.a + r * a.K;
        sx[m] = a.sa + r * KB;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < KB; ++b) {
        const i32x8 wf = load_quarter(w + b * 128, quarter);
        const float swb = sw[b];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const i32x8 xf = load_quarter(x[m] + b * 128, quarter);
            const float s = sx[m][b] * swb;
            const f32x4 p = mfma128(wf, xf, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[m][i] = fmaf(p[i], s, acc[m][i]);
        }
    }
    const int n = n0 + quarter * 4;
    if (n >= a.N)
        return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + l16;
        if (row >= t.rows)
            continue;
        const int64_t at = (t.r0 + row) * a.N + n;
        const u32x2 v = {pack_bf16(acc[m][0], acc[m][1]), pack_bf16(acc[m][2], acc[m][3])};
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + at) = v;
    }
}

// ---------------------------------------------------------------------------
// gated product: a workgroup of 8 waves computes 128 columns of h, wave v the
// gate and the up columns 16 v .. 16 v + 15 of them, so that each lane holds
// both factors; the row's largest magnitude (for the E4M3 output) is the
// maximum over the four lanes that share the row and, through LDS, the waves.
// ---------------------------------------------------------------------------
constexpr int kGatedWaves = 8;

template <int MT, bool OUT_FP8>
__global__ void __launch_bounds__(kGatedWaves * kWave) k_expert_swiglu(ExpertArgs a)
{
    __shared__ float amax[kGatedWaves][16 * MT];
    flag_mismatch(a);
    const Tile t = uniform_tile<16 * MT>(a);
    if (t.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n0 = t.ni * 128 + wave * 16; // columns of h
    const int l16 = lane & 15, quarter = lane >> 4;
    const int KB = a.K >> 7;
    const int64_t wrow = static_cast<int64_t>(t.e) * 2 * a.N + n0 + l16;
    const uint8_t *__restrict__ wg = a.w + wrow * a.K;
    const uint8_t *__restrict__ wu = a.w + (wrow + a.N) * a.K;
    const float *__restrict__ sg = a.sw + (static_cast<int64_t>(t.e) * a.NB + t.ni) * KB;
    const float *__restrict__ su = sg + static_cast<int64_t>(a.N >> 7) * KB;
    const uint8_t *x[MT];
    const float *sx[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t r = t.r0 + min(m * 16 + l16, t.rows - 1);
        x[m] = a.a + r * a.K;
        sx[m] = a.sa + r * KB;
    }
    f32x4 ag[MT], au[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        ag[m] = au[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < KB; ++b) {
        const i32x8 gf = load_quarter(wg + b * 128, quarter);
        const i32x8 uf = load_quarter(wu + b * 128, quarter);
        const float sgb = sg[b], sub = su[b];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const i32x8 xf = load_quarter(x[m] + b * 128, quarter);
            const float s = sx[m][b];
            const f32x4 pg = mfma128(gf, xf, f32x4{0.f, 0.f, 0.f, 0.f});
            const f32x4 pu = mfma128(uf, xf, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ag[m][i] = fmaf(pg[i], s * sgb, ag[m][i]);
                au[m][i] = fmaf(pu[i], s * sub, au[m][i]);
            }
        }
    }
    f32x4 h[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[m][i] = gated(ag[m][i], au[m][i]);
    const int n = n0 + quarter * 4;
    if (OUT_FP8) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float v = fmaxf(fmaxf(fabsf(h[m][0]), fabsf(h[m][1])), fmaxf(fabsf(h[m][2]), fabsf(h[m][3])));
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (quarter == 0)
                amax[wave][m * 16 + l16] = v;
        }
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + l16;
        if (row >= t.rows)
            continue;
        const int64_t r = t.r0 + row;
        if (OUT_FP8) {
            float v = kAmaxFloor;
#pragma unroll
            for (int q = 0; q < kGatedWaves; ++q)
                v = fmaxf(v, amax[q][row]);
            const float inv = __fdiv_rn(kE4M3Max, v);
            *reinterpret_cast<int *>(static_cast<uint8_t *>(a.out) + r * a.N + n) = pack_e4m3(h[m], inv);
            if (wave == 0 && quarter == 0)
                a.out_scale[r * (a.N >> 7) + t.ni] = __fdiv_rn(v, kE4M3Max);
        } else {
            const u32x2 q = {pack_bf16(h[m][0], h[m][1]), pack_bf16(h[m][2], h[m][3])};
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + r * a.N + n) = q;
        }
    }
}

// ---------------------------------------------------------------------------
// Products with many rows per expert: workgroups of 8 waves, one per CU, each
// taking tiles of up to 256 rows by 256 output columns (gated: 128 gate and 128
// up columns) one after the other.  Rows and weights come through LDS 128
// columns (a step) at a time, in two stages: while a step is worked on, the
// next one's data, or the first step's of the next tile, is on its way.
// ---------------------------------------------------------------------------
constexpr int kTileWaves = 8;
constexpr int kTileCols = 256;
constexpr int kTileRows = 256;
constexpr int kTileBlocks = kTileRows / 64; // blocks of 64 rows, 32 per half of the waves
constexpr int kCus = 256;                   // MI355X
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

// LDS of the tile kernel, from address 0.  A row of a stage is 128 bytes, eight
// 16-byte chunks, chunk c kept at place c ^ (row % 8): the rows that a matrix
// operand reads at one chunk then lie in different banks.
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

__device__ __forceinline__ f32x16 mfma64(const i32x8 &a, const i32x8 &b, const f32x16 &c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A group of g rows is cut into the fewest tiles, of equal height but for
// rounding up to whole blocks of 64.
__device__ __forceinline__ int row_tiles(int g) { return (g + kTileRows - 1) / kTileRows; }
__device__ __forceinline__ int tile_height(int g, int mt)
{
    return ((g + mt - 1) / mt + 63) / 64 * 64;
}

// Tables of the tile list, by wave 0: tiles (row tiles * column tiles) before
// each expert, and the groups' first rows, clamped into [0, R].
__device__ void tile_tables(const ExpertArgs &a)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (a.EL + kWave - 1) / kWave;
    const int e0 = min(a.EL, lane * per), e1 = min(a.EL, e0 + per);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int lo = static_cast<int>(group_begin(a, e));
        mine += row_tiles(max(0, static_cast<int>(group_begin(a, e + 1)) - lo)) * a.ntn;
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
        *lds_at<lds_int>(TileLds::kPre + e * 4) = run;
        *lds_at<lds_int>(TileLds::kOff + e * 4) = lo;
        run += row_tiles(max(0, hi - lo)) * a.ntn;
    }
    if (lane == kWave - 1) {
        *lds_at<lds_int>(TileLds::kPre + a.EL * 4) = incl;
        *lds_at<lds_int>(TileLds::kOff + a.EL * 4) = static_cast<int>(group_begin(a, a.EL));
    }
}

// Tile number `id` of the list: experts in order, within one the row tiles in
// groups of 8, within a group the column tiles with the row tiles of each side
// by side (they read the same weights, and the next column tile the same rows).
__device__ __forceinline__ Tile list_tile(const ExpertArgs &a, int id)
{
    const int lane = threadIdx.x & (kWave - 1);
    int e = 0; // experts whose tiles all come before
    for (int x = lane; x < (a.EL + kWave - 1) / kWave * kWave; x += kWave)
        e += __popcll(__ballot(x < a.EL && *lds_at<lds_int>(TileLds::kPre + (x + 1) * 4) <= id));
    e = uniform(e);
    int rest = id - uniform(*lds_at<lds_int>(TileLds::kPre + e * 4));
    const int lo = uniform(*lds_at<lds_int>(TileLds::kOff + e * 4));
    const int g = max(1, uniform(*lds_at<lds_int>(TileLds::kOff + e * 4 + 4)) - lo);
    const int mt = row_tiles(g), bm = tile_height(g, mt);
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
    const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w.off[4 + i] = min((wave * n + i) * 8 + (lane >> 3), t.rows - 1) * static_cast<uint32_t>(a.K) + chunk;
}

template <bool GATED>
__device__ __forceinline__ void aim(const ExpertArgs &a, const Tile &t, TileWave &w)
{
    constexpr int kCols = GATED ? 128 : kTileCols; // output columns
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = uniform(threadIdx.x / kWave);
    const uint32_t K = a.K;
    const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = wave * 32 + i * 8 + (lane >> 3);
        w.off[i] = (GATED ? r & 127 : min(r, a.N - 1 - t.ni * kTileCols)) * K + chunk;
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
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[M - 1][1][i] = fmaf(q[1][i], f1, acc[M - 1][1][i]);
    // accumulator element i of a lane: weight row 8 (i / 4) + 4 upper + i % 4
    const bool whole = t.rows == 64 * M && (GATED || (t.ni + 1) * kTileCols <= a.N);
    if (!GATED) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int row = 64 * m + xrow;
            uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < 4; g += 2) {
                    const int n = t.ni * kTileCols + wn * 64 + j * 32 + g * 8 + upper * 8;
                    const u32x4 v = pack_eights(acc[m][j], g);
                    if (row < t.rows && n < a.N)
                        *reinterpret_cast<u32x4 *>(o + n) = v;
                }
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
        const int row = 64 * m + xrow;
        const int64_t r = t.r0 + row;
        const int n = t.ni * 128 + wn * 32 + upper * 8;
        if (FP8) {
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
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                whole_eights(c[g], c[g + 1]);
                if (row < t.rows)
                    *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + r * a.N + n + g * 8) =
                        u32x2{c[g], c[g + 1]};
            }
            if (wn == 0 && upper == 0 && row < t.rows)
                a.out_scale[r * (a.N >> 7) + t.ni] = __fdiv_rn(v, kE4M3Max);
        } else {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const u32x4 v = pack_eights(acc[m][0], g);
                if (row < t.rows)
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + r * a.N + n + g * 8) = v;
            }
        }
    }
    return whole ? 2 * M : 0;
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
        tile_tables(a);
    // the compiler sees LDS reads and writes but not the loads to LDS, nor
    // what the assembly above does: the array's address escapes here
    asm volatile("" : : "v"(tile_lds) : "memory");
    __syncthreads();
    // Workgroup j runs on XCD j % 8; every XCD takes a run of consecutive
    // tiles, so that its L2 holds what they share, dealt over its workgroups
    // in rounds.  A group's tiles may differ in height and follow each other
    // in a short rhythm, so the dealing shifts from round to round.
    const int total = uniform(*lds_at<lds_int>(L::kPre + a.EL * 4));
    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const int slots = gridDim.x / kXcds;
    const int chunk = (total + kXcds - 1) / kXcds;
    const int first = xcd * chunk, count = min(chunk, total - first);
    const auto tile = [&](int round) {
        const int pos = round * slots + (slot + 5 * round) % slots;
        Tile t = {-1, 0, 0, 0};
        if (pos < count)
            t = list_tile(a, first + pos);
        return t;
    };
    const auto next_tile = [&](int &round) {
        // a round's last places may be beyond the list
        Tile t = tile(++round);
        return t;
    };
    int round = 0;
    Tile t = tile(0);
    if (t.e < 0)
        return;
    TileWave w;
    w.stage = 0;
    w.set = 0;
    const int l32 = lane & 31, upper = lane >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t place = (((i >> 1) * 4 + upper * 2 + (i & 1)) ^ (lane & 7)) * 16;
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
        const Tile next = next_tile(round);
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
// launch
// ---------------------------------------------------------------------------
// The most tiles that `rows` rows in EL groups can make.
static int64_t tiles_max(const ExpertArgs &a, int bm)
{
    const int64_t groups = a.rows_max < a.EL ? a.rows_max : a.EL;
    const int64_t n = (a.rows_max / bm + groups) * a.ntn;
    return (n + kXcds - 1) / kXcds * kXcds;
}

template <int MT>
static hipError_t launch_gemm(ExpertArgs &a, hipStream_t s)
{
    a.ntn = (a.N + 16 * kProdWaves - 1) / (16 * kProdWaves);
    const int64_t nb = tiles_max(a, 16 * MT);
    if (nb > 0xFFFFFFFFll / (kProdWaves * kWave))
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb)), blk(kProdWaves * kWave);
    launch(k_expert_gemm<MT>, g, blk, 0, s, a);
    return hipGetLastError();
}

template <int MT>
static hipError_t launch_swiglu(ExpertArgs &a, hipStream_t s)
{
    a.ntn = a.N >> 7;
    const int64_t nb = tiles_max(a, 16 * MT);
    if (nb > 0xFFFFFFFFll / (kGatedWaves * kWave))
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb)), blk(kGatedWaves * kWave);
    if (a.out_scale)
        launch(k_expert_swiglu<MT, true>, g, blk, 0, s, a);
    else
        launch(k_expert_swiglu<MT, false>, g, blk, 0, s, a);
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

hipError_t launch_expert_product(const ExpertArgs &a0, hipStream_t s)
{
    ExpertArgs a = a0;
    if (a.rows_mean > 32 && a.K >= 256) // (the tile kernel sends for two steps ahead)
        return launch_tile(a, s);
    const bool many = a.rows_mean > 16;
    if (a.gated)
        return many ? launch_swiglu<4>(a, s) : launch_swiglu<1>(a, s);
    return many ? launch_gemm<4>(a, s) : launch_gemm<1>(a, s);
}

}  // namespace moe
