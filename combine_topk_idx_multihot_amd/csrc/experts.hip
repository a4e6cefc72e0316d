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

// Tile number `id` of the list: experts in order, within one the column tiles
// with the row tiles of each side by side (they read the same weights).  The
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
            const int64_t ni = rest / mt, mi = rest - ni * mt;
            t.e = e;
            t.ni = static_cast<int>(ni);
            t.r0 = lo + mi * BM;
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
// Products with many rows per expert: a workgroup of 8 waves computes a tile
// of 32 * MS rows by 256 output columns (gated: 128 gate and 128 up columns),
// both operands staged through LDS 128 columns deep, two stages.
// ---------------------------------------------------------------------------
constexpr int kTileWaves = 8;
constexpr int kTileCols = 256;

// 16 or 4 bytes per lane from base + off to LDS, lane l at `lds` + 16 l (4 l).
// No register receives anything: the data is there once vmcnt says so.  Written
// as assembly because the compiler, given the builtin, waits for every such
// load before any LDS read that follows, those of the other stage among them.
__device__ __forceinline__ void lds_load16(uint32_t lds, uint32_t off, const void *base)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}
__device__ __forceinline__ void lds_load4(uint32_t lds, uint32_t off, const void *base)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}

// This wave's loads to LDS have landed and its LDS reads are done, and so are
// those of every wave of the workgroup.
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A row of a stage is 128 bytes, eight 16-byte chunks, chunk c kept at place
// c ^ (row % 8): the 16 rows that a matrix operand reads at one chunk then lie
// in different banks.
// Loads from memory that nothing writes while the kernel runs, by the scalar
// unit (their wait is apart from the vector loads').
typedef const __attribute__((address_space(4))) float *scalar_floats;

// What every wave of a tile knows.
template <int MS>
struct TileCtx {
    static constexpr int BM = 32 * MS;
    static constexpr int kXBytes = BM * 128;
    static constexpr int kWBytes = kTileCols * 128;
    static constexpr int kStage = kXBytes + kWBytes + BM * 4; // and the rows' scales
    Tile t;
    uint8_t *lds;
    uint32_t xoff[MS / 2], woff[4], soff; // this wave's loads
    const uint8_t *xbase, *wbase;
    const float *sbase;
    int wave, wm, wn, lane;

    __device__ __forceinline__ void load_stage(int b, int st) const
    {
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
                                (__attribute__((address_space(3))) uint8_t *)lds)) + st * kStage;
#pragma unroll
        for (int i = 0; i < MS / 2; ++i)
            lds_load16(at + (wave * (MS / 2) + i) * 1024, xoff[i], xbase + b * 128);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds_load16(at + kXBytes + (wave * 4 + i) * 1024, woff[i], wbase + b * 128);
        if (wave < BM / kWave)
            lds_load4(at + kXBytes + kWBytes + wave * 256, soff, sbase + b);
    }
};

// The tile with M row subtiles per wave (wave wm takes subtiles 2 m + wm):
// M is MS, or fewer for the last rows of a group.
template <int MS, int M, bool GATED, bool FP8>
__device__ __forceinline__ void tile_run(const ExpertArgs &a, const TileCtx<MS> &c)
{
    constexpr int BM = TileCtx<MS>::BM;
    const Tile &t = c.t;
    const int l16 = c.lane & 15, quarter = c.lane >> 4;
    const int wm = c.wm, wn = c.wn;
    const int KB = a.K >> 7;
    const int place = (quarter ^ (c.lane & 7)) * 16;
    const int xrow = wm * 16 + l16;                      // + 32 m
    const int wrow = (GATED ? wn * 32 : wn * 64) + l16;  // + column(j)
    const auto column = [](int j) { return GATED ? (j & 2) * 64 + (j & 1) * 16 : j * 16; };
    const int x_lo = xrow * 128 + place, x_hi = xrow * 128 + (place ^ 64);
    const int w_lo = TileCtx<MS>::kXBytes + wrow * 128 + place;
    const int w_hi = TileCtx<MS>::kXBytes + wrow * 128 + (place ^ 64);
    const int s_at = TileCtx<MS>::kXBytes + TileCtx<MS>::kWBytes + xrow * 4;
    scalar_floats sw0, sw1;
    {
        const int nb = GATED ? t.ni : min((t.ni * kTileCols + wn * 64) >> 7, a.NB - 1);
        const float *p = a.sw + (static_cast<int64_t>(t.e) * a.NB + nb) * KB;
        sw0 = (scalar_floats)p;
        sw1 = (scalar_floats)(GATED ? p + static_cast<int64_t>(a.N >> 7) * KB : p);
    }
    f32x4 acc[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    float s0 = sw0[0], s1 = GATED ? sw1[0] : 0.f;
    c.load_stage(0, 0);
    for (int b = 0; b < KB; ++b) {
        stage_barrier();
        const int next = min(b + 1, KB - 1);
        if (b + 1 < KB)
            c.load_stage(b + 1, (b + 1) & 1);
        const float n0 = sw0[next], n1 = GATED ? sw1[next] : 0.f;
        const uint8_t *st = c.lds + (b & 1) * TileCtx<MS>::kStage;
        i32x8 wf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            wf[j] = join(*reinterpret_cast<const u32x4 *>(st + w_lo + column(j) * 128),
                         *reinterpret_cast<const u32x4 *>(st + w_hi + column(j) * 128));
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const i32x8 xf = join(*reinterpret_cast<const u32x4 *>(st + x_lo + m * 4096),
                                  *reinterpret_cast<const u32x4 *>(st + x_hi + m * 4096));
            const float s = *reinterpret_cast<const float *>(st + s_at + m * 128);
            const float t0 = s * s0, t1 = GATED ? s * s1 : t0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 q = mfma128(wf[j], xf, zero);
                const float f = j < 2 ? t0 : t1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[m][j][i] = fmaf(q[i], f, acc[m][j][i]);
            }
        }
        s0 = n0;
        s1 = n1;
    }
    if (!GATED) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int row = 32 * m + xrow;
            if (row >= t.rows)
                continue;
            uint16_t *o = static_cast<uint16_t *>(a.out) + (t.r0 + row) * a.N;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = t.ni * kTileCols + wn * 64 + j * 16 + quarter * 4;
                const u32x2 v = {pack_bf16(acc[m][j][0], acc[m][j][1]),
                                 pack_bf16(acc[m][j][2], acc[m][j][3])};
                if (n < a.N)
                    *reinterpret_cast<u32x2 *>(o + n) = v;
            }
        }
        return;
    }
    // h in place of the gate
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[m][j][i] = gated(acc[m][j][i], acc[m][j + 2][i]);
    // largest magnitude of each row over the four waves that share it, over
    // the stages once all have read them
    float *amax = reinterpret_cast<float *>(c.lds); // [4][BM]
    if (FP8) {
        stage_barrier();
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v = fmaxf(v, fabsf(acc[m][j][i]));
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
            if (quarter == 0)
                amax[wn * BM + 32 * m + xrow] = v;
        }
        stage_barrier();
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int row = 32 * m + xrow;
        if (row >= t.rows)
            continue;
        const int64_t r = t.r0 + row;
        const int n = t.ni * 128 + wn * 32 + quarter * 4;
        if (FP8) {
            const float v = fmaxf(fmaxf(fmaxf(amax[row], amax[BM + row]),
                                        fmaxf(amax[2 * BM + row], amax[3 * BM + row])),
                                  kAmaxFloor);
            const float inv = __fdiv_rn(kE4M3Max, v);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<int *>(static_cast<uint8_t *>(a.out) + r * a.N + n + j * 16) =
                    pack_e4m3(acc[m][j], inv);
            if (wn == 0 && quarter == 0)
                a.out_scale[r * (a.N >> 7) + t.ni] = __fdiv_rn(v, kE4M3Max);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x2 v = {pack_bf16(acc[m][j][0], acc[m][j][1]),
                                 pack_bf16(acc[m][j][2], acc[m][j][3])};
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + r * a.N + n + j * 16) = v;
            }
        }
    }
}

template <int MS, bool GATED, bool FP8>
__global__ void __launch_bounds__(kTileWaves * kWave) k_expert_tile(ExpertArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * TileCtx<MS>::kStage];
    constexpr int kCols = GATED ? 128 : kTileCols; // output columns
    flag_mismatch(a);
    TileCtx<MS> c;
    c.t = uniform_tile<32 * MS>(a);
    const Tile &t = c.t;
    if (t.e < 0)
        return;
    c.lds = lds;
    c.lane = threadIdx.x & (kWave - 1);
    c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    c.wm = c.wave & 1;
    c.wn = c.wave >> 1;
    const uint32_t K = a.K, KB = a.K >> 7;
    // 8 rows per load: lane l takes row l / 8 and the chunk that belongs at
    // place l % 8
    const uint32_t chunk = ((c.lane & 7) ^ (c.lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < MS / 2; ++i) {
        const int row = (c.wave * (MS / 2) + i) * 8 + (c.lane >> 3);
        c.xoff[i] = min(row, t.rows - 1) * K + chunk;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = (c.wave * 4 + i) * 8 + (c.lane >> 3); // weight row of the stage
        c.woff[i] = (GATED ? col & 127 : min(col, a.N - 1 - t.ni * kTileCols)) * K + chunk;
    }
    c.soff = min(c.wave * kWave + c.lane, t.rows - 1) * KB * 4;
    c.xbase = a.a + t.r0 * a.K;
    c.sbase = a.sa + t.r0 * (a.K >> 7);
    c.wbase = a.w + (static_cast<int64_t>(t.e) * (GATED ? 2 * a.N : a.N) +
                     static_cast<int64_t>(t.ni) * kCols) * a.K;
    if (GATED && c.wave >= kTileWaves / 2) // the stage's rows 128 .. 255: up rows
        c.wbase += static_cast<int64_t>(a.N) * a.K;
    const int mine = (((t.rows + 15) >> 4) - c.wm + 1) >> 1; // subtiles with rows
    if (mine > MS / 2)
        tile_run<MS, MS, GATED, FP8>(a, c);
    else if (mine > MS / 4 || MS < 8)
        tile_run<MS, MS / 2, GATED, FP8>(a, c);
    else
        tile_run<MS, MS / 4, GATED, FP8>(a, c);
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

template <int MS>
static hipError_t launch_tile(ExpertArgs &a, hipStream_t s)
{
    const int cols = a.gated ? 128 : kTileCols;
    a.ntn = (a.N + cols - 1) / cols;
    const int64_t nb = tiles_max(a, 32 * MS);
    if (nb > 0xFFFFFFFFll / (kTileWaves * kWave))
        return hipErrorInvalidConfiguration;
    const dim3 g(static_cast<unsigned>(nb)), blk(kTileWaves * kWave);
    if (!a.gated)
        launch(k_expert_tile<MS, false, false>, g, blk, 0, s, a);
    else if (a.out_scale)
        launch(k_expert_tile<MS, true, true>, g, blk, 0, s, a);
    else
        launch(k_expert_tile<MS, true, false>, g, blk, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_expert_product(const ExpertArgs &a0, hipStream_t s)
{
    ExpertArgs a = a0;
    if (a.rows_mean > 96)
        return launch_tile<8>(a, s);
    if (a.rows_mean > 32)
        return launch_tile<4>(a, s);
    const bool many = a.rows_mean > 16;
    if (a.gated)
        return many ? launch_swiglu<4>(a, s) : launch_swiglu<1>(a, s);
    return many ? launch_gemm<4>(a, s) : launch_gemm<1>(a, s);
}

}  // namespace moe
