// expert_tiles.h -- device code that the experts' products share (experts.hip,
// experts_mx.hip): the list of tiles over groups of rows, loads to LDS, the
// layout of a stage in LDS and the packing of outputs.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

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

__device__ __forceinline__ int64_t group_begin(const ProductArgs &a, int e)
{
    return max<int64_t>(0, min<int64_t>(a.off[e], a.R));
}

__device__ __forceinline__ void flag_mismatch(const ProductArgs &a)
{
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.eager && a.status[0] != a.R)
        atomicOr(&a.status[1], 4);
}

// silu(g) * u
__device__ __forceinline__ float gated(float g, float u)
{
    return g / (1.0f + __expf(-g)) * u;
}

// The local expert of the s-th group that has rows, -1 if there are not so many.
__device__ __forceinline__ int nonempty_expert(const ProductArgs &a, int s)
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

typedef const __attribute__((address_space(3))) u32x4 *lds_chunk;
typedef __attribute__((address_space(3))) float *lds_float;
typedef __attribute__((address_space(3))) int *lds_int;
template <typename P>
__device__ __forceinline__ P lds_at(uint32_t at)
{
    return reinterpret_cast<P>(static_cast<uintptr_t>(at));
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
__device__ void tile_tables(const ProductArgs &a, uint32_t pre, uint32_t off)
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
__device__ __forceinline__ Tile list_tile(const ProductArgs &a, int id, uint32_t pre, uint32_t off)
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
    __device__ __forceinline__ TileList(const ProductArgs &a, uint32_t pre_, uint32_t off_) : pre(pre_), off(off_)
    {
        const int total = uniform(*lds_at<lds_int>(pre + a.EL * 4));
        const int chunk = (total + kXcds - 1) / kXcds;
        first = blockIdx.x % kXcds * chunk;
        count = min(chunk, total - first);
        slot = blockIdx.x / kXcds;
        slots = gridDim.x / kXcds;
        round = 0;
    }
    __device__ __forceinline__ Tile next(const ProductArgs &a)
    {
        const int pos = round * slots + (slot + 5 * round) % slots;
        ++round;
        Tile t = {-1, 0, 0, 0};
        if (pos < count)
            t = list_tile<BM>(a, first + pos, pre, off);
        return t;
    }
};

// The most tiles that `rows` rows in EL groups can make.
inline int64_t tiles_max(const ProductArgs &a, int bm)
{
    const int64_t groups = a.load.rows_max < a.EL ? a.load.rows_max : a.EL;
    const int64_t n = (a.load.rows_max / bm + groups) * a.ntn;
    return (n + kXcds - 1) / kXcds * kXcds;
}

}  // namespace moe
