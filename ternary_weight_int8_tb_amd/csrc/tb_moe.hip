// tb_moe.hip -- an FFN of ternary or sign experts (gfx950): the pairs (token, expert) sorted by
// expert, gate/up with SiLU and the rotation of h, the down product, and the weighted sum.
//
// The products are those of the single-matrix calls, bit for bit: exact integer block sums, the
// terms (scale * dq) * isum, the fixed tree over the blocks of a step (8 ternary or 16 sign
// blocks), and the steps added in order (tb_device.h). A pair's row therefore has the bits that
// tb_gemv_ternary gives it on its expert's matrix, however many rows the expert received.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tb.h"
#include "tb_device.h"
#include "tb_host.h"
#include "tb_rows.h"

namespace {

using namespace tbk;

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kMaxGrid = 1 << 20;
constexpr int kMaxExperts = 65536;
constexpr int kXcds = 8;

// ------------------------------------------------------------------------------------
// Plan: a stable counting sort of the pairs by expert. Workgroup e counts the pairs of lower
// experts (where its list starts) and writes its own pairs in ascending order; workgroup
// `experts` writes the end. No workgroup waits for another. Ids outside [0, experts) are in no
// list.
// ------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

__global__ __launch_bounds__(kPlanThreads) void moe_plan_kernel(const int32_t *__restrict__ ids, int pairs,
                                                                int experts, int32_t *__restrict__ offsets,
                                                                int32_t *__restrict__ order)
{
    __shared__ int less_s[kPlanWaves], same_s[kPlanWaves];
    const int e = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // each wave takes a contiguous range of whole 64-pair groups
    const int groups = (pairs - 1) / 64 + 1;
    const int g0 = part_lo(groups, kPlanWaves, wave), g1 = part_lo(groups, kPlanWaves, wave + 1);
    int less = 0, same = 0;
    for (int g = g0; g < g1; ++g) {
        const int64_t p = (int64_t)g * 64 + lane;
        const int id = p < pairs ? ids[p] : -1;
        less += __popcll(__ballot(id >= 0 && id < e));
        same += __popcll(__ballot(id == e));
    }
    if (lane == 0) {
        less_s[wave] = less;
        same_s[wave] = same;
    }
    __syncthreads();
    int start = 0, before = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        start += less_s[w];
        before += w < wave ? same_s[w] : 0;
    }
    if (threadIdx.x == 0)
        offsets[e] = start;
    if (e == experts)
        return;
    int at = start + before;
    for (int g = g0; g < g1; ++g) {
        const int64_t p = (int64_t)g * 64 + lane;
        const bool mine = p < pairs && ids[p] == e;
        const uint64_t mask = __ballot(mine);
        if (mine)
            order[at + __popcll(mask & ((1ull << lane) - 1))] = (int)p;
        at += __popcll(mask);
    }
}

// ------------------------------------------------------------------------------------
// Tiles: an expert's list is cut into tiles of up to ROWS pairs, numbered over all experts.
// Every wave scans the lists' lengths on its own (all lanes active). Values outside [0, pairs]
// that a caller may have left in offsets are cut, so that no slot past the arrays is touched.
// ------------------------------------------------------------------------------------
struct Tile {
    int expert, slot, rows;   // the tile's first slot and number of pairs
};
template <int ROWS>
struct Tiles {
    int lo, count, tiles, upto;   // of this lane's expert, in the group of 64 that was read last
    __device__ __forceinline__ void read(const int32_t *__restrict__ offsets, int experts, int pairs, int e0)
    {
        const int lane = threadIdx.x & 63, e = e0 + lane;
        lo = 0, count = 0;
        if (e < experts) {
            lo = min(max(offsets[e], 0), pairs);
            count = max(min(offsets[e + 1], pairs) - lo, 0);
        }
        tiles = (count + ROWS - 1) / ROWS;
        upto = tiles;   // inclusive prefix sum over the lanes
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off);
            upto += lane >= off ? o : 0;
        }
    }
    // The number of tiles; leaves the first 64 experts read.
    __device__ __forceinline__ int total(const int32_t *offsets, int experts, int pairs)
    {
        int sum = 0;
        for (int e0 = (experts - 1) / 64 * 64; e0 >= 0; e0 -= 64) {
            read(offsets, experts, pairs, e0);
            sum += __builtin_amdgcn_readlane(upto, 63);
        }
        return sum;
    }
    // Tile t (0 <= t < total), after total().
    __device__ __forceinline__ Tile find(const int32_t *offsets, int experts, int pairs, int t)
    {
        int before = 0, e0 = 0;
        for (;;) {
            const int n = __builtin_amdgcn_readlane(upto, 63);
            if (t < before + n || e0 + 64 >= experts)
                break;
            before += n;
            e0 += 64;
            read(offsets, experts, pairs, e0);
        }
        // wave-uniform values, in scalar registers
        const int src = __ffsll((unsigned long long)__ballot(before + upto > t)) - 1;
        const int r0 = (t - before - __builtin_amdgcn_readlane(upto - tiles, src)) * ROWS;
        return {e0 + src, __builtin_amdgcn_readlane(lo, src) + r0, min(ROWS, __builtin_amdgcn_readlane(count, src) - r0)};
    }
};

// 4x4 byte transpose: o_j = bytes j of a, b, c, d.
__device__ __forceinline__ v4i transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t abl = __builtin_amdgcn_perm(b, a, 0x05010400u), abh = __builtin_amdgcn_perm(b, a, 0x07030602u);
    const uint32_t cdl = __builtin_amdgcn_perm(d, c, 0x05010400u), cdh = __builtin_amdgcn_perm(d, c, 0x07030602u);
    return v4i{(int)__builtin_amdgcn_perm(cdl, abl, 0x05040100u), (int)__builtin_amdgcn_perm(cdl, abl, 0x07060302u),
               (int)__builtin_amdgcn_perm(cdh, abh, 0x05040100u), (int)__builtin_amdgcn_perm(cdh, abh, 0x07060302u)};
}

template <int FMT>
struct Core;
// Ternary: of a block's 8 code words lane group g holds words 2g, 2g + 1; matrix instruction s
// takes word 2g + s, whose decoded bytes are the weights {j, j+4, j+8, j+12}.
template <>
struct Core<TB_FMT_TERNARY2> {
    static constexpr int kStep = 8;        // blocks of a step
    static constexpr int kBlockBytes = 32;
    uint2 w;
    // off: the lane's byte offset in the expert's codes (its row, plus 8 g); block: the same for all lanes
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off, int block)
    {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, off, block * kBlockBytes, 0);
        w = make_uint2(v.x, v.y);
    }
    __device__ __forceinline__ v4i weights(int s) const
    {
        uint32_t a, b, c, d;
        decode_ternary(s ? w.y : w.x, a, b, c, d);
        return v4i{(int)a, (int)b, (int)c, (int)d};
    }
    static __device__ __forceinline__ v4i acts(uint4 lo, uint4 hi, int s)
    {
        return s ? transpose4(hi.x, hi.y, hi.z, hi.w) : transpose4(lo.x, lo.y, lo.z, lo.w);
    }
};
// Sign: lane group g holds word g of a block's 4, the weights 32 g .. 32 g + 31; bit j of its
// bytes are the weights {j, j+8, j+16, j+24}. Instruction s takes j = 4 s .. 4 s + 3, as +1 / -1.
template <>
struct Core<TB_FMT_SIGN1> {
    static constexpr int kStep = 16;
    static constexpr int kBlockBytes = 16;
    uint32_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off, int block)
    {
        w = __builtin_amdgcn_raw_buffer_load_b32(r, off, block * kBlockBytes, 0);
    }
    __device__ __forceinline__ v4i weights(int s) const
    {
        v4i o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = (int)__builtin_amdgcn_perm(0u, 0x000001FFu, (w >> (4 * s + j)) & 0x01010101u);
        return o;
    }
    static __device__ __forceinline__ v4i acts(uint4 lo, uint4 hi, int s)
    {
        return s ? transpose4(lo.y, lo.w, hi.y, hi.w) : transpose4(lo.x, lo.z, hi.x, hi.z);
    }
};

struct MoeArgs {
    const uint8_t *codes[2];
    const uint16_t *scales[2];
    int experts, n, k;
    const int8_t *q;
    const float *dq;
    const int32_t *offsets, *order;
    int pairs, topk;   // gate/up: the activation row of pair p is p / topk
    float *out;        // gate/up: h, a row per slot; down: y, a row per pair
    int8_t *qh;        // gate/up: rotquant(h)
    float *dqh;
    float unit;
};

// ------------------------------------------------------------------------------------
// Products of one expert's weight rows with a tile of its pairs, in two kernels that share this:
//   * The activations are the A operand, the weights the B operand of v_mfma_i32_16x16x64_i8: lane
//     (i, g) = (l % 16, l / 16) supplies row i of either, and ends with A rows 4 g .. 4 g + 3 of
//     weight row i. So a lane folds the row whose codes and scales it loaded itself. Pair t of
//     16 is A row 4 (t % 4) + t / 4: element e of lane group g is pair g + 4 e, and a tile of up to
//     4 pairs folds one element.
//   * A wave owns two tiles of 16 weight rows (gate/up: the same rows of both) through all of k;
//     nothing of a row crosses waves. The blocks of a step are taken in the order in which the
//     step's tree adds them: 0, last, last - 1, last - 2, then the next four downwards. Such a phase
//     of 4 blocks leaves one partial sum, the tree above it one register set per level.
//   * Activations are staged in LDS as the operands read them: byte-transposed, 16 bytes per lane;
//     slot row ^ 2 g keeps reads and writes free of bank conflicts.
//   * Blocks past the end of k have dq = 0 and count +0.
// ------------------------------------------------------------------------------------
constexpr int kTilesPerWave = 2;

// Block `b` (0 .. 3) of phase p: its index in k.
template <int FMT>
__device__ __forceinline__ int phase_block(int p, int b)
{
    constexpr int kStep = Core<FMT>::kStep, kPhases = kStep / 4;
    const int j = 4 * (p % kPhases) + b;
    return p / kPhases * kStep + (j ? kStep - j : 0);
}

// A row of a tile's pair t
__device__ __forceinline__ int pair_row(int t) { return (t & ~15) | (t & 3) << 2 | (t >> 2 & 3); }

// The activation row of a slot.
template <bool TWO>
__device__ __forceinline__ size_t act_row(const MoeArgs &a, int slot)
{
    return TWO ? (unsigned)min(max(a.order[slot], 0), a.pairs - 1) / (unsigned)a.topk : (unsigned)slot;
}

// The lane's rows of a wave's two tiles. Rows past n read the last one and are not stored.
template <int FMT, bool TWO>
struct WeightRows {
    __amdgpu_buffer_rsrc_t codes[2], scales[2];
    uint32_t coff[2], soff[2];   // byte offsets of the row's codes and scales
    int col[2];
    __device__ __forceinline__ WeightRows(const MoeArgs &a, int expert, int n0, int wave, int i, int nb)
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int m = TWO ? r : 0;
            col[r] = n0 + 16 * (TWO ? wave : 2 * wave + r) + i;
            const uint32_t row = min(col[r], a.n - 1);
            const size_t first = (size_t)expert * a.n * nb, blocks = (size_t)a.n * nb;
            codes[r] = buffer_rsrc(a.codes[m] + first * Core<FMT>::kBlockBytes, (uint32_t)(blocks * Core<FMT>::kBlockBytes));
            coff[r] = row * (nb * Core<FMT>::kBlockBytes);
            // the scales buffer starts, and ends, at whole words
            const size_t odd = first & 1;
            scales[r] = buffer_rsrc(a.scales[m] + (first - odd), (uint32_t)((blocks + odd + 1) / 2 * 4));
            soff[r] = (row * nb + (uint32_t)odd) * 2;
        }
    }
};

// The tree over a step's phases: ternary P0 + P1, sign (P0 + P1) + (P2 + P3); v: the sum of phase q.
template <int PHASES>
__device__ __forceinline__ void add_phase(int q, float v, float &part0, float &part1, float &acc)
{
    if (q == 0)
        part0 = v;
    else if (q == 2)
        part1 = v;
    else if (PHASES == 4 && q == 1)
        part0 += v;
    else
        acc += part0 + (PHASES == 4 ? part1 + v : v);
}

// h of a gate/up lane, or the down outputs of its two rows, for pair `tok` of the tile.
template <bool TWO>
__device__ __forceinline__ void store_pair(const MoeArgs &a, const Tile &tile, int tok, const int (&col)[2], float v0, float v1)
{
    if (tok >= tile.rows)
        return;
    const int row = TWO ? tile.slot + tok : a.order[tile.slot + tok];
    if ((unsigned)row >= (unsigned)a.pairs)
        return;
    float *o = a.out + (size_t)row * a.n;
    if (TWO) {
        if (col[0] < a.n)
            o[col[0]] = silu_gate(v0, v1);
    } else {
        if (col[0] < a.n)
            o[col[0]] = v0;
        if (col[1] < a.n)
            o[col[1]] = v1;
    }
}

// This workgroup's item of total * nblk: in expert order, dealt to the XCDs in contiguous ranges
// (workgroup b runs on XCD b % 8), so that an expert's weights and rows are read into one or two
// L2s. False: there is none.
template <int ROWS>
__device__ __forceinline__ bool take_item(const MoeArgs &a, uint32_t b, int nblk, Tile &tile, int &block)
{
    Tiles<ROWS> tiles;
    const uint32_t items = (uint32_t)tiles.total(a.offsets, a.experts, a.pairs) * nblk, per = (items + kXcds - 1) / kXcds;
    const uint32_t item = (b % kXcds) * per + b / kXcds;
    if (b / kXcds >= per || item >= items)
        return false;
    const uint32_t t = item / nblk;
    block = (int)(item - t * nblk);
    tile = tiles.find(a.offsets, a.experts, a.pairs, (int)t);
    return true;
}

// ------------------------------------------------------------------------------------
// Many pairs per expert: 64 pairs, 8 waves, 256 weight rows; gate/up: 128 rows of each, whose h is
// one rotation block, rotated and quantised from LDS at the end. A phase's activations are
// staged, and the next phase's codes and scales loaded, while the last phase computes.
// What bounds it: the fold's vector operations, 16 per lane for a 16x16 tile of one block (convert,
// two products, a sum, 4 values each: 64 cycles) against 32 cycles of matrix instructions.
// ------------------------------------------------------------------------------------
template <int FMT, bool TWO>
struct WideShape {
    static constexpr int kWaves = 8, kThreads = 64 * kWaves;
    static constexpr int kT = 64;                             // pairs of a tile
    static constexpr int kCols = TWO ? 16 * kWaves : 32 * kWaves;
    static constexpr int kPhases = Core<FMT>::kStep / 4;      // phases of a step
    static constexpr int kItems = 4 * kT * 4 / kThreads;      // 32-byte staging items of a thread
    static constexpr int kActBytes = 4 * kT * 128, kDqBytes = 4 * kT * 4;
    static constexpr int kBufBytes = kActBytes + kDqBytes;
    static constexpr int kHPitch = 132;                       // floats of a row of h in LDS
    static constexpr int kLds = 2 * kBufBytes;
    static_assert(kLds >= kT * kHPitch * 4, "h of the tile takes the staging buffers");
};

// NT: 16-pair groups in the tile.
template <int FMT, bool TWO, int NT>
__device__ __forceinline__ void wide_product(const MoeArgs &a, const Tile &tile, int n0, uint8_t *lds)
{
    using C = Core<FMT>;
    using S = WideShape<FMT, TWO>;
    constexpr int R = kTilesPerWave;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 15, g = l >> 4;
    const int nb = a.k / kBlock, np = (nb + C::kStep - 1) / C::kStep * S::kPhases;

    const WeightRows<FMT, TWO> rows(a, tile.expert, n0, wave, i, nb);
    C w[R][4];
    uint16_t sc[R][4];
    auto load_weights = [&](int h, int p) {   // blocks 2h, 2h + 1 of phase p
#pragma unroll
        for (int b = 2 * h; b < 2 * h + 2; ++b) {
            const int at = min(phase_block<FMT>(p, b), nb - 1);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                w[r][b].load(rows.codes[r], rows.coff[r] + g * (C::kBlockBytes / 4), at);
                sc[r][b] = __builtin_amdgcn_raw_buffer_load_b16(rows.scales[r], rows.soff[r], at * 2, 0);
            }
        }
    };
    load_weights(0, 0);
    load_weights(1, 0);

    // staging: a thread takes 32 activations (lane group sg of a block of a pair) at a time, a
    // wave 16 pairs of one block
    const int sg = tid & 3;
    const int8_t *src[S::kItems];
#pragma unroll
    for (int it = 0; it < S::kItems; ++it) {
        const int tok = (tid / 4 + it * (S::kThreads / 4)) % S::kT;
        src[it] = a.q + act_row<TWO>(a, tile.slot + min(tok, tile.rows - 1)) * a.k + sg * 32;
    }
    const float *dsrc = a.dq + act_row<TWO>(a, tile.slot + min(l, tile.rows - 1)) * nb;
    uint4 lo[S::kItems], hi[S::kItems];
    float dv;
    auto stage_load = [&](int p) {
#pragma unroll
        for (int it = 0; it < S::kItems; ++it) {
            const int u = (16 * wave + it * (S::kThreads / 4)) / S::kT;
            const uint4 *q = reinterpret_cast<const uint4 *>(src[it] + (size_t)min(phase_block<FMT>(p, u), nb - 1) * kBlock);
            lo[it] = q[0];
            hi[it] = q[1];
        }
        const int blk = wave < 4 ? phase_block<FMT>(p, wave) : nb;
        dv = blk < nb ? dsrc[blk] : 0.0f;
    };
    auto stage_store = [&](int p) {
        uint8_t *buf = lds + (p & 1) * S::kBufBytes;
#pragma unroll
        for (int it = 0; it < S::kItems; ++it) {
            const int u = (16 * wave + it * (S::kThreads / 4)) / S::kT, tok = (tid / 4 + it * (S::kThreads / 4)) % S::kT;
            v4i *q = reinterpret_cast<v4i *>(buf) + (u * 8 + sg) * S::kT + (pair_row(tok) ^ (2 * sg));
            q[0] = C::acts(lo[it], hi[it], 0);
            q[4 * S::kT] = C::acts(lo[it], hi[it], 1);
        }
        if (wave < 4)
            reinterpret_cast<float *>(buf + S::kActBytes)[wave * S::kT + pair_row(l)] = dv;
    };

    float acc[R][NT][4], part0[R][NT][4], part1[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[r][t][e] = 0.0f;
    stage_load(0);
    stage_store(0);
    __syncthreads();

    for (int p0 = 0; p0 < np; p0 += S::kPhases) {
#pragma unroll
        for (int j = 0; j < S::kPhases; ++j) {
            const int p = p0 + j;
            if (p + 1 < np)
                stage_load(p + 1);
            const uint8_t *buf = lds + (p & 1) * S::kBufBytes;
            const v4i *act = reinterpret_cast<const v4i *>(buf) + g * S::kT;
            const float *d = reinterpret_cast<const float *>(buf + S::kActBytes) + 4 * g;
            float sum[R][NT][4];
            // operands of group x = (half of the phase, 16 pairs): the next group's are read
            // before this one is multiplied and folded (sign's tree has no registers left for it)
            v4i av[2][2][2];
            float dq[2][2][4];
            auto operands = [&](int x) {
                const int h = x / NT, t = x % NT;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int blk = 2 * h + b, slot = 16 * t + (i ^ (2 * g));
                    av[x & 1][b][0] = act[(blk * 2) * 4 * S::kT + slot];
                    av[x & 1][b][1] = act[(blk * 2 + 1) * 4 * S::kT + slot];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dq[x & 1][b][e] = d[blk * S::kT + 16 * t + e];
                }
            };
            constexpr bool kEarly = FMT == TB_FMT_TERNARY2;
            if (kEarly)
                operands(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // blocks 2h, 2h + 1
                v4i wt[R][2][2];
                float s[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        wt[r][b][0] = w[r][2 * h + b].weights(0);
                        wt[r][b][1] = w[r][2 * h + b].weights(1);
                        s[r][b] = half_bits_to_float(sc[r][2 * h + b]);
                    }
                if (p + 1 < np)
                    load_weights(h, p + 1);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int x = h * NT + t;
                    if (!kEarly)
                        operands(x);
                    else if (x + 1 < 2 * NT)
                        operands(x + 1);
                    float term[R][2][4];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            v4i z = {0, 0, 0, 0};
                            z = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[x & 1][b][0], wt[r][b][0], z, 0, 0, 0);
                            z = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[x & 1][b][1], wt[r][b][1], z, 0, 0, 0);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                term[r][b][e] = (s[r][b] * dq[x & 1][b][e]) * (float)z[e];
                        }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = term[r][0][e] + term[r][1][e];
                            sum[r][t][e] = h ? sum[r][t][e] + v : v;
                            // the group's operations are pure: held here, or they sink below
                            // the next groups' operand reads, which then all stay in registers
                            asm volatile("" : "+v"(sum[r][t][e]));
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        add_phase<S::kPhases>(j, sum[r][t][e], part0[r][t][e], part1[r][t][e], acc[r][t][e]);
            if (p + 1 < np)
                stage_store(p + 1);
            __syncthreads();
        }
    }

    if constexpr (TWO) {   // h of the tile through LDS (the staging buffers are free), then its rotation
        float *hs = reinterpret_cast<float *>(lds);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                hs[(16 * t + g + 4 * e) * S::kHPitch + 16 * wave + i] = silu_gate(acc[0][t][e], acc[1][t][e]);
        __syncthreads();
        const int lane16 = tid & 15;
        for (int tok = tid >> 4; tok < tile.rows; tok += S::kThreads / 16) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = hs[tok * S::kHPitch + lane16 * 8 + e];
            uint32_t packed[2];
            float dq;
            int qsum;
            rotquant_regs(v, lane16, a.unit, packed, dq, qsum);
            const size_t slot = tile.slot + tok;
            *reinterpret_cast<uint2 *>(a.qh + slot * a.n + n0 + lane16 * 8) = make_uint2(packed[0], packed[1]);
            if (lane16 == 0)
                a.dqh[slot * (a.n / kBlock) + n0 / kBlock] = dq;
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store_pair<TWO>(a, tile, 16 * t + g + 4 * e, rows.col, acc[0][t][e], acc[1][t][e]);
    }
}

template <int FMT, bool TWO>
__global__ __launch_bounds__(512) void moe_wide_kernel(MoeArgs a, uint32_t first)
{
    using S = WideShape<FMT, TWO>;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    Tile tile;
    int block;
    if (!take_item<S::kT>(a, first + blockIdx.x, (a.n + S::kCols - 1) / S::kCols, tile, block))
        return;
    const int n0 = block * S::kCols;
    if (tile.rows <= 16)
        wide_product<FMT, TWO, 1>(a, tile, n0, lds);
    else if (tile.rows <= 32)
        wide_product<FMT, TWO, 2>(a, tile, n0, lds);
    else if (tile.rows <= 48)
        wide_product<FMT, TWO, 3>(a, tile, n0, lds);
    else
        wide_product<FMT, TWO, 4>(a, tile, n0, lds);
}

// ------------------------------------------------------------------------------------
// Few pairs per expert: 16 pairs, 4 waves of 32 weight rows, so that the experts' rows spread over
// the chip; the weights' way from memory bounds it. A wave loads a whole step of its rows at once,
// 256 bytes per row in four loads of 64 (smaller pieces fetch each 128-byte line several times),
// one step ahead; lane swaps (v_permlane32_swap, sign also v_permlane16_swap) then deal the 16
// bytes that lane group g holds, part of one block, out to all groups. Up to 32 blocks of the
// activations there are are staged at a time.
// ------------------------------------------------------------------------------------
template <int FMT, bool TWO>
struct NarrowShape {
    static constexpr int kWaves = 4, kThreads = 64 * kWaves;
    static constexpr int kT = 16;
    static constexpr int kCols = TWO ? 16 * kWaves : 32 * kWaves;
    static constexpr int kPhases = Core<FMT>::kStep / 4;
    static constexpr int kBlocks = 32;                        // staged at a time
    static constexpr int kActBytes = kBlocks * kT * 128, kDqBytes = kBlocks * kT * 4;
    static constexpr int kLds = kActBytes + kDqBytes;
};

// A step of the lane's row: codes[x] is bytes 64 x + 16 g .. + 15 of the step's 256, scales the step's.
template <int FMT>
struct StepRow {
    static constexpr int kScaleWords = Core<FMT>::kStep / 2;
    uint4 codes[4];
    uint32_t scales[kScaleWords + 1];   // the aligned words from the one that holds the first scale on
    // coff, soff: byte offsets of the row's codes (plus 16 g) and of its first scale's word. All
    // offsets are lane offsets, which the buffers check: what lies past an expert reads zeros.
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t c, __amdgpu_buffer_rsrc_t s, uint32_t coff, uint32_t soff, int nb, int step)
    {
        constexpr int kStep = Core<FMT>::kStep;
        const uint32_t co = coff + step * 256, so = soff + step * (2 * kStep);
#pragma unroll
        for (int x = 0; x < 4; ++x)
            codes[x] = buffer_load16(c, co + x * 64, 0);
        if ((step + 1) * kStep <= nb) {   // the same for all lanes
#pragma unroll
            for (int x = 0; x < kScaleWords; x += 4) {
                const uint4 v = buffer_load16(s, so + x * 4, 0);
                scales[x] = v.x, scales[x + 1] = v.y, scales[x + 2] = v.z, scales[x + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int x = 0; x < kScaleWords; ++x)
                scales[x] = buffer_load_u32(s, so + x * 4);
        }
        scales[kScaleWords] = buffer_load_u32(s, so + kScaleWords * 4);
    }
    // After the loads: each block's codes in all lane groups, scales from bit 0 of scales[0] on.
    // odd: the row's first scale is the upper half of its word
    __device__ __forceinline__ void deal(bool odd)
    {
#pragma unroll
        for (int x = 0; x < kScaleWords; ++x)
            scales[x] = __builtin_amdgcn_alignbit(scales[x + 1], scales[x], odd ? 16 : 0);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            swap32(codes[x].x, codes[x].z);
            swap32(codes[x].y, codes[x].w);
            if (FMT == TB_FMT_SIGN1) {
                swap16(codes[x].x, codes[x].y);
                swap16(codes[x].z, codes[x].w);
            }
        }
    }
    static __device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
    {
        const auto v = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = v[0], b = v[1];
    }
    static __device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
    {
        const auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = v[0], b = v[1];
    }
    __device__ __forceinline__ float scale(int b) const { return half_bits_to_float((uint16_t)(scales[b / 2] >> (16 * (b % 2)))); }
    // Ternary: codes[x] holds blocks 2x (x, y) and 2x + 1 (z, w), in lane group g words (0, 4, 2, 6)[g]
    // and the one after. Sign: word b of codes[x] is word g of block 4x + b.
    __device__ __forceinline__ Core<FMT> block(int b) const
    {
        Core<FMT> c;
        if constexpr (FMT == TB_FMT_TERNARY2) {
            c.w = b % 2 ? make_uint2(codes[b / 2].z, codes[b / 2].w) : make_uint2(codes[b / 2].x, codes[b / 2].y);
        } else {
            const uint4 v = codes[b / 4];
            c.w = b % 4 == 0 ? v.x : b % 4 == 1 ? v.y : b % 4 == 2 ? v.z : v.w;
        }
        return c;
    }
};

// NE: elements that hold pairs.
template <int FMT, bool TWO, int NE>
__device__ __forceinline__ void narrow_product(const MoeArgs &a, const Tile &tile, int n0, uint8_t *lds)
{
    using C = Core<FMT>;
    using S = NarrowShape<FMT, TWO>;
    constexpr int R = kTilesPerWave;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 15, g = l >> 4;
    const int nb = a.k / kBlock, steps = (nb + C::kStep - 1) / C::kStep;

    const WeightRows<FMT, TWO> rows(a, tile.expert, n0, wave, i, nb);
    StepRow<FMT> w[2][R];
    auto load_weights = [&](int j, int step) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            w[j][r].load(rows.codes[r], rows.scales[r], rows.coff[r] + g * 16, rows.soff[r] & ~3u, nb, step);
    };
    load_weights(0, 0);

    // staging: 128 threads for the 4 lane groups (32 activations each) of 32 blocks of a pair
    const int sg = tid & 3, u = (tid & 127) >> 2;
    // the lane group that reads the words of staging group sg
    const int to = FMT == TB_FMT_TERNARY2 ? (sg & 1) << 1 | sg >> 1 : sg;
    auto stage = [&](int c0) {
        const int blk = c0 + u, at = min(blk, nb - 1);
#pragma unroll 4
        for (int tok = wave >> 1; tok < tile.rows; tok += S::kThreads / 128) {
            const size_t row = act_row<TWO>(a, tile.slot + tok);
            const uint4 *p = reinterpret_cast<const uint4 *>(a.q + row * a.k + (size_t)at * kBlock + sg * 32);
            const uint4 lo = p[0], hi = p[1];
            const float dq = blk < nb ? a.dq[row * nb + at] : 0.0f;
            v4i *o = reinterpret_cast<v4i *>(lds) + (u * 8 + to) * S::kT + (pair_row(tok) ^ (2 * to));
            o[0] = C::acts(lo, hi, 0);
            o[4 * S::kT] = C::acts(lo, hi, 1);
            if (sg == 0)
                reinterpret_cast<float *>(lds + S::kActBytes)[u * S::kT + pair_row(tok)] = dq;
        }
    };
    if (steps > 1)
        load_weights(1, 1);
    stage(0);
    __syncthreads();

    float acc[R][NE];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < NE; ++e)
            acc[r][e] = 0.0f;
    for (int s0 = 0; s0 < steps; s0 += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int step = s0 + j;
            if (step < steps) {   // the same for all waves
                constexpr int kPer = S::kBlocks / C::kStep;   // steps staged at a time
                if (step && step % kPer == 0) {
                    __syncthreads();
                    stage(step * C::kStep);
                    __syncthreads();
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    w[j][r].deal(rows.soff[r] & 2);
                const int u0 = step % kPer * C::kStep;
                const v4i *act = reinterpret_cast<const v4i *>(lds) + (u0 * 8 + g) * S::kT + (i ^ (2 * g));
                const float *d = reinterpret_cast<const float *>(lds + S::kActBytes) + u0 * S::kT + 4 * g;
                float part0[R][NE], part1[R][NE];
#pragma unroll
                for (int q = 0; q < S::kPhases; ++q) {
                    float sum[R][NE];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float term[R][2][NE];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int x = 4 * q + 2 * h + b, blk = x ? C::kStep - x : 0;
                            const v4i a0 = act[blk * 8 * S::kT], a1 = act[(blk * 8 + 4) * S::kT];
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                const C core = w[j][r].block(blk);
                                v4i z = {0, 0, 0, 0};
                                z = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, core.weights(0), z, 0, 0, 0);
                                z = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, core.weights(1), z, 0, 0, 0);
                                const float s = w[j][r].scale(blk);
#pragma unroll
                                for (int e = 0; e < NE; ++e)
                                    term[r][b][e] = (s * d[blk * S::kT + e]) * (float)z[e];
                            }
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int e = 0; e < NE; ++e) {
                                const float v = term[r][0][e] + term[r][1][e];
                                sum[r][e] = h ? sum[r][e] + v : v;
                            }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            add_phase<S::kPhases>(q, sum[r][e], part0[r][e], part1[r][e], acc[r][e]);
                            asm volatile("" : "+v"(sum[r][e]));
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (step + 2 < steps)
                    load_weights(j, step + 2);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < NE; ++e)
        store_pair<TWO>(a, tile, g + 4 * e, rows.col, acc[0][e], acc[1][e]);
}

template <int FMT, bool TWO>
__global__ __launch_bounds__(256) void moe_narrow_kernel(MoeArgs a, uint32_t first)
{
    using S = NarrowShape<FMT, TWO>;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    Tile tile;
    int block;
    if (!take_item<S::kT>(a, first + blockIdx.x, (a.n + S::kCols - 1) / S::kCols, tile, block))
        return;
    const int n0 = block * S::kCols;
    if (tile.rows <= 4)
        narrow_product<FMT, TWO, 1>(a, tile, n0, lds);
    else if (tile.rows <= 8)
        narrow_product<FMT, TWO, 2>(a, tile, n0, lds);
    else
        narrow_product<FMT, TWO, 4>(a, tile, n0, lds);
}

// rotquant of the slots in use: rows [0, offsets[experts]) of h. One 128-block per 16 lanes.
constexpr int kRotThreads = 256;
__global__ __launch_bounds__(kRotThreads) void moe_rotquant_kernel(const float *__restrict__ h, int nb, int pairs,
                                                                   const int32_t *__restrict__ used,
                                                                   int8_t *__restrict__ q, float *__restrict__ dq, float unit)
{
    const size_t blocks = (size_t)min(max(*used, 0), pairs) * nb, stride = (size_t)gridDim.x * (kRotThreads / 16);
    for (size_t b = (size_t)blockIdx.x * (kRotThreads / 16) + (threadIdx.x >> 4); b < blocks; b += stride)
        rotquant16<false>(h + b * kBlock, q + b * kBlock, dq + b, threadIdx.x & 15, unit);
}

// out[t] = sum over j, ascending, of weights[t][j] * y[t topk + j], leaving out pairs of no expert.
template <class T>
__device__ __forceinline__ void put(T *p, float v)
{
    p->bits = (uint16_t)tbr::pack(v, 0.0f, T());
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }

template <class T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float *__restrict__ y, const float *__restrict__ weights,
                                                          const int32_t *__restrict__ ids, int tokens, int topk,
                                                          int experts, int n, T *__restrict__ out)
{
    const size_t total = (size_t)tokens * n, stride = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const size_t t = i / n, c = i % n;
        float s = 0.0f;
        for (int j = 0; j < topk; ++j) {
            const size_t p = t * topk + j;
            if ((unsigned)ids[p] < (unsigned)experts)
                s = fmaf(weights[p], y[p * n + c], s);
        }
        put(out + i, s);
    }
}

size_t block_bytes(int fmt) { return fmt == TB_FMT_TERNARY2 ? 32 : 16; }
size_t codes_bytes(const tb_experts *w) { return (size_t)w->experts * w->n * (w->k / kBlock) * block_bytes(w->fmt); }
size_t scales_bytes(const tb_experts *w) { return (size_t)w->experts * w->n * (w->k / kBlock) * 2; }

int check_experts(const tb_experts *w)
{
    if (!w || !w->codes || !w->scales || w->experts < 1 || w->n < 1 || w->k < kBlock || w->k % kBlock)
        return TB_EINVAL;
    if (w->fmt == TB_FMT_SIGN1_RI4)
        return TB_EUNSUPPORTED;
    if (w->fmt != TB_FMT_TERNARY2 && w->fmt != TB_FMT_SIGN1)
        return TB_EINVAL;
    if (!tbh::aligned16(w->codes) || !tbh::aligned16(w->scales))
        return TB_EALIGN;
    // buffer addressing: each expert's arrays must stay below 2 GiB
    const size_t blocks = (size_t)w->n * (w->k / kBlock);
    return w->experts > kMaxExperts || blocks * block_bytes(w->fmt) >= ((size_t)1 << 31) ? TB_EUNSUPPORTED : TB_OK;
}

// tokens * topk pairs: TB_OK if they can be counted in 31 bits
int check_pairs(int tokens, int topk)
{
    if (tokens < 1 || topk < 1)
        return TB_EINVAL;
    return (int64_t)tokens * topk > 0x7fffffc0 ? TB_EUNSUPPORTED : TB_OK;
}

template <class S>
int launch_tiles(const MoeArgs &a, void (*kernel)(MoeArgs, uint32_t), hipStream_t stream)
{
    // every expert's last tile may be partly filled, and no tile is empty
    const int64_t tiles = std::min<int64_t>(a.pairs, (int64_t)a.pairs / S::kT + a.experts);
    const int64_t total = tiles * ((a.n + S::kCols - 1) / S::kCols);
    if (total > 0x7fffffff)
        return TB_EUNSUPPORTED;
    for (int64_t first = 0; first < total; first += kMaxGrid) {
        const int64_t grid = std::min<int64_t>((total - first + kXcds - 1) / kXcds * kXcds, kMaxGrid);
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(S::kThreads), 0, stream, a, (uint32_t)first);
        if (hipGetLastError() != hipSuccess)
            return TB_EHIP;
    }
    return TB_OK;
}

// Wide tiles from an average of 16 pairs per expert on.
bool wide_tiles(int pairs, int experts) { return (int64_t)pairs >= (int64_t)experts * 16; }

template <int FMT, bool TWO>
int launch_product_as(const MoeArgs &a, hipStream_t stream)
{
    return wide_tiles(a.pairs, a.experts) ? launch_tiles<WideShape<FMT, TWO>>(a, moe_wide_kernel<FMT, TWO>, stream)
                                          : launch_tiles<NarrowShape<FMT, TWO>>(a, moe_narrow_kernel<FMT, TWO>, stream);
}
template <bool TWO>
int launch_product(const MoeArgs &a, int fmt, hipStream_t stream)
{
    return fmt == TB_FMT_TERNARY2 ? launch_product_as<TB_FMT_TERNARY2, TWO>(a, stream) : launch_product_as<TB_FMT_SIGN1, TWO>(a, stream);
}

template <class T>
int launch_combine(const float *y, const float *weights, const int32_t *ids, int tokens, int topk, int experts, int n,
                   void *out, hipStream_t stream)
{
    const int grid = (int)std::min<size_t>(((size_t)tokens * n + 255) / 256, kMaxGrid);
    hipLaunchKernelGGL(moe_combine_kernel<T>, dim3(grid), dim3(256), 0, stream, y, weights, ids, tokens, topk, experts, n,
                       static_cast<T *>(out));
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

}  // namespace

extern "C" {

int tb_moe_plan(const int32_t *ids, int tokens, int topk, int experts, int32_t *offsets, int32_t *order, void *stream)
{
    int rc = check_pairs(tokens, topk);
    if (rc == TB_EINVAL || experts < 1)
        return TB_EINVAL;
    if (rc || experts > kMaxExperts)
        return TB_EUNSUPPORTED;
    const int pairs = tokens * topk;
    const tbh::Arg a[] = {{ids, (size_t)pairs * 4, false}, {offsets, (size_t)(experts + 1) * 4, true}, {order, (size_t)pairs * 4, true}};
    if ((rc = tbh::check_args(a)))
        return rc;
    hipLaunchKernelGGL(moe_plan_kernel, dim3(experts + 1), dim3(kPlanThreads), 0, static_cast<hipStream_t>(stream), ids, pairs,
                       experts, offsets, order);
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

int tb_moe_gateup_silu(const tb_experts *wg, const tb_experts *wu, const int8_t *q, const float *dq, int tokens, int topk,
                       const int32_t *offsets, const int32_t *order, float *h, int8_t *qh, float *dqh, void *stream)
{
    int rc;
    if ((rc = check_experts(wg)) || (rc = check_experts(wu)) || (rc = check_pairs(tokens, topk)))
        return rc;
    if (wg->experts != wu->experts || wg->n != wu->n || wg->k != wu->k || wg->fmt != wu->fmt || wg->n % kBlock)
        return TB_EINVAL;
    const size_t pairs = (size_t)tokens * topk, nb = wg->k / kBlock, n = wg->n;
    const tbh::Arg a[] = {{wg->codes, codes_bytes(wg), false}, {wg->scales, scales_bytes(wg), false},
                          {wu->codes, codes_bytes(wu), false}, {wu->scales, scales_bytes(wu), false},
                          {q, (size_t)tokens * wg->k, false},  {dq, (size_t)tokens * nb * 4, false},
                          {offsets, (size_t)(wg->experts + 1) * 4, false}, {order, pairs * 4, false},
                          {h, pairs * n * 4, true}, {qh, pairs * n, true}, {dqh, pairs * (n / kBlock) * 4, true}};
    if ((rc = tbh::check_args(a)))
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const MoeArgs args = {{static_cast<const uint8_t *>(wg->codes), static_cast<const uint8_t *>(wu->codes)},
                          {wg->scales, wu->scales}, wg->experts, wg->n, wg->k, q, dq, offsets, order, (int)pairs, topk, h, qh, dqh,
                          tbh::dq_unit()};
    if ((rc = launch_product<true>(args, wg->fmt, st)) || wide_tiles((int)pairs, wg->experts))
        return rc;
    const size_t blocks = pairs * (n / kBlock);
    const int grid = (int)std::min<size_t>((blocks + kRotThreads / 16 - 1) / (kRotThreads / 16), kMaxGrid);
    hipLaunchKernelGGL(moe_rotquant_kernel, dim3(grid), dim3(kRotThreads), 0, st, h, (int)(n / kBlock), (int)pairs,
                       offsets + wg->experts, qh, dqh, tbh::dq_unit());
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

int tb_moe_down(const tb_experts *wd, const int8_t *qh, const float *dqh, int pairs, const int32_t *offsets,
                const int32_t *order, float *y, void *stream)
{
    int rc;
    if ((rc = check_experts(wd)) || (rc = check_pairs(pairs, 1)))
        return rc;
    const tbh::Arg a[] = {{wd->codes, codes_bytes(wd), false}, {wd->scales, scales_bytes(wd), false},
                          {qh, (size_t)pairs * wd->k, false}, {dqh, (size_t)pairs * (wd->k / kBlock) * 4, false},
                          {offsets, (size_t)(wd->experts + 1) * 4, false}, {order, (size_t)pairs * 4, false},
                          {y, (size_t)pairs * wd->n * 4, true}};
    if ((rc = tbh::check_args(a)))
        return rc;
    const MoeArgs args = {{static_cast<const uint8_t *>(wd->codes), nullptr}, {wd->scales, nullptr}, wd->experts, wd->n, wd->k,
                          qh, dqh, offsets, order, pairs, 1, y, nullptr, nullptr, 0.0f};
    return launch_product<false>(args, wd->fmt, static_cast<hipStream_t>(stream));
}

int tb_moe_combine(const float *y, const float *weights, const int32_t *ids, int tokens, int topk, int experts, int n,
                   void *out, int dtype, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    int rc = check_pairs(tokens, topk);
    if (rc == TB_EINVAL || experts < 1 || n < 1 || !eb)
        return TB_EINVAL;
    if (rc || experts > kMaxExperts)
        return TB_EUNSUPPORTED;
    const size_t pairs = (size_t)tokens * topk;
    const tbh::Arg a[] = {{y, pairs * n * 4, false}, {weights, pairs * 4, false}, {ids, pairs * 4, false}, {out, (size_t)tokens * n * eb, true}};
    if ((rc = tbh::check_args(a)))
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case TB_F32: return launch_combine<float>(y, weights, ids, tokens, topk, experts, n, out, st);
    case TB_BF16: return launch_combine<tbr::Bf16>(y, weights, ids, tokens, topk, experts, n, out, st);
    default: return launch_combine<tbr::F16>(y, weights, ids, tokens, topk, experts, n, out, st);
    }
}

}  // extern "C"
