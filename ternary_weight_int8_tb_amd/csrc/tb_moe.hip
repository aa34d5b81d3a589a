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
// list. Bound: the latency of the loads (8 ids of 64 experts 3.6 us, 32768 ids 8.9).
// ------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanLoads = 4;   // loads of 256 ids that a wave has in flight

__global__ __launch_bounds__(kPlanThreads) void moe_plan_kernel(const int32_t *__restrict__ ids, int pairs,
                                                                int experts, int32_t *__restrict__ offsets,
                                                                int32_t *__restrict__ order)
{
    __shared__ int less_s[kPlanWaves], same_s[kPlanWaves];
    const int e = blockIdx.x, waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // each wave takes a contiguous range of whole groups of 256 ids, lane l ids 4 l .. 4 l + 3
    const unsigned groups = (pairs - 1) / 256 + 1;   // below 2^23: times 16 waves, it fits
    const int g0 = groups * wave / waves, g1 = groups * (wave + 1) / waves;
    auto read = [&](int g, int (&id)[4]) {
        const int64_t p = (int64_t)g * 256 + lane * 4;
        if (g < g1 && p + 4 <= pairs) {
            const int4 v = *reinterpret_cast<const int4 *>(ids + p);
            id[0] = v.x, id[1] = v.y, id[2] = v.z, id[3] = v.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                id[c] = g < g1 && p + c < pairs ? ids[p + c] : -1;
        }
    };
    int less = 0, same = 0;
    for (int g = g0; g < g1; g += kPlanLoads) {
        int id[kPlanLoads][4];
#pragma unroll
        for (int x = 0; x < kPlanLoads; ++x)
            read(g + x, id[x]);
#pragma unroll
        for (int x = 0; x < kPlanLoads; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                less += __popcll(__ballot((unsigned)id[x][c] < (unsigned)e));
                same += __popcll(__ballot(id[x][c] == e));
            }
    }
    if (lane == 0) {
        less_s[wave] = less;
        same_s[wave] = same;
    }
    __syncthreads();
    int start = 0, before = 0;
    for (int w = 0; w < waves; ++w) {
        start += less_s[w];
        before += w < wave ? same_s[w] : 0;
    }
    if (threadIdx.x == 0)
        offsets[e] = start;
    if (e == experts || same == 0)
        return;
    int at = start + before;
    const uint64_t lower = (1ull << lane) - 1;
    for (int g = g0; g < g1; g += kPlanLoads) {
        int id[kPlanLoads][4];
#pragma unroll
        for (int x = 0; x < kPlanLoads; ++x)
            read(g + x, id[x]);
#pragma unroll
        for (int x = 0; x < kPlanLoads; ++x) {
            int ahead = 0, all = 0;   // of this group: in lower lanes, and in all
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint64_t mask = __ballot(id[x][c] == e);
                ahead += __popcll(mask & lower);
                all += __popcll(mask);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (id[x][c] == e)
                    order[at + ahead++] = (g + x) * 256 + lane * 4 + c;
            at += all;
        }
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
        const int src = max(__ffsll((unsigned long long)__ballot(before + upto > t)) - 1, 0);
        const int r0 = (t - before - __builtin_amdgcn_readlane(upto - tiles, src)) * ROWS;
        // cut once more: where offsets are no plan's, the numbers of tiles may not fit 32 bits
        const int slot = min(max(__builtin_amdgcn_readlane(lo, src) + r0, 0), pairs - 1);
        return {min(e0 + src, experts - 1), slot, min(max(min(ROWS, __builtin_amdgcn_readlane(count, src) - r0), 1), pairs - slot)};
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

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v8i join(v4i a, v4i b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

template <int FMT>
struct Core;
// Ternary: of a block's 8 code words lane group g holds words 2g, 2g + 1; matrix instruction s
// takes word 2g + s, whose decoded bytes are the weights {j, j+4, j+8, j+12}.
template <>
struct Core<TB_FMT_TERNARY2> {
    static constexpr int kStep = 8;        // blocks of a step
    static constexpr int kBlockBytes = 32;
    uint2 w;
    __device__ __forceinline__ v4i weights(int s) const
    {
        uint32_t a, b, c, d;
        decode_ternary(s ? w.y : w.x, a, b, c, d);
        return v4i{(int)a, (int)b, (int)c, (int)d};
    }
    // As 4-bit floats 2 w: word x makes the registers of its even and of its odd weights. A code's
    // upper bit is the sign, the difference of its bits the 2: 3 is -0. Six operations for 16 weights.
    __device__ __forceinline__ v8i floats() const
    {
        v8i o = {};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t v = x ? w.y : w.x, r = (v & 0xAAAAAAAAu) | ((v ^ (v >> 1)) & 0x55555555u);
            o[2 * x] = (int)((r << 2) & 0xCCCCCCCCu);
            o[2 * x + 1] = (int)(r & 0xCCCCCCCCu);
        }
        return o;
    }
};
// Sign: lane group g holds word g of a block's 4, the weights 32 g .. 32 g + 31; bit j of its
// bytes are the weights {j, j+8, j+16, j+24}. Instruction s takes j = 4 s .. 4 s + 3, as +1 / -1.
template <>
struct Core<TB_FMT_SIGN1> {
    static constexpr int kStep = 16;
    static constexpr int kBlockBytes = 16;
    uint32_t w;
    __device__ __forceinline__ v4i weights(int s) const
    {
        v4i o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = (int)__builtin_amdgcn_perm(0u, 0x000001FFu, (w >> (4 * s + j)) & 0x01010101u);
        return o;
    }
    // As 4-bit floats -2 w (a set bit, +1, is the sign): register x holds the weights 4 n + x. Seven
    // operations for 32 weights.
    __device__ __forceinline__ v8i floats() const
    {
        v8i o = {};
#pragma unroll
        for (int x = 0; x < 4; ++x)
            o[x] = (int)(((w << (3 - x)) & 0x88888888u) | 0x44444444u);
        return o;
    }
};

// rotquant_regs of a block of h held by 16 lanes, but for a block whose rotation is not finite: codes 0
// and dq a NaN. rotquant_regs' maximum passes over a NaN, and would make a block of zeros of it.
__device__ __forceinline__ void rotquant_h(float (&v)[8], int lane16, float unit, uint32_t (&packed)[2], float &dq)
{
    int qsum;
    rotquant_regs(v, lane16, unit, packed, dq, qsum);   // v is the rotation now
    float z = 0.0f;   // 0 times an infinity or a NaN is a NaN
#pragma unroll
    for (int e = 0; e < 8; ++e)
        z = fmaf(v[e], 0.0f, z);
    const bool bad = __ballot(z != 0.0f) >> (threadIdx.x & 48) & 0xffff;
    packed[0] = bad ? 0u : packed[0];
    packed[1] = bad ? 0u : packed[1];
    dq = bad ? NAN : dq;
}

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
//   * A wave owns tiles of 16 weight rows through all of k; nothing of a row crosses waves. The
//     blocks of a step are taken in the order in which the step's tree adds them: 0, last, last - 1,
//     last - 2, then the next four downwards. Such a phase of 4 blocks leaves one partial sum, the tree
//     above it one register set per level.
//   * Activations are staged in LDS as the operands read them: byte-transposed, 16 bytes per lane,
//     in planes (block, instruction, lane group) of A rows.
//   * Blocks past the end of k have dq = 0 and count +0.
// ------------------------------------------------------------------------------------
// Stages piece `unit` (16 activations) of block u of A row `row`: lanes 8 x .. 8 x + 7 hold the pieces of
// a block. A piece goes to the plane (block, instruction s, lane group g) whose code word it meets
// (StepRow), row ^ g of it. A plane has T rows of 16 bytes, T a multiple of 16: lane groups g and g + 1
// then read the same 16 columns of banks in the halves that one LDS cycle serves, without conflict
// (a plane of 49 rows cost a cycle of conflict for each of the reads), and the exchange within four
// rows spreads the pieces that a wave stages.
template <int FMT, int T>
__device__ __forceinline__ void stage_piece(uint8_t *lds, int u, int row, int unit, uint4 v)
{
    v4i o;
    int s, g;
    if constexpr (FMT == TB_FMT_TERNARY2) {
        // word w: instruction w % 2, lane group 0, 2, 1, 3 for words 0, 2, 4, 6
        s = unit & 1;
        g = (unit & 2) | unit >> 2;
        o = transpose4(v.x, v.y, v.z, v.w);
    } else {
        // a word meets two pieces: the even lane makes instruction 0's bytes, the odd lane 1's
        s = unit & 1;
        g = unit >> 1;
        const uint32_t x = row_xor(s ? v.x : v.y, 1), y = row_xor(s ? v.z : v.w, 1);
        o = s ? transpose4(x, y, v.y, v.w) : transpose4(v.x, v.z, x, y);
    }
    reinterpret_cast<v4i *>(lds)[(u * 8 + s * 4 + g) * T + (row ^ g)] = o;
}

// For the few-pairs kernel: the activations as the sum of two 8-bit floats (4 exponent bits), each with
// the sign and half of the magnitude: |q| = 16 h + l, and the bytes 0 .. 15 are the floats
// 0 .. 15 x 2^-9, for the numbers below 2^-6 and the binade from there on are spaced alike. So one
// instruction of 128 elements, whose operands carry powers of two as scales, multiplies a block by
// 4-bit weights, which cost a third of the operations that bytes cost to make. Its sums are whole
// numbers below 2^24, exact in fp32, and need no conversion.
// The instruction's 8-bit operand: lane group g's 16-byte chunks c = 0, 1 meet the 4-bit registers
// 2 (g % 2) and the next of lane group 2 c + g / 2. So piece s of lane group G goes to plane
// (c, g) = (G / 2, 2 (G % 2) + s) of the block. Rows 2 NE (t % 4) + 2 (t / 4) and the next hold pair
// t's lower and upper halves, so that both sums end in one lane. Row r stands at r ^ 2 g: the pieces
// that a wave stages spread over the banks.
// Sign: the 4-bit floats are the negatives of the weights, so the activations' signs are turned.
template <int FMT, int NE>
__device__ __forceinline__ void stage_split(uint8_t *lds, int u, int t, int unit, uint4 v)
{
    uint32_t x[4];
    int G;
    if constexpr (FMT == TB_FMT_TERNARY2) {
        G = (unit & 2) | unit >> 2;   // words 0, 2, 4, 6 are held by lane groups 0, 2, 1, 3 (StepRow)
        x[0] = __builtin_amdgcn_perm(v.y, v.x, 0x06040200u), x[1] = __builtin_amdgcn_perm(v.w, v.z, 0x06040200u);
        x[2] = __builtin_amdgcn_perm(v.y, v.x, 0x07050301u), x[3] = __builtin_amdgcn_perm(v.w, v.z, 0x07050301u);
    } else {
        // a code word meets two pieces: the even lane makes registers 0 and 1's chunk, the odd one the other
        G = unit >> 1;
        const bool odd = unit & 1;
        const v4i o = transpose4(v.x, v.y, v.z, v.w);
        const uint32_t p = row_xor((uint32_t)(odd ? o[0] : o[2]), 1), q = row_xor((uint32_t)(odd ? o[1] : o[3]), 1);
        x[0] = odd ? p : o[0], x[1] = odd ? o[2] : p, x[2] = odd ? q : o[1], x[3] = odd ? o[3] : q;
    }
    v4i low, high;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t sign = x[j] & 0x80808080u, ones = sign >> 7, mag = (x[j] ^ ((sign - ones) | sign)) + ones;
        const uint32_t top = FMT == TB_FMT_SIGN1 ? sign ^ 0x80808080u : sign;
        low[j] = (int)((mag & 0x0F0F0F0Fu) | top);
        high[j] = (int)(((mag >> 4) & 0x0F0F0F0Fu) | top);
    }
    const int c = G >> 1, g = 2 * (G & 1) + (unit & 1);
    const int row = 2 * NE * (t & 3) + 2 * (t >> 2);
    v4i *plane = reinterpret_cast<v4i *>(lds) + (u * 8 + c * 4 + g) * (8 * NE);
    plane[row ^ (2 * g)] = low;
    plane[(row + 1) ^ (2 * g)] = high;
}

// A row of a tile's pair t
__device__ __forceinline__ int pair_row(int t) { return (t & ~15) | (t & 3) << 2 | (t >> 2 & 3); }

// The activation row of a slot.
template <bool TWO>
__device__ __forceinline__ size_t act_row(const MoeArgs &a, int slot)
{
    return TWO ? (unsigned)min(max(a.order[slot], 0), a.pairs - 1) / (unsigned)a.topk : (unsigned)slot;
}

// A lane's weight row: column `at` of the output, of matrix m. Rows past n read the last one and are
// not stored.
template <int FMT>
struct WeightRows {
    __amdgpu_buffer_rsrc_t codes, scales;
    uint32_t coff, soff;   // byte offsets of the row's codes and scales
    int col;
    uint32_t base;
    __device__ __forceinline__ WeightRows(const MoeArgs &a, int m, int expert, int at, int nb)
    {
        col = at;
        const uint32_t row = min(at, a.n - 1);
        const size_t first = (size_t)expert * a.n * nb, blocks = (size_t)a.n * nb;
        codes = buffer_rsrc((m ? a.codes[1] : a.codes[0]) + first * Core<FMT>::kBlockBytes, (uint32_t)(blocks * Core<FMT>::kBlockBytes));
        coff = row * (nb * Core<FMT>::kBlockBytes);
        // the scales buffer starts, and ends, at whole words
        const size_t odd = first & 1;
        scales = buffer_rsrc((m ? a.scales[1] : a.scales[0]) + (first - odd), (uint32_t)((blocks + odd + 1) / 2 * 4));
        soff = (row * nb + (uint32_t)odd) * 2;
        base = (uint32_t)odd * 2;
    }
    __device__ __forceinline__ void move(const MoeArgs &a, int at, int nb)
    {
        const uint32_t row = min(at, a.n - 1);
        coff = row * (nb * Core<FMT>::kBlockBytes);
        soff = row * nb * 2 + base;
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

// The output row of pair `tok` of the tile (gate/up: h of its slot); null: there is none.
template <bool TWO>
__device__ __forceinline__ float *pair_out(const MoeArgs &a, const Tile &tile, int tok)
{
    if (tok >= tile.rows)
        return nullptr;
    const int row = TWO ? tile.slot + tok : a.order[tile.slot + tok];
    return (unsigned)row < (unsigned)a.pairs ? a.out + (size_t)row * a.n : nullptr;
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

// A step of the lane's row, loaded as a whole: 256 bytes of codes in four loads of 64 per row (loads of
// a block, 8 bytes a lane, kept the address unit busy for 40% of the wide kernel's time, and
// fetched each 128-byte line several times). codes[x] is bytes 64 x + 16 g .. + 15 of the step's 256.
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
    // After the loads, by lane swaps: each block's codes, 16 bytes of which one lane group loaded, in
    // all groups; scales from bit 0 of scales[0] on.
    // odd: the row's first scale is the upper half of its word; left: blocks from this step's first on
    __device__ __forceinline__ void deal(bool odd, int left)
    {
#pragma unroll
        for (int x = 0; x < kScaleWords; ++x)
            scales[x] = __builtin_amdgcn_alignbit(scales[x + 1], scales[x], odd ? 16 : 0);
        if (left < Core<FMT>::kStep)   // what follows are the next row's: 0 times an infinity is no 0
#pragma unroll
            for (int x = 0; x < kScaleWords; ++x)
                scales[x] &= 2 * x + 1 < left ? 0xffffffffu : 2 * x < left ? 0xffffu : 0u;
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

// ------------------------------------------------------------------------------------
// Many pairs per expert: 48 pairs, 16 waves of 16 weight rows; gate/up: 128 rows of each, whose h is
// one rotation block, rotated and quantised from LDS at the end. Up to 16 blocks of the pairs'
// activations stay in LDS; a workgroup takes several row groups with them, and while they fit
// (k <= 2048) its waves run through them without meeting. The next step's codes are loaded while the
// last half phase of a step is multiplied.
// Bound: vector operations, 34 for a 16x16 tile of one block: 16 of the fold (a difference, two
// products, a sum, for 4 values), 6 of the decode, shared by 48 pairs, 8 of SiLU and rotation. 32768
// pairs over 64 experts, ternary, 2 x 1024 x 2048: 314 to 340 us by the card, 143 M of them, one every 4.3 cycles of a SIMD;
// down 198 to 209 us. Sign: 369 to 378 and 320 to 327 us.
// 16 waves per CU, because a wave alone issues a vector operation every 5 to 6 cycles and four of a
// SIMD together one every 2.3. The 128 registers that this leaves a wave do not hold everything: 15
// (ternary) and 47 (sign) of gate/up and 4 and 30 of down lie in scratch memory. Ternary reads them back
// outside the loop over the steps but for one; sign reads 28 and 24 within its three loops (of 1, 2 and 3 groups of
// pairs), which is part of why it is slower, by how much is not known.
// ------------------------------------------------------------------------------------
template <int FMT, bool TWO>
struct WideShape {
    static constexpr int kWaves = 16, kThreads = 64 * kWaves;
    static constexpr int kT = 48;                             // pairs of a tile
    static constexpr int kPairsPerWave = kT / kWaves;         // that a wave stages
    static constexpr int kCols = TWO ? 8 * kWaves : 16 * kWaves;
    static constexpr int kPhases = Core<FMT>::kStep / 4;      // phases of a step
    static constexpr int kBlocks = 16;                        // staged at a time
    static constexpr int kActBytes = kBlocks * 8 * kT * 16, kDqBytes = kBlocks * kT * 4;
    static constexpr int kHPitch = 132;                       // floats of a row of g or u in LDS
    static constexpr int kLds = kActBytes + kDqBytes + (TWO ? 2 * kT * kHPitch * 4 : 0);
    static_assert(kLds <= 160 * 1024 && kBlocks * kT <= kThreads, "");
};

// The block sum's fp32 value comes from the integer accumulator by one subtraction: it starts at
// the bits of 1.5 * 2^23, so that its bits are those of 1.5 * 2^23 + sum (|sum| <= 128 * 127 < 2^22).
constexpr int kMagicBits = 0x4B400000;
constexpr float kMagic = 12582912.0f;

// Row groups [j0, j1) of the tile's expert. NT: 16-pair groups in the tile.
template <int FMT, bool TWO, int NT>
__device__ __forceinline__ void wide_product(const MoeArgs &a, const Tile &tile, int j0, int j1, uint8_t *lds)
{
    using C = Core<FMT>;
    using S = WideShape<FMT, TWO>;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 15, g = l >> 4;
    const int nb = a.k / kBlock, steps = (nb + C::kStep - 1) / C::kStep;
    const int col0 = 16 * (TWO ? wave & 7 : wave) + i, mat = TWO ? wave >> 3 : 0;
    float *dq_s = reinterpret_cast<float *>(lds + S::kActBytes);

    StepRow<FMT> w;
    WeightRows<FMT> rows(a, mat, tile.expert, j0 * S::kCols + col0, nb);
    auto load_weights = [&](int step) { w.load(rows.codes, rows.scales, rows.coff + g * 16, rows.soff & ~3u, nb, step); };
    load_weights(0);

    // blocks [c0, c0 + kBlocks): a wave takes kPairsPerWave pairs, 1 KB of each at a time
    auto stage = [&](int c0) {
        uint4 v[S::kPairsPerWave][2];
#pragma unroll
        for (int t = 0; t < S::kPairsPerWave; ++t) {
            const int tok = min(wave * S::kPairsPerWave + t, tile.rows - 1);
            const int8_t *src = a.q + act_row<TWO>(a, tile.slot + tok) * a.k;
#pragma unroll
            for (int h = 0; h < 2; ++h)   // pieces past the end of k read its last block
                v[t][h] = *reinterpret_cast<const uint4 *>(src + min((c0 + 8 * h) * kBlock + l * 16, (nb - 1) * kBlock + (l & 7) * 16));
        }
        float d = 0.0f;
        if (tid < S::kBlocks * S::kT && c0 + tid % S::kBlocks < nb)
            d = a.dq[act_row<TWO>(a, tile.slot + min(tid / S::kBlocks, tile.rows - 1)) * nb + c0 + tid % S::kBlocks];
#pragma unroll
        for (int t = 0; t < S::kPairsPerWave; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                stage_piece<FMT, S::kT>(lds, 8 * h + (l >> 3), pair_row(wave * S::kPairsPerWave + t), l & 7, v[t][h]);
        if (tid < S::kBlocks * S::kT)
            dq_s[tid % S::kBlocks * S::kT + pair_row(tid / S::kBlocks)] = d;
    };
    stage(0);
    __syncthreads();

    for (int jn = j0; jn < j1; ++jn) {
        const int n0 = jn * S::kCols;
        float acc[NT][4], part0[NT][4], part1[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[t][e] = 0.0f;
        for (int step = 0; step < steps; ++step) {
            const int u0 = step * C::kStep % S::kBlocks;
            if (nb > S::kBlocks && u0 == 0 && (step || jn > j0)) {
                __syncthreads();
                stage(step * C::kStep);
                __syncthreads();
            }
            const v4i *act = reinterpret_cast<const v4i *>(lds) + (u0 * 8 + g) * S::kT + (i ^ g);
            const float *d = dq_s + u0 * S::kT + 4 * g;
            w.deal(rows.soff & 2, nb - step * C::kStep);
#pragma unroll
            for (int j = 0; j < S::kPhases; ++j) {
                float sum[NT][4] = {};
                // A phase past the end is left out (sign, 8 blocks of 16: 338 us to 296; half phases to 276, but
                // rows of whole steps 5% slower). The first holds block 0, the last makes room for the next codes.
                const bool any = j == 0 || j == S::kPhases - 1 || C::kStep - 4 * j - 3 < nb - step * C::kStep;
#pragma unroll
                for (int h = 0; any && h < 2; ++h) {   // two blocks of the phase
                    int blk[2];
                    v4i wt[2][2];
                    float s[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int x = 4 * j + 2 * h + b;
                        blk[b] = x ? C::kStep - x : 0;   // block of the step
                        const C core = w.block(blk[b]);
                        wt[b][0] = core.weights(0);
                        wt[b][1] = core.weights(1);
                        s[b] = w.scale(blk[b]);
                        // decoded here, not below the loads that take the codes' registers
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            asm volatile("" : "+v"(wt[b][0][e]), "+v"(wt[b][1][e]));
                        asm volatile("" : "+v"(s[b]));
                    }
                    if (j == S::kPhases - 1 && h == 1) {   // the step's codes are used up
                        if (step + 1 < steps) {
                            load_weights(step + 1);
                        } else if (jn + 1 < j1) {
                            rows.move(a, col0 + n0 + S::kCols, nb);
                            load_weights(0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float term[2][4];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const v4i a0 = act[blk[b] * 8 * S::kT + 16 * t], a1 = act[(blk[b] * 8 + 4) * S::kT + 16 * t];
                            v4i z = {kMagicBits, kMagicBits, kMagicBits, kMagicBits};
                            z = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, wt[b][0], z, 0, 0, 0);
                            z = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, wt[b][1], z, 0, 0, 0);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                term[b][e] = (s[b] * d[blk[b] * S::kT + 16 * t + e]) * (__int_as_float(z[e]) - kMagic);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = term[0][e] + term[1][e];
                            sum[t][e] = h ? sum[t][e] + v : v;
                            // the group's operations are pure: held here, or they sink below the
                            // next groups' operand reads, which then all stay in registers
                            asm volatile("" : "+v"(sum[t][e]));
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        add_phase<S::kPhases>(j, sum[t][e], part0[t][e], part1[t][e], acc[t][e]);
            }
        }

        if constexpr (TWO) {   // g and u through LDS, then h and its rotation
            float *hs = reinterpret_cast<float *>(lds + S::kActBytes + S::kDqBytes);
            __syncthreads();   // the last row group's h has been read
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    hs[(mat * S::kT + 16 * t + g + 4 * e) * S::kHPitch + col0] = acc[t][e];
            __syncthreads();
            const int lane16 = tid & 15, pair = tid >> 4;
            static_assert(S::kThreads / 16 >= S::kT, "16 lanes for each pair");
            if (pair < tile.rows) {
                const float *gp = hs + pair * S::kHPitch + lane16 * 8, *up = gp + S::kT * S::kHPitch;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = silu_gate(gp[e], up[e]);
                uint32_t packed[2];
                float dq;
                rotquant_h(v, lane16, a.unit, packed, dq);
                const size_t slot = tile.slot + pair;
                *reinterpret_cast<uint2 *>(a.qh + slot * a.n + n0 + lane16 * 8) = make_uint2(packed[0], packed[1]);
                if (lane16 == 0)
                    a.dqh[slot * (a.n / kBlock) + n0 / kBlock] = dq;
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (float *o = pair_out<TWO>(a, tile, 16 * t + g + 4 * e))
                        if (n0 + col0 < a.n)
                            o[n0 + col0] = acc[t][e];
        }
    }
}

// groups: workgroups of a tile; each takes its share of the row groups.
template <int FMT, bool TWO>
__global__ __launch_bounds__(1024) void moe_wide_kernel(MoeArgs a, uint32_t first, int groups)
{
    using S = WideShape<FMT, TWO>;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    Tile tile;
    int group;
    if (!take_item<S::kT>(a, first + blockIdx.x, groups, tile, group))
        return;
    const int nblk = (a.n + S::kCols - 1) / S::kCols, j0 = part_lo(nblk, groups, group), j1 = part_lo(nblk, groups, group + 1);
    if (tile.rows <= 16)
        wide_product<FMT, TWO, 1>(a, tile, j0, j1, lds);
    else if (tile.rows <= 32)
        wide_product<FMT, TWO, 2>(a, tile, j0, j1, lds);
    else
        wide_product<FMT, TWO, 3>(a, tile, j0, j1, lds);
}

// ------------------------------------------------------------------------------------
// Few pairs per expert: tiles of 8 pairs, 8 waves of 16 weight rows. The operations that make operands
// of the codes serve 8 pairs at most and count most here, so the product is of 4-bit by 8-bit floats
// (stage_split). At 5 pairs of each of 16 experts, sign, k = 5120, gate/up of 2176 rows took 40 us, down
// 34, as products of bytes in tiles of 16 pairs; 22 to 30 (by the longest lists) and 18 so. Codes are
// loaded a step ahead. Bound: nothing alone. A unit of 16 rows by a block takes 22 vector
// operations and 2 KB from LDS, and a workgroup spends about as long again on the chain of its first
// loads (offsets, order, activations) and on staging. Two row tiles a wave, which halve what is
// read from LDS, and loads by whole lines, which take lane exchanges, measured the same within 5%.
// ------------------------------------------------------------------------------------
template <int FMT, bool TWO>
struct NarrowShape {
    static constexpr int kWaves = 8, kThreads = 64 * kWaves;
    static constexpr int kT = 8;
    static constexpr int kCols = TWO ? 8 * kWaves : 16 * kWaves;   // gate/up: the upper waves take up's rows
    static constexpr int kPhases = Core<FMT>::kStep / 4;
    static constexpr int kActBytes = 64 * 1024, kDqBytes = 1024;
    static constexpr int kLds = kActBytes + kDqBytes;
};

// NE: elements that hold pairs.
template <int FMT, bool TWO, int NE>
__device__ __forceinline__ void narrow_product(const MoeArgs &a, const Tile &tile, int n0, uint8_t *lds)
{
    using C = Core<FMT>;
    using S = NarrowShape<FMT, TWO>;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 15, g = l >> 4;
    const int nb = a.k / kBlock, steps = (nb + C::kStep - 1) / C::kStep;

    constexpr int T = 4 * NE, kBlocks = 64 / NE;   // pairs of a tile, blocks staged at a time
    constexpr int kBlockPieces = 8 * 2 * T;        // 16-byte pieces of a block: 8 planes of 2 T rows
    static_assert(kBlocks * kBlockPieces * 16 == S::kActBytes && kBlocks * T * 4 == S::kDqBytes, "");
    float *dq_s = reinterpret_cast<float *>(lds + S::kActBytes);
    const int act_scale = 127 + 9 + 4 * (i & 1);   // of A row i, lower or upper halves: 2^9 or 2^13

    const int m = TWO && wave >= S::kWaves / 2, col = n0 + 16 * (TWO ? wave % (S::kWaves / 2) : wave) + i;
    const WeightRows<FMT> rows(a, m, tile.expert, col, nb);
    StepRow<FMT> w[2];
    auto load_weights = [&](int j, int step) { w[j].load(rows.codes, rows.scales, rows.coff + g * 16, rows.soff & ~3u, nb, step); };
    const int my_row = (int)act_row<TWO>(a, tile.slot + min(l & 7, tile.rows - 1));   // of pair l % 8
    load_weights(0, 0);

    // Staging: the pieces of all pairs are dealt to the threads, all loads in flight at once.
    auto stage = [&](int c0) {
        constexpr int kLoads = T * kBlocks * 8 / S::kThreads, kDq = (T * kBlocks + S::kThreads - 1) / S::kThreads;
        // whole steps: blocks past the end read the last one (what is left in LDS may be NaN), with dq 0
        const int blocks = min(kBlocks, nb - c0), padded = (blocks + C::kStep - 1) / C::kStep * C::kStep;
        const int items = tile.rows * padded;
        // x / padded for x < 512: x + 1/2 over it is farther from a whole number than the product's rounding
        const float inv = 1.0f / (float)padded;
        auto split = [&](int x, int &tok, int &u) {
            tok = (int)(((float)x + 0.5f) * inv);
            u = x - tok * padded;
        };
        float dv[kDq];
        uint4 v[kLoads];
        int tok, u;
#pragma unroll
        for (int j = 0; j < kDq; ++j) {
            split(tid + j * S::kThreads, tok, u);
            const int row = __shfl(my_row, tok & 7);
            dv[j] = 0.0f;
            if (tid + j * S::kThreads < items && u < blocks)
                dv[j] = a.dq[(size_t)row * nb + c0 + u];
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (j * (S::kThreads / 8) < items) {   // the same for all lanes
                split(min(j * (S::kThreads / 8) + (tid >> 3), items - 1), tok, u);
                const int row = __shfl(my_row, tok);
                v[j] = *reinterpret_cast<const uint4 *>(a.q + (size_t)row * a.k + (c0 + min(u, blocks - 1)) * kBlock + (tid & 7) * 16);
            }
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (j * (S::kThreads / 8) < items) {
                split(min(j * (S::kThreads / 8) + (tid >> 3), items - 1), tok, u);
                stage_split<FMT, NE>(lds, u, tok, tid & 7, v[j]);
            }
#pragma unroll
        for (int j = 0; j < kDq; ++j) {
            split(tid + j * S::kThreads, tok, u);
            if (tid + j * S::kThreads < items)
                dq_s[u * T + NE * (tok & 3) + (tok >> 2)] = dv[j];
        }
    };
    stage(0);
    if (steps > 1)
        load_weights(1, 1);
    __syncthreads();

    float acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e)
        acc[e] = 0.0f;
    for (int s0 = 0; s0 < steps; s0 += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int step = s0 + j;
            if (step < steps) {   // the same for all waves
                constexpr int kPer = kBlocks / C::kStep;   // steps staged at a time
                if (step && step % kPer == 0) {
                    __syncthreads();
                    stage(step * C::kStep);
                    __syncthreads();
                }
                const int u0 = step % kPer * C::kStep, left = nb - step * C::kStep;
                w[j].deal(rows.soff & 2, left);
                const v4i *act = reinterpret_cast<const v4i *>(lds) + u0 * kBlockPieces + g * (2 * T) +
                                 ((NE == 1 ? 2 * (i >> 2) + (i & 1) : i) ^ (2 * g));
                const float *d = dq_s + u0 * T + NE * g;
                float part0[NE], part1[NE];
#pragma unroll
                for (int q = 0; q < S::kPhases; ++q) {
                    float sum[NE] = {};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if ((q == 0 && h == 0) || C::kStep - (4 * q + 2 * h + 1) < left) {   // else both are past the end
                            float term[2][NE];
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const int x = 4 * q + 2 * h + b, blk = x ? C::kStep - x : 0;
                                const v4i *p = act + blk * kBlockPieces;
                                // the weights' scale takes back their 2, the activations' makes whole numbers of
                                // their lower and upper halves
                                const v4f z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    join(p[0], p[4 * 2 * T]), w[j].block(blk).floats(), v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 4, 0, act_scale, 0, 126);
                                const float s = w[j].scale(blk);
#pragma unroll
                                for (int e = 0; e < NE; ++e)
                                    term[b][e] = (s * d[blk * T + e]) * (z[2 * e] + z[2 * e + 1]);
                            }
#pragma unroll
                            for (int e = 0; e < NE; ++e) {
                                const float v = term[0][e] + term[1][e];
                                sum[e] = h ? sum[e] + v : v;
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        add_phase<S::kPhases>(q, sum[e], part0[e], part1[e], acc[e]);
                        asm volatile("" : "+v"(sum[e]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (step + 2 < steps)
                    load_weights(j, step + 2);
            }
        }
    }
    if constexpr (TWO) {   // u through LDS to the lanes that hold its g
        float *u = reinterpret_cast<float *>(lds) + (wave % (S::kWaves / 2)) * (64 * NE) + l;
        __syncthreads();
        if (m)
#pragma unroll
            for (int e = 0; e < NE; ++e)
                u[64 * e] = acc[e];
        __syncthreads();
        if (m)
            return;
#pragma unroll
        for (int e = 0; e < NE; ++e)
            acc[e] = silu_gate(acc[e], u[64 * e]);
    }
#pragma unroll
    for (int e = 0; e < NE; ++e)
        if (float *o = pair_out<TWO>(a, tile, g + 4 * e))
            if (col < a.n)
                o[col] = acc[e];
}

template <int FMT, bool TWO>
__global__ __launch_bounds__(512, 4) void moe_narrow_kernel(MoeArgs a, uint32_t first)
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
    else
        narrow_product<FMT, TWO, 2>(a, tile, n0, lds);
}

// rotquant of the slots in use: rows [0, offsets[experts]) of h. One 128-block per 16 lanes.
constexpr int kRotThreads = 256;
__global__ __launch_bounds__(kRotThreads) void moe_rotquant_kernel(const float *__restrict__ h, int nb, int pairs,
                                                                   const int32_t *__restrict__ used,
                                                                   int8_t *__restrict__ q, float *__restrict__ dq, float unit)
{
    const size_t blocks = (size_t)min(max(*used, 0), pairs) * nb, stride = (size_t)gridDim.x * (kRotThreads / 16);
    const int lane16 = threadIdx.x & 15;
    for (size_t b = (size_t)blockIdx.x * (kRotThreads / 16) + (threadIdx.x >> 4); b < blocks; b += stride) {
        float v[8], d;
        uint32_t packed[2];
        tbr::Eight<float> h8;
        h8.load(h + b * kBlock + lane16 * 8);
        h8.get(v);
        rotquant_h(v, lane16, unit, packed, d);
        *reinterpret_cast<uint2 *>(q + b * kBlock + lane16 * 8) = make_uint2(packed[0], packed[1]);
        if (lane16 == 0)
            dq[b] = d;
    }
}

// out[t] = sum over j, ascending, of weights[t][j] * y[t topk + j], leaving out pairs of no expert.
// A workgroup takes one token and up to 256 * VEC columns, VEC of them (one 16-byte load, where n
// allows it) a thread; four pairs' loads are in flight. Bound: memory (4096 tokens of 8 pairs x 2048,
// bf16: 43 us, 6.7 TB/s, part of y still in the last cache).
template <class T>
__device__ __forceinline__ void put(T *p, const float (&v)[1])
{
    p->bits = (uint16_t)tbr::pack(v[0], 0.0f, T());
}
__device__ __forceinline__ void put(float *p, const float (&v)[1]) { *p = v[0]; }
template <class T>
__device__ __forceinline__ void put(T *p, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(tbr::pack(v[0], v[1], T()), tbr::pack(v[2], v[3], T()));
}
__device__ __forceinline__ void put(float *p, const float (&v)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

constexpr int kCombineThreads = 256;
template <class T, int VEC>
__global__ __launch_bounds__(kCombineThreads) void moe_combine_kernel(const float *__restrict__ y, const float *__restrict__ weights,
                                                                      const int32_t *__restrict__ ids, int64_t items, int parts,
                                                                      int topk, int experts, int n, T *__restrict__ out)
{
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int t = (int)(item / parts), c = ((int)(item - (int64_t)t * parts) * kCombineThreads + (int)threadIdx.x) * VEC;
        if (c >= n)
            continue;
        float s[VEC] = {};
        for (int j0 = 0; j0 < topk; j0 += 4) {
            float v[4][VEC], w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const size_t p = (size_t)t * topk + min(j0 + j, topk - 1);
                const bool on = j0 + j < topk && (unsigned)ids[p] < (unsigned)experts;   // the same for all lanes
                w[j] = on ? weights[p] : 0.0f;
#pragma unroll
                for (int x = 0; x < VEC; ++x)
                    v[j][x] = 0.0f;
                if (on) {
                    if (VEC == 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(y + p * n + c);
                        v[j][0] = q.x, v[j][1 % VEC] = q.y, v[j][2 % VEC] = q.z, v[j][3 % VEC] = q.w;
                    } else {
                        v[j][0] = y[p * n + c];
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < VEC; ++x)
                    s[x] = fmaf(w[j], v[j][x], s[x]);   // a pair left out adds 0 * 0
        }
        put(out + (size_t)t * n + c, s);
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

// Launches items of tiles * parts in grids of up to kMaxGrid workgroups.
template <class F>
int launch_items(int64_t tiles, int parts, F &&launch)
{
    const int64_t total = tiles * parts;
    if (total > 0x7fffffff)
        return TB_EUNSUPPORTED;
    for (int64_t first = 0; first < total; first += kMaxGrid) {
        launch(dim3((unsigned)std::min<int64_t>((total - first + kXcds - 1) / kXcds * kXcds, kMaxGrid)), (uint32_t)first);
        if (hipGetLastError() != hipSuccess)
            return TB_EHIP;
    }
    return TB_OK;
}
// Tiles of `rows` pairs at most: every expert's last may be partly filled, and none is empty.
int64_t most_tiles(const MoeArgs &a, int rows) { return std::min<int64_t>(a.pairs, (int64_t)a.pairs / rows + a.experts); }

// Wide tiles from this many pairs per expert on, on the average: earlier for ternary codes, whose
// decode costs the narrow tiles more, and where the experts' row groups fill the chip. gate/up + down in
// narrow and in wide tiles, us, by pairs per expert: 16 experts, ternary, 2048 x 1024, 16: 32 and 37, 24: 38
// and 38, 32: 44 and 39; 64 experts, 12: 62 and 56, 16: 75 and 58, 24: 103 and 73; 64 experts, 5120 x 2176, 12: 222
// and 266, 16: 280 and 271; 16 experts, sign, 5120 x 2176, 24: 110 and 154, 32: 137 and 155, 48: 188 and 156;
// 64 experts, sign, 2048 x 1024, 24: 101 and 93, 32: 124 and 94.
bool wide_tiles(const MoeArgs &a, int fmt)
{
    const bool full = (int64_t)a.experts * ((a.n + 127) / 128) >= 512;
    return (int64_t)a.pairs >= (int64_t)a.experts * (fmt == TB_FMT_TERNARY2 ? (full ? 14 : 24) : (full ? 28 : 36));
}

// Into how many workgroups a tile's row groups go. A CU holds one; to start and to stage takes it the time
// of some 11 blocks of a row group (10 us), which speaks for few, and what counts is the rounds that they
// make on 256 CUs, a last one that is not full by half, for tiles that are not full are faster. tiles: one
// per expert, or about half a tile of each not full and some more. gate/up in us, as few parts as leave two
// workgroups for each CU, and so: 147 tiles x 5 groups x 28 blocks 165 and 87; 51 x 8 x 16 39 and 33;
// 31 x 17 x 40 (sign) 147 and 103; 218 x 4 x 9 (sign) 63 and 54; 125 x 17 x 40 329 and 296, 72 x 17 x 40 203
// and 200; 722 x 8 x 16 one part both ways, 290 (in 2 349, in 8 422).
int wide_groups(int64_t tiles, int nblk, int blocks)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int p = 1; p <= nblk && p <= 256; ++p) {
        const int64_t work = tiles * p, full = (work + 255) / 256 * 256;
        const int64_t cost = (full + std::max<int64_t>(work, 256)) * (11 + (int64_t)blocks * ((nblk + p - 1) / p));
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}

template <int FMT, bool TWO>
int launch_product_as(const MoeArgs &a, hipStream_t stream)
{
    if (!wide_tiles(a, FMT)) {
        using S = NarrowShape<FMT, TWO>;
        return launch_items(most_tiles(a, S::kT), (a.n + S::kCols - 1) / S::kCols, [&](dim3 grid, uint32_t first) {
            hipLaunchKernelGGL((moe_narrow_kernel<FMT, TWO>), grid, dim3(S::kThreads), 0, stream, a, first);
        });
    }
    using S = WideShape<FMT, TWO>;
    const int64_t tiles = most_tiles(a, S::kT);
    const int nblk = (a.n + S::kCols - 1) / S::kCols, steps = (a.k / kBlock + Core<FMT>::kStep - 1) / Core<FMT>::kStep;
    const int likely = std::max(std::min(a.pairs, a.experts), a.pairs / S::kT + (a.experts * 5 + 7) / 8);
    const int groups = wide_groups(likely, nblk, steps * Core<FMT>::kStep);
    return launch_items(tiles, groups, [&](dim3 grid, uint32_t first) {
        hipLaunchKernelGGL((moe_wide_kernel<FMT, TWO>), grid, dim3(S::kThreads), 0, stream, a, first, groups);
    });
}
template <bool TWO>
int launch_product(const MoeArgs &a, int fmt, hipStream_t stream)
{
    return fmt == TB_FMT_TERNARY2 ? launch_product_as<TB_FMT_TERNARY2, TWO>(a, stream) : launch_product_as<TB_FMT_SIGN1, TWO>(a, stream);
}

template <class T, int VEC>
int launch_combine_as(const float *y, const float *weights, const int32_t *ids, int tokens, int topk, int experts, int n,
                      void *out, hipStream_t stream)
{
    const int parts = (n + kCombineThreads * VEC - 1) / (kCombineThreads * VEC);
    const int64_t items = (int64_t)tokens * parts;
    hipLaunchKernelGGL((moe_combine_kernel<T, VEC>), dim3((unsigned)std::min<int64_t>(items, kMaxGrid)), dim3(kCombineThreads), 0, stream,
                       y, weights, ids, items, parts, topk, experts, n, static_cast<T *>(out));
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}
template <class T>
int launch_combine(const float *y, const float *weights, const int32_t *ids, int tokens, int topk, int experts, int n,
                   void *out, hipStream_t stream)
{
    return n % 4 ? launch_combine_as<T, 1>(y, weights, ids, tokens, topk, experts, n, out, stream)
                 : launch_combine_as<T, 4>(y, weights, ids, tokens, topk, experts, n, out, stream);
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
    const int waves = std::min(kPlanWaves, (pairs - 1) / 256 + 1);
    hipLaunchKernelGGL(moe_plan_kernel, dim3(experts + 1), dim3(64 * waves), 0, static_cast<hipStream_t>(stream), ids, pairs, experts,
                       offsets, order);
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
    if ((rc = launch_product<true>(args, wg->fmt, st)) || wide_tiles(args, wg->fmt))
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
    // the columns of the last workgroup, those past n too, in 31 bits
    if (rc || experts > kMaxExperts || n > 0x7fffffff - kCombineThreads * 4)
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
