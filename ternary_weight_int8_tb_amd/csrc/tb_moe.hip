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
// Tiles: an expert's list is cut into tiles of up to ROWS pairs. find_tile gives the expert of
// tile t, counted over all experts, and the tile's first slot and rows; false past the last.
// Every wave runs it on its own (all lanes active). Values outside [0, pairs] that a caller
// may have left in offsets are cut, so that no slot past the arrays is touched.
// ------------------------------------------------------------------------------------
struct Tile {
    int expert, slot, rows;
};
template <int ROWS>
__device__ __forceinline__ bool find_tile(const int32_t *__restrict__ offsets, int experts, int pairs, int t, Tile &out)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, count = 0;
        if (e < experts) {
            lo = min(max(offsets[e], 0), pairs);
            count = max(min(offsets[e + 1], pairs) - lo, 0);
        }
        const int tiles = (count + ROWS - 1) / ROWS;
        int upto = tiles;   // inclusive prefix sum over the lanes
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off);
            upto += lane >= off ? o : 0;
        }
        const uint64_t past = __ballot(before + upto > t);
        if (past) {
            const int src = __ffsll((unsigned long long)past) - 1;
            const int first = __shfl(before + upto - tiles, src), c = __shfl(count, src), l = __shfl(lo, src);
            const int r0 = (t - first) * ROWS;
            out.expert = e0 + src;
            out.slot = l + r0;
            out.rows = min(ROWS, c - r0);
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

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
    __device__ __forceinline__ void load(const uint8_t *block, int g) { w = *reinterpret_cast<const uint2 *>(block + g * 8); }
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
    __device__ __forceinline__ void load(const uint8_t *block, int g) { w = *reinterpret_cast<const uint32_t *>(block + g * 4); }
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

// ------------------------------------------------------------------------------------
// Product of 16 weight rows with up to 16 pairs of one expert per workgroup. The unit of work is a
// pair of blocks of one step: the two terms that the step's tree adds first, (0, last), then
// (last - 1, last - 2), and so on. Waves take units in turn; the tree's upper levels and the sum over
// steps run over the units' sums in LDS.
// ------------------------------------------------------------------------------------
constexpr int kRowsWaves = 8;

struct MoeArgs {
    const uint8_t *codes[2];
    const uint16_t *scales[2];
    int experts, n, k;
    const int8_t *q;
    const float *dq;
    const int32_t *offsets, *order;
    int pairs, topk;   // gate/up: the activation row of pair p is p / topk
    float *out;        // gate/up: h, a row per slot; down: y, a row per pair
};

template <int FMT, bool TWO>
__global__ __launch_bounds__(64 * kRowsWaves) void moe_rows_kernel(MoeArgs a, int tiles)
{
    using C = Core<FMT>;
    constexpr int kMats = TWO ? 2 : 1, kUnits = 32 / kMats;   // units in LDS at a time
    constexpr int kPairs = C::kStep / 2, kSteps = kUnits / kPairs, kBlocks = kSteps * C::kStep;
    __shared__ float4 part[kMats][kUnits][64];
    __shared__ float4 scale_s[kMats][kBlocks][4];   // [block][row]
    __shared__ float dq_s[kBlocks][16];             // [block][pair]
    const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, i = l & 15, g = l >> 4;
    const int nb = a.k / kBlock, ntiles = (a.n + 15) / 16;
    const size_t total = (size_t)tiles * ntiles;
    for (size_t item = blockIdx.x; item < total; item += gridDim.x) {
        Tile tile;
        if (!find_tile<16>(a.offsets, a.experts, a.pairs, (int)(item / ntiles), tile))
            return;   // tiles ascend with the item: the same for every wave
        const int n0 = (int)(item % ntiles) * 16;
        const size_t first = (size_t)tile.expert * a.n;
        const size_t jr = first + min(n0 + i, a.n - 1);
        // the lane's activation row; rows past the tile read its last one and are not stored
        const int slot = tile.slot + min(i, tile.rows - 1);
        size_t ar = slot;
        if (TWO)
            ar = (size_t)min(max(a.order[slot], 0), a.pairs - 1) / a.topk;
        const int8_t *q = a.q + ar * a.k + g * 32;

        float sum[4] = {0.f, 0.f, 0.f, 0.f};   // waves 0 .. kMats - 1: 4 outputs of matrix `wave`
        for (int c0 = 0; c0 < nb; c0 += kBlocks) {
            const int cb = min(kBlocks, nb - c0);   // blocks of this part
            for (int u = tid; u < 16 * cb; u += blockDim.x) {
                const int r = u / cb, b = u % cb;
                const size_t row = first + min(n0 + r, a.n - 1);
#pragma unroll
                for (int m = 0; m < kMats; ++m)
                    reinterpret_cast<float *>(scale_s[m][b])[r] = half_bits_to_float(a.scales[m][row * nb + c0 + b]);
            }
            for (int u = tid; u < 16 * cb; u += blockDim.x) {
                const int r = u / cb, b = u % cb;
                const int sl = tile.slot + min(r, tile.rows - 1);
                size_t rr = sl;
                if (TWO)
                    rr = (size_t)min(max(a.order[sl], 0), a.pairs - 1) / a.topk;
                dq_s[b][r] = a.dq[rr * nb + c0 + b];
            }
            __syncthreads();
            const int units = (cb + C::kStep - 1) / C::kStep * kPairs;
            for (int u = wave; u < units; u += kRowsWaves) {
                const int s0 = u / kPairs * C::kStep, j = u % kPairs;
                const int blk[2] = {s0 + (j ? C::kStep - 2 * j : 0), s0 + C::kStep - 1 - 2 * j};
                float t[kMats][4];
#pragma unroll
                for (int m = 0; m < kMats; ++m)
                    t[m][0] = t[m][1] = t[m][2] = t[m][3] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (blk[h] >= cb)
                        continue;   // a block that is not there counts +0
                    const int b = blk[h];
                    const uint4 lo = *reinterpret_cast<const uint4 *>(q + (size_t)(c0 + b) * kBlock);
                    const uint4 hi = *reinterpret_cast<const uint4 *>(q + (size_t)(c0 + b) * kBlock + 16);
                    const v4i b0 = C::acts(lo, hi, 0), b1 = C::acts(lo, hi, 1);
                    const float d = dq_s[b][i];
#pragma unroll
                    for (int m = 0; m < kMats; ++m) {
                        C core;
                        core.load(a.codes[m] + (jr * nb + c0 + b) * C::kBlockBytes, g);
                        v4i z = {0, 0, 0, 0};
                        z = __builtin_amdgcn_mfma_i32_16x16x64_i8(core.weights(0), b0, z, 0, 0, 0);
                        z = __builtin_amdgcn_mfma_i32_16x16x64_i8(core.weights(1), b1, z, 0, 0, 0);
                        const float4 sc = scale_s[m][b][g];
                        t[m][0] += (sc.x * d) * (float)z[0];
                        t[m][1] += (sc.y * d) * (float)z[1];
                        t[m][2] += (sc.z * d) * (float)z[2];
                        t[m][3] += (sc.w * d) * (float)z[3];
                    }
                }
#pragma unroll
                for (int m = 0; m < kMats; ++m)
                    part[m][u][l] = make_float4(t[m][0], t[m][1], t[m][2], t[m][3]);
            }
            __syncthreads();
            if (wave < kMats) {
                for (int s = 0; s < units; s += kPairs) {
                    float4 p[kPairs];
#pragma unroll
                    for (int j = 0; j < kPairs; ++j)
                        p[j] = part[wave][s + j][l];
#pragma unroll
                    for (int w = kPairs / 2; w >= 1; w >>= 1)
#pragma unroll
                        for (int j = 0; j < w; ++j) {
                            p[j].x = p[2 * j].x + p[2 * j + 1].x;
                            p[j].y = p[2 * j].y + p[2 * j + 1].y;
                            p[j].z = p[2 * j].z + p[2 * j + 1].z;
                            p[j].w = p[2 * j].w + p[2 * j + 1].w;
                        }
                    sum[0] += p[0].x;
                    sum[1] += p[0].y;
                    sum[2] += p[0].z;
                    sum[3] += p[0].w;
                }
            }
            __syncthreads();
        }
        if (TWO) {   // wave 1 hands u to wave 0
            if (wave == 1)
                part[0][0][l] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            __syncthreads();
            if (wave == 0) {
                const float4 u = part[0][0][l];
                sum[0] = silu_gate(sum[0], u.x);
                sum[1] = silu_gate(sum[1], u.y);
                sum[2] = silu_gate(sum[2], u.z);
                sum[3] = silu_gate(sum[3], u.w);
            }
        }
        if (wave == 0 && i < tile.rows) {
            const int row = TWO ? tile.slot + i : a.order[tile.slot + i];
            if ((unsigned)row < (unsigned)a.pairs) {
                float *o = a.out + (size_t)row * a.n + n0 + 4 * g;
                for (int r = 0; r < 4 && n0 + 4 * g + r < a.n; ++r)
                    o[r] = sum[r];
            }
        }
        __syncthreads();   // part is written again
    }
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
    return w->experts > kMaxExperts ? TB_EUNSUPPORTED : TB_OK;
}

// tokens * topk pairs: TB_OK if they can be counted in 31 bits
int check_pairs(int tokens, int topk)
{
    if (tokens < 1 || topk < 1)
        return TB_EINVAL;
    return (int64_t)tokens * topk > 0x7fffffc0 ? TB_EUNSUPPORTED : TB_OK;
}

template <bool TWO>
int launch_rows(const MoeArgs &a, int fmt, hipStream_t stream)
{
    // every expert's last tile may be partly filled, and no tile is empty
    const int tiles = (int)std::min<int64_t>(a.pairs, (int64_t)a.pairs / 16 + a.experts);
    const size_t total = (size_t)tiles * ((a.n + 15) / 16);
    const dim3 grid((unsigned)std::min<size_t>(total, kMaxGrid)), block(64 * kRowsWaves);
    if (fmt == TB_FMT_TERNARY2)
        hipLaunchKernelGGL((moe_rows_kernel<TB_FMT_TERNARY2, TWO>), grid, block, 0, stream, a, tiles);
    else
        hipLaunchKernelGGL((moe_rows_kernel<TB_FMT_SIGN1, TWO>), grid, block, 0, stream, a, tiles);
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
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
                          {wg->scales, wu->scales}, wg->experts, wg->n, wg->k, q, dq, offsets, order, (int)pairs, topk, h};
    if ((rc = launch_rows<true>(args, wg->fmt, st)))
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
                          qh, dqh, offsets, order, pairs, 1, y};
    return launch_rows<false>(args, wd->fmt, static_cast<hipStream_t>(stream));
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
