// tb_mx.hip -- microscaled 4-bit floating point (OCP MX, e2m1 elements, one e8m0 scale per 32):
// quantiser, its inverse, and the product on the scaled matrix instructions of gfx950.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tb.h"
#include "tb_host.h"
#include "tb_rows.h"

namespace {

using namespace tbr;

constexpr int kBlock = 128;   // elements of a rotation block, and of one matrix instruction's k
constexpr int kMxBlock = 32;  // elements that share a scale
constexpr int kNanScale = 255;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------------------------
// Quantiser. 16 lanes hold a 128-block, 8 elements each; the 4 lanes of a quad hold the 32
// elements of one scale (chunk_of permutes within quads only). With E the biased exponent of
// the largest magnitude, the scale byte is E - 2, so that the largest element lands in
// [4, 8) (it saturates at 6); v_cvt_scalef32_pk_fp4_f32 divides by the scale and rounds to
// nearest, ties to even. Bound: memory (17408 x 5120 bf16: 44 to 51 us, 4.4 to 5.1 TB/s).
// ------------------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kMaxGrid = 1 << 20;

template <class T, bool ROT>
__global__ __launch_bounds__(kQuantThreads) void mx_quant_kernel(const T *__restrict__ x, size_t blocks,
                                                                 uint32_t *__restrict__ codes,
                                                                 uint32_t *__restrict__ scales, float norm)
{
    const int lane16 = threadIdx.x & 15, chunk = chunk_of(lane16);
    const float sign = chunk_sign(lane16) * norm;
    const size_t stride = (size_t)gridDim.x * (kQuantThreads / 16);
    for (size_t b = (size_t)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4); b < blocks; b += stride) {
        Eight<T> ex;
        float v[8];
        ex.load(x + b * kBlock + chunk * 8);
        ex.get(v);
        if (ROT) {
            rotate_signed(v, lane16);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] *= sign;
        }
        const uint32_t top = amax_bits<2>(v) >> 23;   // biased exponent; 255: not finite
        uint32_t byte = top > 2 ? top - 2 : 0, w = 0;
        if (byte && top < 255) {
            const float scale = __uint_as_float(byte << 23);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
        }
        if (top == 255)
            byte = kNanScale;
        codes[b * 16 + chunk] = w;
        // lane 0 collects the four quads' bytes: row_ror:n hands lane 0 the value of lane 16 - n
        const uint32_t b1 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x12C, 0xF, 0xF, false);
        const uint32_t b2 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x128, 0xF, 0xF, false);
        const uint32_t b3 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x124, 0xF, 0xF, false);
        if (lane16 == 0)
            scales[b] = byte | b1 << 8 | b2 << 16 | b3 << 24;
    }
}

// Values of the codes, 8 per thread.
template <class T>
__global__ __launch_bounds__(kQuantThreads) void mx_dequant_kernel(const uint32_t *__restrict__ codes,
                                                                   const uint8_t *__restrict__ scales, size_t words,
                                                                   T *__restrict__ y)
{
    const size_t stride = (size_t)gridDim.x * kQuantThreads;
    for (size_t i = (size_t)blockIdx.x * kQuantThreads + threadIdx.x; i < words; i += stride) {
        const uint32_t w = codes[i];
        const int byte = scales[i / 4];
        const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3)};
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = byte == kNanScale ? __uint_as_float(0x7fc00000u) : ldexpf(p[e >> 1][e & 1], byte - 127);
        Eight<T> o;
        o.set(v);
        o.store(y + i * 8);
    }
}

// ------------------------------------------------------------------------------------
// Product, few rows. v_mfma_scale_f32_16x16x128_f8f6f4: lane (i, g) = (lane % 16, lane / 16)
// supplies 32 codes (16 bytes) of one block of row i and their scale, for A and B alike, of any
// block as long as both agree; lane l ends with rows 4 g + 0 .. 3 of A against row l % 16 of B. A is
// the weights, B the activation, so an operand of either comes from its row, with no exchange and no
// LDS. k goes in halves of 256 elements, a 128-byte line of codes; lane group g takes blocks 2 g and
// 2 g + 1 of a half, whose two scales are one 16-bit load.
// A workgroup owns 16 weight rows and all activation rows (the plan gives it up to kRowsMost, the operand
// holds 16); its waves split k, and add their
// sums through LDS in wave order: the order depends on k alone. Bound: the weights' way from
// memory; a wave has the loads of U halves in flight at a time.
// ------------------------------------------------------------------------------------
constexpr int kRowWaves = 8;

__device__ __forceinline__ v8i operand(uint4 w) { return v8i{(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0}; }

__device__ __forceinline__ void put4(float *p, const float (&v)[4], int count)
{
    if (count == 4 && ((uintptr_t)p & 15) == 0)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        for (int i = 0; i < count; ++i)
            p[i] = v[i];
}
template <class T>
__device__ __forceinline__ void put4(T *p, const float (&v)[4], int count)
{
    const uint32_t a = pack(v[0], v[1], T()), b = pack(v[2], v[3], T());
    if (count == 4 && ((uintptr_t)p & 7) == 0) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
    } else {
        const uint16_t h[4] = {(uint16_t)a, (uint16_t)(a >> 16), (uint16_t)b, (uint16_t)(b >> 16)};
        for (int i = 0; i < count; ++i)
            p[i].bits = h[i];
    }
}

// A lane's share of a half of its row.
struct Half {
    uint4 c[2];
    int scale;   // of both blocks, a byte each
    // codes, scales: the row's, from the lane's first block on; blocks past the row's kb are zeros
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, int h, int kb, int g)
    {
        if ((h + 1) * 8 <= kb || h * 8 + 2 * g < kb) {
            c[0] = *reinterpret_cast<const uint4 *>(codes + (size_t)h * 128);
            c[1] = *reinterpret_cast<const uint4 *>(codes + (size_t)h * 128 + 16);
            scale = *reinterpret_cast<const uint16_t *>(scales + (size_t)h * 8);
        } else {
            c[0] = c[1] = make_uint4(0, 0, 0, 0);
            scale = 0x7f7f;
        }
    }
};

template <class T>
__global__ __launch_bounds__(64 * kRowWaves) void mx_rows_kernel(const uint8_t *__restrict__ wc,
                                                                 const uint8_t *__restrict__ ws,
                                                                 const uint8_t *__restrict__ ac,
                                                                 const uint8_t *__restrict__ as, int m, int n, int k,
                                                                 T *__restrict__ y)
{
    constexpr int U = 4;   // halves in flight
    __shared__ float4 part[kRowWaves][64];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 15, g = l >> 4;
    const int waves = blockDim.x >> 6, kb = k / kMxBlock, halves = (kb + 7) / 8;
    const int n0 = blockIdx.x * 16;
    const int h0 = halves * wave / waves, h1 = halves * (wave + 1) / waves;
    // rows past the end read the last one; what they give is not stored
    const size_t jr = min(n0 + i, n - 1), r = min(i, m - 1);
    const uint8_t *pc = wc + jr * (k / 2) + g * 32, *ps = ws + jr * kb + g * 2;
    const uint8_t *qc = ac + r * (k / 2) + g * 32, *qs = as + r * kb + g * 2;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int h = h0; h < h1; h += U) {
        Half a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {   // the same for all lanes
                a[u].load(pc, ps, h + u, kb, g);
                b[u].load(qc, qs, h + u, kb, g);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h + u < h1) {
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a[u].c[0]), operand(b[u].c[0]), acc, 4, 4, 0, a[u].scale, 0, b[u].scale);
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a[u].c[1]), operand(b[u].c[1]), acc, 4, 4, 1, a[u].scale, 1, b[u].scale);
            }
    }
    part[wave][l] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (wave == 0) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) {
            const float4 p = part[w][l];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
        const int j = n0 + 4 * g;
        if (i < m && j < n)
            put4(y + (size_t)i * n + j, v, min(4, n - j));
    }
}

// ------------------------------------------------------------------------------------
// Product, many rows. v_mfma_scale_f32_32x32x64_f8f6f4: lane (i, g) = (l % 32, l / 32) supplies one
// 32-element block of row i of either operand, and any block of the row will do as long as A and B
// agree. k is taken in halves of 256 (8 blocks, a 128-byte line of codes); lane group g takes blocks
// 4 g .. 4 g + 3 of a half, so that its scales are one word, whose bytes the instruction picks one by
// one (opsel). Two halves are a group, whose scales are loaded together.
//   * A workgroup of 4 waves makes 64 TI weight rows x 64 TJ activation rows, a wave 32 TI x 32 TJ.
//   * Codes go from memory straight to LDS (buffer_load ... lds, 16 bytes a lane), half a group (256
//     elements, 128 bytes a row) at a time into one of two buffers while the other is multiplied.
//     Block j of row r lies at place j ^ ((r / 2) % 8) of the row's 8, so that the 16 lanes that one
//     LDS cycle serves read 16 different columns of banks. A group's scales go the same way.
// Bound: matrix rate. Per 64 elements of k a wave's TI TJ instructions take 32 TI TJ cycles and TI + TJ
// reads of 1 KB: at 4 x 4 all four waves read 64 bytes a cycle of the 128 that LDS gives. Measured:
// 8192 x 17408 x 5120 430 to 500 us by the card, 2.9 to 3.4 PFLOP/s; the instruction alone, on random codes, runs at
// 6.6 to 7.5 (9.9 on zeros: power bounds it). 4 x 4 leaves one wave a SIMD, which stands at every barrier.
// ------------------------------------------------------------------------------------
constexpr int kGroup = 512;              // elements of k whose scales are loaded together
constexpr uint32_t kBufWord3 = 0x00020000u;
constexpr uint32_t kOutOfRange = 0x80000000u;   // a lane offset past every buffer: the load gives zeros

typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, (int)kBufWord3);
}
// 16 (or 4) bytes a lane, to consecutive places from dst on; a lane whose offset is out of range
// stores zeros
__device__ __forceinline__ void load_to_lds16(__amdgpu_buffer_rsrc_t r, uint8_t *dst, uint32_t off, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, off, soff, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(__amdgpu_buffer_rsrc_t r, uint8_t *dst, uint32_t off, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 4, off, soff, 0, 0);
}

struct MxArgs {
    const uint8_t *wc, *ws, *ac, *as;
    int m, n, k;
    void *y;
    float *part;    // sums of a part of k, [parts][m][n]; null: y is written
    int parts;
};

// All tiles of one step; S picks a byte of the scales, a constant of the instruction. After each row of
// tiles `also(ti)` issues its share of the next step's reads and of the next half's loads: a wave
// issues in order, and waits behind a burst of either with nothing to multiply.
template <int S, int TI, int TJ, class F>
__device__ __forceinline__ void mx_step(v16f (&acc)[TI][TJ], const uint4 (&wa)[TI], const uint4 (&xb)[TJ], const uint32_t (&sa)[TI][2],
                                        const uint32_t (&sb)[TJ][2], int q, F &&also)
{
#pragma unroll
    for (int ti = 0; ti < TI; ++ti) {
#pragma unroll
        for (int tj = 0; tj < TJ; ++tj) {
            acc[ti][tj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(wa[ti]), operand(xb[tj]), acc[ti][tj], 4, 4, S,
                                                                          (int)sa[ti][q], S, (int)sb[tj][q]);
            // the instructions are pure: held here, or they sink below the next barrier
            asm volatile("" : "+a"(acc[ti][tj]));
        }
        also(ti);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int TI, int TJ, class T>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs a)
{
    constexpr int kRows = 64 * (TI + TJ);   // weight rows, then activation rows
    // two buffers of codes, arrays of their own: a read of one then waits for no load of the other
    __shared__ __align__(16) uint8_t buf0[kRows * 128];
    __shared__ __align__(16) uint8_t buf1[kRows * 128];
    __shared__ __align__(16) uint8_t sbuf[kRows * 16];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, i = l & 31, g = l >> 5;
    const int wi = wave & 1, wj = wave >> 1;
    const int ntn = (a.n + 64 * TI - 1) / (64 * TI), ntm = (a.m + 64 * TJ - 1) / (64 * TJ);
    // tiles in blocks of 8 along n, dealt to the XCDs in contiguous ranges (workgroup b runs on XCD
    // b % 8): the tiles that run on an XCD at a time share their rows in its L2
    const int tiles = ntn * ntm, per = (tiles + 7) / 8, b = blockIdx.x, item = (b % 8) * per + b / 8;
    if (b / 8 >= per || item >= tiles)
        return;
    const int band = item / (8 * ntm), width = min(8, ntn - band * 8), r = item - band * 8 * ntm;
    const int n0 = (band * 8 + r % width) * 64 * TI, m0 = r / width * 64 * TJ;
    const int kb = a.k / kMxBlock, groups = (kb + 15) / 16;
    const int part = blockIdx.y, g0 = (int)((long long)groups * part / a.parts), g1 = (int)((long long)groups * (part + 1) / a.parts);
    const int pitch = a.k / 2, spitch = kb;

    // staging: a wave takes 8 rows at a time, lane l place l % 8 of row l / 8; rows past the end are
    // the last one, and what they give is not stored
    constexpr int kLoads = kRows / 32;
    const __amdgpu_buffer_rsrc_t wr = buffer(a.wc + (size_t)n0 * pitch, (uint32_t)(min(a.n - n0, 64 * TI) * pitch));
    const __amdgpu_buffer_rsrc_t ar = buffer(a.ac + (size_t)m0 * pitch, (uint32_t)(min(a.m - m0, 64 * TJ) * pitch));
    const __amdgpu_buffer_rsrc_t wsr = buffer(a.ws + (size_t)n0 * spitch, (uint32_t)(min(a.n - n0, 64 * TI) * spitch));
    const __amdgpu_buffer_rsrc_t asr = buffer(a.as + (size_t)m0 * spitch, (uint32_t)(min(a.m - m0, 64 * TJ) * spitch));
    const int j = (l & 7) ^ ((wave & 1) * 4 + (l >> 4));   // the lane's block of the half group
    uint32_t off[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
        const int row = x * 32 + wave * 8 + (l >> 3);
        off[x] = (x < 2 * TI ? min(row, a.n - n0 - 1) : min(row - 64 * TI, a.m - m0 - 1)) * pitch + j * 16;
    }
    static_assert(kLoads == 2 * (TI + TJ) && TJ <= TI, "half of the loads, and all reads, in the TI rows of a step");
    auto load = [&](uint8_t *buf, int grp, int q, int x) {   // load x of half q of a group
        const bool none = grp * 16 + q * 8 + j >= kb;
        load_to_lds16(x < 2 * TI ? wr : ar, buf + (x * 32 + wave * 8) * 128, none ? kOutOfRange : off[x], grp * 256 + q * 128);
    };
    // 16 bytes of a row a lane; of a last group that is not full, word by word, as the row's end allows
    auto load_scales = [&](uint8_t *buf, int grp) {
        if (grp * 16 + 16 <= kb) {
#pragma unroll
            for (int x = 0; x < (kRows + 255) / 256; ++x) {
                if (kRows % 256 && x * 256 + wave * 64 >= kRows)
                    continue;
                const int row = x * 256 + tid;
                const bool w = x * 256 + wave * 64 < 64 * TI;   // the same for all lanes
                load_to_lds16(w ? wsr : asr, buf + (x * 256 + wave * 64) * 16,
                                (w ? min(row, a.n - n0 - 1) : min(row - 64 * TI, a.m - m0 - 1)) * spitch, grp * 16);
            }
        } else {
            for (int x = 0; x < kRows / 64; ++x) {
                const int row = x * 64 + (tid >> 2), word = tid & 3;
                const bool w = x < TI;
                load_to_lds4(w ? wsr : asr, buf + (x * 64 + wave * 16) * 16,
                               grp * 16 + word * 4 >= kb ? kOutOfRange
                                                         : (w ? min(row, a.n - n0 - 1) : min(row - 64 * TI, a.m - m0 - 1)) * spitch + word * 4,
                               grp * 16);
            }
        }
    };

    v16f acc[TI][TJ];
#pragma unroll
    for (int ti = 0; ti < TI; ++ti)
#pragma unroll
        for (int tj = 0; tj < TJ; ++tj)
            acc[ti][tj] = v16f{};
    uint32_t sa[TI][2], sb[TJ][2], na[TI][2], nb[TJ][2];   // scales of a group, and of the next
    auto read_scales = [&](uint32_t (&xa)[TI][2], uint32_t (&xb)[TJ][2]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int ti = 0; ti < TI; ++ti)
                xa[ti][q] = *reinterpret_cast<const uint32_t *>(sbuf + (wi * 32 * TI + ti * 32 + i) * 16 + q * 8 + g * 4);
#pragma unroll
            for (int tj = 0; tj < TJ; ++tj)
                xb[tj][q] = *reinterpret_cast<const uint32_t *>(sbuf + (64 * TI + wj * 32 * TJ + tj * 32 + i) * 16 + q * 8 + g * 4);
        }
    };
    const int wrow = (wi * 32 * TI + i) * 128, arow = (64 * TI + wj * 32 * TJ + i) * 128, swz = (i >> 1) & 7;
    uint4 wa[2][TI], xb[2][TJ];   // operands of a step, and of the next while it is multiplied
    auto operand_pair = [&](const uint8_t *buf, int s, int t) {
        const int place = ((4 * g + s) ^ swz) * 16;
        wa[s & 1][t] = *reinterpret_cast<const uint4 *>(buf + wrow + t * 4096 + place);
        if (t < TJ)
            xb[s & 1][t] = *reinterpret_cast<const uint4 *>(buf + arow + t * 4096 + place);
    };
    // row ti's share of the first (from = 0) or second half of a half group's loads
    auto load_share = [&](uint8_t *buf, int grp, int q, int from, int ti) {
#pragma unroll
        for (int x = (TI + TJ) * ti / TI; x < (TI + TJ) * (ti + 1) / TI; ++x)
            load(buf, grp, q, from * (TI + TJ) + x);
    };
    // Half q from `buf`, whose first step's operands are read. Loads of the next half into `next` were
    // begun by the last step before; the loads after that go to `buf` from the barrier on, where
    // every wave has read it. So a half's loads have two steps to arrive in after the last is issued.
    auto multiply = [&](uint8_t *buf, uint8_t *next, int q, int grp) {
        const int ngrp = q ? grp + 1 : grp;   // of the next half
        mx_step<0>(acc, wa[0], xb[0], sa, sb, q, [&](int ti) {
            operand_pair(buf, 1, ti);
            if (ngrp < g1)
                load_share(next, ngrp, 1 - q, 1, ti);
        });
        if (q && ngrp < g1)
            load_scales(sbuf, ngrp);
        mx_step<1>(acc, wa[1], xb[1], sa, sb, q, [&](int ti) { operand_pair(buf, 2, ti); });
        mx_step<2>(acc, wa[0], xb[0], sa, sb, q, [&](int ti) { operand_pair(buf, 3, ti); });
        __syncthreads();   // the next half (and its scales) have arrived, and buf has been read
        if (q)
            read_scales(na, nb);
        mx_step<3>(acc, wa[1], xb[1], sa, sb, q, [&](int ti) {
            operand_pair(next, 0, ti);
            if (grp + 1 < g1)
                load_share(buf, grp + 1, q, 0, ti);
        });
    };

#pragma unroll
    for (int x = 0; x < kLoads; ++x)
        load(buf0, g0, 0, x);
    load_scales(sbuf, g0);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < TI + TJ; ++x)
        load(buf1, g0, 1, x);
    read_scales(sa, sb);
#pragma unroll
    for (int t = 0; t < TI; ++t)
        operand_pair(buf0, 0, t);
    for (int grp = g0; grp < g1; ++grp) {
        multiply(buf0, buf1, 0, grp);
        multiply(buf1, buf0, 1, grp);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int ti = 0; ti < TI; ++ti)
                sa[ti][q] = na[ti][q];
#pragma unroll
            for (int tj = 0; tj < TJ; ++tj)
                sb[tj][q] = nb[tj][q];
        }
    }

    // Lane l has, of each 32 x 32 tile, weight rows 8 v + 4 g + 0 .. 3 (v = 0 .. 3) of activation row
    // l % 32. Stored so, a row would be written 8 or 16 bytes at a time; a wave passes 32 rows at a
    // time through its part of LDS instead and writes whole lines.
    // (Place c ^ r of row r for its 16-byte column c: no bank conflicts.)
    constexpr int kLanes = 8 * TI, kPer = 64 / kLanes;   // lanes of a row, rows of a store
    static_assert(4 * 32 * kLanes * 16 <= kRows * 128 || TJ < TI, "the waves' rows take a code buffer");
    constexpr bool kApart = 4 * 32 * kLanes * 16 > kRows * 128;   // or both
    float4 *mine = reinterpret_cast<float4 *>(kApart && wave >= 2 ? buf1 : buf0) + (kApart ? wave % 2 : wave) * 32 * kLanes;
    const int col = n0 + wi * 32 * TI + l % kLanes * 4;
    __syncthreads();
#pragma unroll
    for (int tj = 0; tj < TJ; ++tj) {
#pragma unroll
        for (int ti = 0; ti < TI; ++ti)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                mine[i * kLanes + ((ti * 8 + 2 * v + g) ^ (i % kLanes))] =
                    make_float4(acc[ti][tj][4 * v], acc[ti][tj][4 * v + 1], acc[ti][tj][4 * v + 2], acc[ti][tj][4 * v + 3]);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // a wave reads what its own lanes wrote
        for (int x = 0; x < 32 / kPer; ++x) {
            const int r = x * kPer + l / kLanes, row = m0 + wj * 32 * TJ + tj * 32 + r;
            const float4 o = mine[r * kLanes + (l % kLanes ^ r % kLanes)];
            if (row < a.m && col < a.n) {
                const float f[4] = {o.x, o.y, o.z, o.w};
                if (a.part)
                    put4(a.part + ((size_t)part * a.m + row) * a.n + col, f, min(4, a.n - col));
                else
                    put4(static_cast<T *>(a.y) + (size_t)row * a.n + col, f, min(4, a.n - col));
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// y = the sum of the parts, in order. VEC elements a thread (4, where rows of 4 fit), six parts' loads in
// flight: a part after the other took 4.8 us for the 12 of 24 x 5120, 3.8 so.
template <class T, int VEC>
__global__ __launch_bounds__(256) void mx_sum_kernel(const float *__restrict__ part, size_t count, int parts, T *__restrict__ y)
{
    constexpr int kLoads = 6;
    const size_t stride = (size_t)gridDim.x * 256 * VEC;
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * VEC; i < count; i += stride) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int p0 = 0; p0 < parts; p0 += kLoads) {
            float x[kLoads][4] = {};
#pragma unroll
            for (int p = 0; p < kLoads; ++p)
                if (p0 + p < parts) {   // the same for all lanes
                    const float *q = part + (size_t)(p0 + p) * count + i;
                    if (VEC == 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(q);
                        x[p][0] = w.x, x[p][1] = w.y, x[p][2] = w.z, x[p][3] = w.w;
                    } else {
                        x[p][0] = *q;
                    }
                }
#pragma unroll
            for (int p = 0; p < kLoads; ++p)
                if (p0 + p < parts)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        v[e] += x[p][e];
        }
        put4(y + i, v, VEC);
    }
}

// How a product is run: ti = 0: few rows (mx_rows_kernel); else in tiles of 64 ti x 64 tj, k in `parts`.
struct MxPlan {
    int ti, tj, parts;
};
// Up to 8 rows of up to 8192 elements, and 2^20 x 48 weights: one launch of the row kernel; the tiles, which
// stream the weights through LDS in whole lines, need a second launch for the sums, and a workspace. us a
// call in a captured graph, row kernel and tiles: 1 x 5120 x 4096 5.6 and 7.8, 1 x 9216 x 5120 9.3 and 9.8,
// 8 x 9216 x 5120 10.8 and 10.2 (what the rule gives away for one rule up to 8 rows). Beyond it, enqueued
// one by one: 16 x 9216 x 5120 12.2 and 10.2, 1 x 17408 x 5120 13.7 and 13.2, 8 x 17408 x 5120 16.3 and 13.6,
// 1 x 5120 x 17408 16.5 and 12.8.
constexpr int kRowsMost = 8, kRowsMostK = 8192;
constexpr int64_t kRowsMostWeights = 48 << 20;
int64_t tile_count(int64_t m, int64_t n, int ti, int tj) { return (m + 64 * tj - 1) / (64 * tj) * ((n + 64 * ti - 1) / (64 * ti)); }
MxPlan plan_gemm(int m, int n, int k)
{
    if (m <= kRowsMost && k <= kRowsMostK && (int64_t)n * k <= kRowsMostWeights)
        return {0, 0, 1};
    // By the tiles alone, whatever m is: few rows of a very wide layer multiply rows that are not there. 1, 8 and
    // 64 x 160000 x 5120 take 136, 136 and 149 us, where reading the weights would take 74.
    if (tile_count(m, n, 4, 4) >= 192)
        return {4, 4, 1};
    // 128 x 64 tiles while they are few; k in parts until there are two workgroups for each of the chip's 256
    // CUs, or one where the parts' sums are many. us a call in a captured graph: 24 x 5120 x 17408 15.3 in 6 parts,
    // 14.7 in 12; 256 x 5120 x 5120 17.4 in 3, 17.0 in 1; 509 x 5120 x 4096 17.0 as 128 x 128 and 16.7 as 128 x 64;
    // 512 x 9216 x 5120 25.4 as 128 x 128 and 27.7 as 128 x 64.
    const int tj = tile_count(m, n, 2, 1) <= 512 ? 1 : 2, groups = (k + kGroup - 1) / kGroup;
    const int64_t tiles = tile_count(m, n, 2, tj), most = m <= 64 ? 512 : 256;
    return {2, tj, (int)std::min<int64_t>(std::max<int64_t>(1, most / tiles), std::max(1, groups / 2))};
}

template <class T>
int launch_gemm(const tb_mxfp4 *w, const uint8_t *codes, const uint8_t *scales, int m, T *y, float *part, hipStream_t stream)
{
    const MxPlan plan = plan_gemm(m, w->n, w->k);
    if (plan.ti) {
        const dim3 grid((unsigned)((tile_count(m, w->n, plan.ti, plan.tj) + 7) / 8 * 8), plan.parts);
        const MxArgs a = {w->codes, w->scales, codes, scales, m, w->n, w->k, y, plan.parts > 1 ? part : nullptr, plan.parts};
        if (plan.ti == 4)
            hipLaunchKernelGGL((mx_tile_kernel<4, 4, T>), grid, dim3(256), 0, stream, a);
        else if (plan.tj == 2)
            hipLaunchKernelGGL((mx_tile_kernel<2, 2, T>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((mx_tile_kernel<2, 1, T>), grid, dim3(256), 0, stream, a);
        if (hipGetLastError() != hipSuccess)
            return TB_EHIP;
        if (plan.parts > 1) {
            const size_t count = (size_t)m * w->n;
            const int each = count % 4 ? 256 : 1024;   // elements of a workgroup
            const dim3 sums((unsigned)std::min<size_t>((count + each - 1) / each, kMaxGrid));
            if (count % 4)
                hipLaunchKernelGGL((mx_sum_kernel<T, 1>), sums, dim3(256), 0, stream, part, count, plan.parts, y);
            else
                hipLaunchKernelGGL((mx_sum_kernel<T, 4>), sums, dim3(256), 0, stream, part, count, plan.parts, y);
        }
        return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
    }
    const int waves = std::min(kRowWaves, (w->k + 255) / 256);
    hipLaunchKernelGGL((mx_rows_kernel<T>), dim3((w->n + 15) / 16), dim3(64 * waves), 0, stream, w->codes, w->scales, codes, scales, m,
                       w->n, w->k, y);
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

template <class T>
int launch_quant(const void *x, size_t blocks, uint8_t *codes, uint8_t *scales, bool rotate, hipStream_t stream)
{
    const int per = kQuantThreads / 16;
    const int grid = (int)std::min<size_t>((blocks + per - 1) / per, kMaxGrid);
    const float norm = (float)(1.0 / std::sqrt(128.0));
    if (rotate)
        hipLaunchKernelGGL((mx_quant_kernel<T, true>), dim3(grid), dim3(kQuantThreads), 0, stream, static_cast<const T *>(x), blocks,
                           reinterpret_cast<uint32_t *>(codes), reinterpret_cast<uint32_t *>(scales), norm);
    else
        hipLaunchKernelGGL((mx_quant_kernel<T, false>), dim3(grid), dim3(kQuantThreads), 0, stream, static_cast<const T *>(x), blocks,
                           reinterpret_cast<uint32_t *>(codes), reinterpret_cast<uint32_t *>(scales), norm);
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

template <class T>
int launch_dequant(const uint8_t *codes, const uint8_t *scales, size_t elems, void *y, hipStream_t stream)
{
    const size_t words = elems / 8;
    const int grid = (int)std::min<size_t>((words + kQuantThreads - 1) / kQuantThreads, kMaxGrid);
    hipLaunchKernelGGL(mx_dequant_kernel<T>, dim3(grid), dim3(kQuantThreads), 0, stream,
                       reinterpret_cast<const uint32_t *>(codes), scales, words, static_cast<T *>(y));
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

size_t code_bytes(int rows, int k) { return (size_t)rows * (k / 2); }
size_t scale_bytes(int rows, int k) { return (size_t)rows * (k / kMxBlock); }

bool mx_ok(const tb_mxfp4 *w) { return w && w->n >= 1 && w->k >= kBlock && w->k % kBlock == 0; }
// Lane offsets within a tile's rows, and the tiles of a launch, in 31 bits.
bool gemm_fits(const tb_mxfp4 *w, int m) { return w->k < 1 << 24 && tile_count(m, w->n, 2, 2) <= 1 << 23; }

}  // namespace

extern "C" {

int tb_mxfp4_quant(const void *x, int dtype, int m, int k, int rotate, uint8_t *codes, uint8_t *scales, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    if (!eb || m < 1 || k < kBlock || k % kBlock || (rotate & ~1))
        return TB_EINVAL;
    const tbh::Arg a[] = {{x, (size_t)m * k * eb, false}, {codes, code_bytes(m, k), true}, {scales, scale_bytes(m, k), true}};
    if (int rc = tbh::check_args(a))
        return rc;
    const size_t blocks = (size_t)m * (k / kBlock);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case TB_F32: return launch_quant<float>(x, blocks, codes, scales, rotate, st);
    case TB_BF16: return launch_quant<Bf16>(x, blocks, codes, scales, rotate, st);
    default: return launch_quant<F16>(x, blocks, codes, scales, rotate, st);
    }
}

int tb_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, int m, int k, void *y, int dtype, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    if (!eb || m < 1 || k < kBlock || k % kBlock)
        return TB_EINVAL;
    const tbh::Arg a[] = {{codes, code_bytes(m, k), false}, {scales, scale_bytes(m, k), false}, {y, (size_t)m * k * eb, true}};
    if (int rc = tbh::check_args(a))
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case TB_F32: return launch_dequant<float>(codes, scales, (size_t)m * k, y, st);
    case TB_BF16: return launch_dequant<Bf16>(codes, scales, (size_t)m * k, y, st);
    default: return launch_dequant<F16>(codes, scales, (size_t)m * k, y, st);
    }
}

size_t tb_mxfp4_gemm_workspace_bytes(const tb_mxfp4 *w, int m)
{
    if (!mx_ok(w) || m < 1 || !gemm_fits(w, m))
        return 0;
    const MxPlan plan = plan_gemm(m, w->n, w->k);
    return plan.parts > 1 ? (size_t)plan.parts * m * w->n * 4 : 0;
}

int tb_mxfp4_gemm(const tb_mxfp4 *w, const uint8_t *codes, const uint8_t *scales, int m, void *y, int dtype, void *ws,
                  size_t ws_bytes, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    if (!eb || !mx_ok(w) || m < 1)
        return TB_EINVAL;
    if (!gemm_fits(w, m))
        return TB_EUNSUPPORTED;
    const size_t need = tb_mxfp4_gemm_workspace_bytes(w, m);
    const tbh::Arg a[] = {{w->codes, code_bytes(w->n, w->k), false},
                          {w->scales, scale_bytes(w->n, w->k), false},
                          {codes, code_bytes(m, w->k), false},
                          {scales, scale_bytes(m, w->k), false},
                          {y, (size_t)m * w->n * eb, true},
                          {ws, need, true}};
    if (need && ws_bytes < need)
        return TB_EINVAL;
    if (int rc = tbh::check_args(a, need ? 6 : 5))
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case TB_F32: return launch_gemm(w, codes, scales, m, static_cast<float *>(y), static_cast<float *>(ws), st);
    case TB_BF16: return launch_gemm(w, codes, scales, m, static_cast<Bf16 *>(y), static_cast<float *>(ws), st);
    default: return launch_gemm(w, codes, scales, m, static_cast<F16 *>(y), static_cast<float *>(ws), st);
    }
}

}  // extern "C"
