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
// nearest, ties to even. Bound: memory.
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
// supplies the 32 codes (16 bytes) and the scale of block g of row i, for A and B alike; lane l
// ends with rows 4 g + 0 .. 3 of A against row l % 16 of B. A is the weights, B the activation, so
// an operand of either is one 16-byte load from its row, with no exchange and no LDS.
// A workgroup owns 16 weight rows and 16 * MT activation rows; its waves split k, and add their
// sums through LDS in wave order: the order depends on (n, k) alone.
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

template <int MT, class T>
__global__ __launch_bounds__(64 * kRowWaves) void mx_rows_kernel(const uint8_t *__restrict__ wc,
                                                                 const uint8_t *__restrict__ ws,
                                                                 const uint8_t *__restrict__ ac,
                                                                 const uint8_t *__restrict__ as, int m, int n, int k,
                                                                 T *__restrict__ y)
{
    __shared__ float4 part[kRowWaves][MT][64];
    const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, i = l & 15, g = l >> 4;
    const int waves = blockDim.x >> 6, steps = k / kBlock;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
    const int s0 = (int)((long long)steps * wave / waves), s1 = (int)((long long)steps * (wave + 1) / waves);
    // rows past the end read the last one; what they give is not stored
    const size_t jr = min(n0 + i, n - 1);
    const uint8_t *pc = wc + jr * (k / 2) + g * 16, *ps = ws + jr * (k / kMxBlock) + g;
    const uint8_t *qc[MT], *qs[MT];
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const size_t r = min(m0 + t * 16 + i, m - 1);
        qc[t] = ac + r * (k / 2) + g * 16;
        qs[t] = as + r * (k / kMxBlock) + g;
        acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        const v8i a = operand(*reinterpret_cast<const uint4 *>(pc + (size_t)s * 64));
        const int sa = ps[s * 4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const v8i b = operand(*reinterpret_cast<const uint4 *>(qc[t] + (size_t)s * 64));
            const int sb = qs[t][s * 4];
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[t], 4, 4, 0, sa, 0, sb);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
        part[wave][t][l] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    for (int u = tid; u < MT * 64; u += blockDim.x) {
        const int t = u >> 6, ul = u & 63;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < waves; ++w) {
            const float4 p = part[w][t][ul];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
        const int r = m0 + t * 16 + (ul & 15), j = n0 + 4 * (ul >> 4);
        if (r < m && j < n)
            put4(y + (size_t)r * n + j, v, min(4, n - j));
    }
}

template <class T>
int launch_gemm(const tb_mxfp4 *w, const uint8_t *codes, const uint8_t *scales, int m, T *y, hipStream_t stream)
{
    const int waves = std::min(kRowWaves, w->k / kBlock);
    const int mt = m <= 16 ? 1 : m <= 32 ? 2 : 4;
    const int per = 65535 * 16 * mt;   // activation rows of one launch (grid.y)
    for (int r0 = 0; r0 < m; r0 += per) {
        const int mc = std::min(per, m - r0);
        const dim3 grid((w->n + 15) / 16, (mc + 16 * mt - 1) / (16 * mt));
        const uint8_t *ac = codes + (size_t)r0 * (w->k / 2), *as = scales + (size_t)r0 * (w->k / kMxBlock);
        T *out = y + (size_t)r0 * w->n;
        if (mt == 1)
            hipLaunchKernelGGL((mx_rows_kernel<1, T>), grid, dim3(64 * waves), 0, stream, w->codes, w->scales, ac, as, mc, w->n, w->k, out);
        else if (mt == 2)
            hipLaunchKernelGGL((mx_rows_kernel<2, T>), grid, dim3(64 * waves), 0, stream, w->codes, w->scales, ac, as, mc, w->n, w->k, out);
        else
            hipLaunchKernelGGL((mx_rows_kernel<4, T>), grid, dim3(64 * waves), 0, stream, w->codes, w->scales, ac, as, mc, w->n, w->k, out);
        if (hipGetLastError() != hipSuccess)
            return TB_EHIP;
    }
    return TB_OK;
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
    (void)w;
    (void)m;
    return 0;
}

int tb_mxfp4_gemm(const tb_mxfp4 *w, const uint8_t *codes, const uint8_t *scales, int m, void *y, int dtype, void *ws,
                  size_t ws_bytes, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    if (!eb || !mx_ok(w) || m < 1)
        return TB_EINVAL;
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
    case TB_F32: return launch_gemm(w, codes, scales, m, static_cast<float *>(y), st);
    case TB_BF16: return launch_gemm(w, codes, scales, m, static_cast<Bf16 *>(y), st);
    default: return launch_gemm(w, codes, scales, m, static_cast<F16 *>(y), st);
    }
}

}  // extern "C"
