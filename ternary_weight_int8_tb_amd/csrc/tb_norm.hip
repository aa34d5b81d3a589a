// tb_norm.hip -- residual addition, root-mean-square norm and rotated int8 rows (gfx950).
//
//   s = round_T(x + res)             T: the type of the rows; sums in fp32
//   r = 1 / sqrt(mean(s^2) + eps)
//   u = H (s * gamma)                per 128-block; the sums of tb_rotate_quant_i8
//   q = rint(u * (127 / amax)), dq = amax * (r * unit), amax = max |u|
//   y = round_T((s * r) * gamma)     if it is wanted
//
// The quantiser does not see a factor that a whole block shares, so r, the one number that needs
// the whole row, goes into dq alone: q is final as soon as its block has been read, and the row
// is read once. It also makes q independent of how the row's squares are summed.
//
// Bound: memory. A workgroup holds a whole row; 16 lanes hold a 128-block, 8 elements each, and all
// exchanges are DPP. Squares are taken and summed in fp64, where those of any fp32 number fit, so that
// neither the rows' magnitude, nor their length, nor the order of the waves shows in the fp32 result.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tb.h"
#include "tb_host.h"
#include "tb_rows.h"

namespace {

using namespace tbr;

constexpr int kBlock = 128;
constexpr int kMaxThreads = 1024;
constexpr int kMaxGrid = 1 << 20;   // workgroups of a launch; each takes every kMaxGrid-th row
// A block whose largest |u| is below this counts as zero (127 / amax must stay finite).
constexpr float kZeroBlock = 0x1p-100f;

// s of the lane's 8 elements, rounded to T, in fp32.
template <class T>
__device__ __forceinline__ void add_rows(const Eight<T> &x, const Eight<T> &res, bool has_res, Eight<T> &s, float (&v)[8])
{
    x.get(v);
    s = x;
    if (has_res) {
        float b[8];
        res.get(b);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += b[e];
        s.set(v);
        s.get(v);
    }
}

// The lane's 8 of u * r's codes, the sign of rotate_signed taken back; amax: the block's.
__device__ __forceinline__ uint2 codes(const float (&u)[8], float amax, float sign)
{
    uint32_t w[2] = {0u, 0u};
    if (amax >= kZeroBlock && amax < INFINITY) {
        const float inv = (127.0f / amax) * sign;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // |u * inv| <= 127 (1 + 2^-23); adding 1.5 * 2^23 rounds it to an integer, ties
            // to even, whose low byte is the code
            const uint32_t c = __float_as_uint(u[e] * inv + 12582912.0f) & 0xffu;
            w[e >> 2] |= c << (8 * (e & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}

// The block's amax in dq: 0 if it counts as zero, a NaN if it is not finite (infinite ones too: the
// block has no codes).
__device__ __forceinline__ float kept_amax(float amax)
{
    return amax < kZeroBlock ? 0.0f : amax < INFINITY ? amax : NAN;
}

// The sum over a wave's lanes, in every lane.
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const uint64_t b = (uint64_t)__double_as_longlong(v);
        v += __longlong_as_double((long long)((uint64_t)partner((uint32_t)(b >> 32), s) << 32 | partner((uint32_t)b, s)));
    }
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// r of a row from its waves' sums, as up * f: fp32 holds neither 1 / sqrt(mean) of rows of subnormal numbers nor
// its product with unit of the largest rows with all bits. Multiplied by up first, a power of two, s and amax
// give what they would with an r of any exponent.
struct Norm {
    float f, up;
};
__device__ __forceinline__ Norm norm_of(const double *part, int waves, int k, float eps)
{
    double total = 0.0;
    for (int w = 0; w < waves; ++w)
        total += part[w];
    const double mean = total / (double)k + (double)eps;
    if (mean == 0.0)   // a row of zeros, eps = 0
        return {0.0f, 1.0f};
    const float up = mean < 0x1p-200 ? 0x1p64f : mean > 0x1p200 ? 0x1p-64f : 1.0f;
    return {(float)(1.0 / sqrt(mean) / (double)up), up};
}

// Rows of up to 64 blocks: a lane's 8 elements of a row stay in registers until y, those of gamma for
// all rows of the workgroup, and the next row's are on their way while this one's norm is
// summed (8192 rows of 5120 bf16 with res: 85 us with a row per workgroup, which waits for its loads and
// then for its sum; 56 us so).
// LDS is used in turn by odd and even rows, so that one barrier per row is enough.
template <class T>
__global__ __launch_bounds__(kMaxThreads) void add_rmsnorm_quant_kernel(
    const T *x, const T *res, const float *__restrict__ gamma, int m, int nb, float eps, float unit, T *res_out, T *y,
    int8_t *__restrict__ q, float *__restrict__ dq)
{
    __shared__ float amax_s[2][kMaxThreads / 16];
    __shared__ double part_s[2][kMaxThreads / 64];
    const int tid = threadIdx.x, lane16 = tid & 15, b = tid >> 4, waves = blockDim.x >> 6;
    const bool on = b < nb;   // else the group holds no block: it computes with zeros
    const float sign = chunk_sign(lane16);
    const int at = min(b, nb - 1) * kBlock + chunk_of(lane16) * 8;
    float g[8];
    {
        Eight<float> eg;
        eg.load(gamma + at);
        eg.get(g);
    }
    Eight<T> ex, er;
    auto load = [&](size_t row) {
        const size_t i = row * (size_t)nb * kBlock + at;
        ex.load(x + i);
        if (res)
            er.load(res + i);
    };
    load(blockIdx.x);
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)m; row += gridDim.x, turn ^= 1) {
        const size_t i = row * (size_t)nb * kBlock + at;
        Eight<T> es;
        float v[8], u[8];
        add_rows(ex, er, res != nullptr, es, v);
        if (row + gridDim.x < (size_t)m)
            load(row + gridDim.x);
        if (res_out && on)
            es.store(res_out + i);
        double sq = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sq = fma((double)v[e], (double)v[e], sq);
            u[e] = v[e] * g[e];
        }
        const double sum = wave_sum(on ? sq : 0.0);
        if ((tid & 63) == 0)
            part_s[turn][tid >> 6] = sum;
        rotate_signed(u, lane16);
        const float amax = __uint_as_float(amax_bits<4>(u));
        const uint2 c = codes(u, amax, sign);
        if (on)
            *reinterpret_cast<uint2 *>(q + i) = c;
        if (lane16 == 0)
            amax_s[turn][b] = kept_amax(amax);
        __syncthreads();
        if (tid >= 64 && !y)
            continue;
        const Norm r = norm_of(part_s[turn], waves, nb * kBlock, eps);
        if (tid < nb)   // the first wave's lanes
            dq[row * nb + tid] = amax_s[turn][tid] * r.up * (r.f * unit);   // f is finite, or the row holds a NaN
        if (y && on) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (v[e] * r.up * r.f) * g[e];
            es.set(v);
            es.store(y + i);
        }
    }
}

// Longer rows: a row per workgroup, in passes of 64 blocks; for y it is read again.
template <class T>
__global__ __launch_bounds__(kMaxThreads) void add_rmsnorm_quant_long_kernel(
    const T *x, const T *res, const float *__restrict__ gamma, int m, int nb, float eps, float unit, T *res_out, T *y,
    int8_t *__restrict__ q, float *__restrict__ dq)
{
    extern __shared__ float amax_s[];   // [nb]
    __shared__ double part_s[kMaxThreads / 64];
    const int tid = threadIdx.x, lane16 = tid & 15, groups = blockDim.x >> 4;
    const float sign = chunk_sign(lane16);
    const int at = chunk_of(lane16) * 8;

    for (size_t row = blockIdx.x; row < (size_t)m; row += gridDim.x) {
        const size_t base = row * (size_t)nb * kBlock;
        double sum = 0.0;
        for (int b = tid >> 4; b < nb; b += groups) {
            const size_t i = base + (size_t)b * kBlock + at;
            Eight<T> ex, er, es;
            Eight<float> eg;
            ex.load(x + i);
            if (res)
                er.load(res + i);
            eg.load(gamma + b * kBlock + at);
            float v[8], g[8];
            add_rows(ex, er, res != nullptr, es, v);
            if (res_out)
                es.store(res_out + i);
            eg.get(g);
            double sq = 0.0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sq = fma((double)v[e], (double)v[e], sq);
                v[e] *= g[e];
            }
            sum += sq;
            rotate_signed(v, lane16);
            const float amax = __uint_as_float(amax_bits<4>(v));
            *reinterpret_cast<uint2 *>(q + i) = codes(v, amax, sign);
            if (lane16 == 0)
                amax_s[b] = kept_amax(amax);
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0)
            part_s[tid >> 6] = sum;
        __syncthreads();
        const Norm r = norm_of(part_s, blockDim.x >> 6, nb * kBlock, eps);
        for (int b = tid; b < nb; b += blockDim.x)
            dq[row * nb + b] = amax_s[b] * r.up * (r.f * unit);   // f is finite, or the row holds a NaN

        if (y)
            for (int b = tid >> 4; b < nb; b += groups) {
                const size_t i = base + (size_t)b * kBlock + at;
                Eight<T> ex, er, es;
                Eight<float> eg;
                float v[8], g[8];
                // res_out may be x or res itself: what this lane stored there is s
                ex.load(res_out ? res_out + i : x + i);
                if (res && !res_out)
                    er.load(res + i);
                eg.load(gamma + b * kBlock + at);
                add_rows(ex, er, res && !res_out, es, v);
                eg.get(g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = (v[e] * r.up * r.f) * g[e];
                es.set(v);
                es.store(y + i);
            }
        __syncthreads();   // the next row's maxima and sums take this one's place
    }
}

template <class T>
int launch(const void *x, const void *res, const float *gamma, int m, int k, float eps, void *res_out, void *y,
           int8_t *q, float *dq, hipStream_t stream)
{
    const int nb = k / kBlock;
    const T *xs = static_cast<const T *>(x), *rs = static_cast<const T *>(res);
    T *ro = static_cast<T *>(res_out), *ys = static_cast<T *>(y);
    if (nb <= kMaxThreads / 16) {
        // as many workgroups as the chip holds: 256 CUs of 32 waves
        const int waves = (nb + 3) / 4;
        hipLaunchKernelGGL(add_rmsnorm_quant_kernel<T>, dim3(std::min(m, 256 * (32 / waves))), dim3(64 * waves), 0, stream,
                           xs, rs, gamma, m, nb, eps, tbh::dq_unit(), ro, ys, q, dq);
    } else {
        // the row's blocks in as few equal passes as 1024 threads allow
        const int passes = (nb + kMaxThreads / 16 - 1) / (kMaxThreads / 16);
        const int waves = ((nb + passes - 1) / passes + 3) / 4;
        hipLaunchKernelGGL(add_rmsnorm_quant_long_kernel<T>, dim3(std::min(m, kMaxGrid)), dim3(64 * waves), (size_t)nb * 4,
                           stream, xs, rs, gamma, m, nb, eps, tbh::dq_unit(), ro, ys, q, dq);
    }
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

}  // namespace

extern "C" int tb_add_rmsnorm_quant_i8(const void *x, const void *res, const float *gamma, int dtype, int m, int k,
                                       float eps, void *res_out, void *y, int8_t *q, float *dq, void *stream)
{
    const size_t eb = tbh::dtype_bytes(dtype);
    if (!eb || m < 1 || k < kBlock || k % kBlock || !(eps >= 0.0f) || eps > 3.0e38f)
        return TB_EINVAL;
    const size_t rows = (size_t)m * (size_t)k * eb;
    // res_out may be x or res itself: each element is read by the lane that then writes it
    tbh::Arg a[8] = {{gamma, (size_t)k * 4, false},
                     {q, (size_t)m * k, true},
                     {dq, (size_t)m * (k / kBlock) * 4, true},
                     {x, rows, res_out == x}};
    size_t n = 4;
    if (res && res != x)
        a[n++] = {res, rows, res_out == res};
    if (y)
        a[n++] = {y, rows, true};
    if (res_out && res_out != x && res_out != res)
        a[n++] = {res_out, rows, true};
    if (int rc = tbh::check_args(a, n))
        return rc;
    // block maxima wait in LDS for the row's norm
    if (k / kBlock > 15 * 1024)
        return TB_EUNSUPPORTED;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
    case TB_F32: return launch<float>(x, res, gamma, m, k, eps, res_out, y, q, dq, st);
    case TB_BF16: return launch<Bf16>(x, res, gamma, m, k, eps, res_out, y, q, dq, st);
    default: return launch<F16>(x, res, gamma, m, k, eps, res_out, y, q, dq, st);
    }
}
