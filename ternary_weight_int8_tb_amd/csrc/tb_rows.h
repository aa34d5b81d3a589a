// tb_rows.h -- device building blocks of the row operators (norm, 4-bit quantiser): loads and
// stores of 8 elements in three types, and the 128-block Walsh-Hadamard transform in registers.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "tb.h"

namespace tbr {

// Eight consecutive elements of type T, as fp32. bf16 and fp16 come as one 16-byte load.
struct Bf16 {
    uint16_t bits;
};
struct F16 {
    uint16_t bits;
};
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack(uint32_t w, float &lo, float &hi, Bf16)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(uint32_t w, float &lo, float &hi, F16)
{
    const h2 v = __builtin_bit_cast(h2, w);
    lo = (float)v.x;
    hi = (float)v.y;
}
// Two values rounded to nearest, ties to even.
__device__ __forceinline__ uint32_t pack(float lo, float hi, Bf16)
{
    return __builtin_bit_cast(uint32_t, b2{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, F16)
{
    return __builtin_bit_cast(uint32_t, h2{(_Float16)lo, (_Float16)hi});
}

template <class T>
struct Eight {
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        unpack(w.x, v[0], v[1], T());
        unpack(w.y, v[2], v[3], T());
        unpack(w.z, v[4], v[5], T());
        unpack(w.w, v[6], v[7], T());
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        w = make_uint4(pack(v[0], v[1], T()), pack(v[2], v[3], T()), pack(v[4], v[5], T()), pack(v[6], v[7], T()));
    }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = w; }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
};

// The 8-element chunk of a 128-block that lane L (0 .. 15) of its 16-lane group holds. The
// four lane exchanges of the transform are single DPP operations: quad_perm (lane ^ 1, ^ 2),
// row_half_mirror (lane ^ 7) and row_ror:8 (lane ^ 8). Their partners differ in exactly one
// bit of this chunk index, in ascending order.
__device__ __forceinline__ int chunk_of(int lane16) { return lane16 ^ ((lane16 & 4) ? 3 : 0); }

// One exchange stage on 8 registers: v += c * v(partner), c = +1 in the lane whose chunk bit is
// 0 and -1 in the other. The first lane then holds a + b; the second holds b - a where the
// transform wants a - b: all later stages see that sign on both partners, so it stays a sign
// of the lane (chunk_sign) until the end, and every sum is one fp32 rounding of the exact
// a + b or a - b. s_nop 1: a DPP read needs two wait states after a VALU write.
#define TBR_STAGE(CTRL)                                                                    \
    asm("s_nop 1\n\t"                                                                      \
        "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                \
        "s_nop 1"                                                                          \
        : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]),          \
          "+v"(v[6]), "+v"(v[7])                                                           \
        : "v"(c))

__device__ __forceinline__ float chunk_sign(int lane16)
{
    return (__builtin_popcount(chunk_of(lane16)) & 1) ? -1.0f : 1.0f;
}

// u = H v of one 128-block held by 16 lanes (all active), spans 1, 2, ..., 64 in that order, each
// (a, b) -> (a + b, a - b) in fp32: the sums that tb_rotate_quant_i8 makes, bit for bit, except
// that lane L's results carry the factor chunk_sign(L) (which the caller folds into a product).
__device__ __forceinline__ void rotate_signed(float (&v)[8], int lane16)
{
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!(e & h)) {
                const float a = v[e], b = v[e + h];
                v[e] = a + b;
                v[e + h] = a - b;
            }
        }
    }
    const int ch = chunk_of(lane16);
    float c = (ch & 1) ? -1.0f : 1.0f;
    TBR_STAGE("quad_perm:[1,0,3,2]");
    c = (ch & 2) ? -1.0f : 1.0f;
    TBR_STAGE("quad_perm:[2,3,0,1]");
    c = (ch & 4) ? -1.0f : 1.0f;
    TBR_STAGE("row_half_mirror");
    c = (ch & 8) ? -1.0f : 1.0f;
    TBR_STAGE("row_ror:8");
}
#undef TBR_STAGE

// The value of the lane's exchange partner of stage s (0 .. 3), by DPP.
__device__ __forceinline__ uint32_t partner(uint32_t v, int s)
{
    switch (s) {
    case 0: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
    case 1: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
    case 2: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);
    default: return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false);
    }
}

// Largest |v| over the 16 lanes' registers (in every lane). STAGES: 4 for the whole block, 2 for
// the lane's 32 elements. On bit patterns: the order of non-negative floats, with a NaN above
// infinity, so a value that is not finite shows in the result.
template <int STAGES>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        a = max(a, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
        a = max(a, partner(a, s));
    return a;
}

}  // namespace tbr
