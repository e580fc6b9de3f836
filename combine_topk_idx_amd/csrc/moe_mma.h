// Device building blocks of the expert products: matrix-instruction fragments,
// block scales, and the E4M3 quantization of a row group held in registers.
#pragma once

#include "moe_device.h"
#include "moe_experts_internal.h"

namespace moe {
namespace dev {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr bool per_row_weight_scale(int quant) { return quant == MOE_QUANT_MXFP8; }

// fp32 -> bf16 bits, round to nearest even; infinities and NaN stay what they are.
__device__ __forceinline__ uint32_t bf16_bits(float f)
{
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return bf16_bits(lo) | bf16_bits(hi) << 16; }

// 16 E4M3 values (16 bytes) times a power of two -> two bf16 operands of 8, exact.
__device__ __forceinline__ void to_bf16(const u32x4 &v, float scale, bf16x8 &lo, bf16x8 &hi)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], scale, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], scale, true);
        lo[4 * j] = a[0], lo[4 * j + 1] = a[1], lo[4 * j + 2] = b[0], lo[4 * j + 3] = b[1];
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + j], scale, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + j], scale, true);
        hi[4 * j] = c[0], hi[4 * j + 1] = c[1], hi[4 * j + 2] = d[0], hi[4 * j + 3] = d[1];
    }
}

// One lane's share of a row's block of 128 channels -- the 16 bytes at 16 g (lo)
// and at 64 + 16 g (hi) -- as four bf16 operands of v_mfma_f32_16x16x32_bf16,
// times the block's scale where that is a power of two (`s`: as it is stored; the
// word of four bytes for MXFP8, whose blocks g / 2 and 2 + g / 2 the lane has).
// The conversion takes the scale's exponent field alone: byte 0 is 2^-127, 255 NaN.
// Exact while the value fits bf16 (2^-133 .. 2^128): for bytes 3 .. 246 all do.
template <int QUANT>
__device__ __forceinline__ void block_to_bf16(const u32x4 &lo, const u32x4 &hi, uint32_t s, int g, bf16x8 v[4])
{
    float a = 1.0f, b = 1.0f;
    if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
        a = b = __uint_as_float(s << 23);
    } else if constexpr (QUANT == MOE_QUANT_MXFP8) {
        const uint32_t two = s >> (4 * (g & 2));
        a = __uint_as_float((two & 0xFFu) << 23);
        b = __uint_as_float((two >> 16 & 0xFFu) << 23);
    }
    to_bf16(lo, a, v[0], v[1]);
    to_bf16(hi, b, v[2], v[3]);
}

// silu(g) * u
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// The scale of a block with largest magnitude `amax`, the factor that E4M3
// values are made with, and how the scale is stored -- for finite values the
// rules of the dispatch (store_item in moe_device.h).  A maximum passes over NaN.
template <int QUANT>
struct BlockScale {
    float s;        // FP8_F32: values are divided by it; power-of-two formats: multiplied by it
    uint32_t byte;  // power-of-two formats: the stored exponent byte
    __device__ __forceinline__ explicit BlockScale(float amax)
    {
        const float af = fmaxf(amax, 1e-10f);
        byte = 0;
        if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            s = af / 448.0f;
        } else {
            const uint32_t ab = __float_as_uint(af);
            int e = (int)(ab >> 23) - 127 - 8;
            if (QUANT == MOE_QUANT_FP8_UE8M0)
                e += (ab & 0x7FFFFFu) > 0x600000u ? 1 : 0;
            s = __uint_as_float((uint32_t)(127 - e) << 23);
            byte = (uint32_t)(e + 127);
        }
    }
    __device__ __forceinline__ float apply(float v) const
    {
        const float d = QUANT == MOE_QUANT_FP8_F32 ? v / s : v * s;
        const float in = fminf(fmaxf(d, -448.0f), 448.0f);
        return d != d ? d : in;  // the clamp alone would make a NaN -448
    }
};

}  // namespace dev
}  // namespace moe
