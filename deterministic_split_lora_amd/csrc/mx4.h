// MX4 building blocks: E2M1 codes in pairs (element 2i in the low four bits of
// byte i), one E8M0 scale byte b for kMxBlock elements, value = code 2^(b-127);
// b = 255 makes the block NaN.
#pragma once

#include "device.h"
#include "step_kernels.h"

namespace lora {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The scale 2^(b-127) as the fp32 operand of the conversion instructions, which
// take its exponent field alone (so 0 stands for 2^-127 and 255 for NaN).
__device__ __forceinline__ float mx_scale_f32(uint32_t b)
{
    return __builtin_bit_cast(float, b << 23);
}

// Eight codes (one 32-bit word) as bf16, times the scale.  Exact: a code has two
// significant bits.
__device__ __forceinline__ bf16x8 mx4_to_bf16(uint32_t w, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

constexpr int kFp4 = 4;                      // the matrix-core format selector of E2M1

// One operand row's blocks of a step: codes and scale.
struct MxOperand {
    u32x4 q;
    uint32_t s;
};

__device__ __forceinline__ f32x4 mfma_mx4(const MxOperand& w, const MxOperand& x, f32x4 acc)
{
    const i32x8 a = {(int)w.q[0], (int)w.q[1], (int)w.q[2], (int)w.q[3], 0, 0, 0, 0};
    const i32x8 b = {(int)x.q[0], (int)x.q[1], (int)x.q[2], (int)x.q[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, 0, (int)w.s, 0, (int)x.s);
}

// Eight bf16 (in pairs) divided by the scale, as codes: nearest, ties to even,
// saturated at 6.  (The words are copied out first: a bit cast straight from a
// vector's element reads its first element.)
__device__ __forceinline__ uint32_t bf16_to_mx4(u32x4 v, float scale)
{
    const uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v0), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v1), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v2), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v3), scale, 3);
}

// Codes of block g in lane group g, element pairs 4d .. 4d+3 in word d, to the
// words of block s in q[s], lane group g holding word g: a 4 x 4 transpose of
// (lane group, word).
__device__ __forceinline__ void transpose_groups(u32x4& q)
{
    uint32_t a = q[0], b = q[1], c = q[2], d = q[3];
    const auto ac = __builtin_amdgcn_permlane32_swap(a, c, false, false);
    const auto bd = __builtin_amdgcn_permlane32_swap(b, d, false, false);
    const auto ab = __builtin_amdgcn_permlane16_swap(ac[0], bd[0], false, false);
    const auto cd = __builtin_amdgcn_permlane16_swap(ac[1], bd[1], false, false);
    q = u32x4{ab[0], ab[1], cd[0], cd[1]};
}

}  // namespace lora
