// Device and host helpers of the 8-bit kernels: e4m3 values with one binary32 scale per 128 inputs.
//
// A group of up to 128 values v is held as e4m3 numbers q and one scale s:
//   m = max |v|,  s = max(m / 448, 2^-126),  q = e4m3(v * (1/s)),
// m / 448, 1 / s and the product each rounded once to binary32, then to the nearest e4m3 (ties to
// even).  448 is the largest finite e4m3 value, so |v * (1/s)| stays below 464, the first value that
// would round past it.  m is taken over the bit patterns of |v| as integers: NaN > infinity > finite,
// so a group that holds either gets a NaN or infinite scale and reads back as NaN throughout.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_common.h"

namespace moe {

constexpr int kFp8Group = 128;  // inputs per scale
constexpr int kFp8Frag = 2048;  // bytes of a fragment: 16 rows x 128 inputs

inline int fp8_groups(int n) { return (n + kFp8Group - 1) / kFp8Group; }

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float fp8_scale(uint32_t max_bits) {
    const float s = as_f32(max_bits) / 448.0f;
    return s < 0x1p-126f ? 0x1p-126f : s;  // a NaN scale stays
}

// four values times r -> four e4m3 bytes, the first in the lowest byte (round to nearest even)
__device__ __forceinline__ uint32_t fp8_pack4(float v0, float v1, float v2, float v3, float r) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v0 * r, v1 * r, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v2 * r, v3 * r, w, true);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return as_u32(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// largest value of the 16 lanes of a row, in all of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = umax(v, dpp_u32<0xB1>(v));   // lane ^ 1
    v = umax(v, dpp_u32<0x4E>(v));   // lane ^ 2
    v = umax(v, dpp_u32<0x141>(v));  // the partner quad of 8
    return umax(v, dpp_u32<0x140>(v));  // the partner 8 lanes of 16
}
// largest value of lanes l, l ^ 16, l ^ 32, l ^ 48, in all of them
__device__ __forceinline__ uint32_t quarter_max(uint32_t v) {
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const uint32_t a0 = a[0], a1 = a[1];
    v = umax(a0, a1);
    auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const uint32_t b0 = b[0], b1 = b[1];
    return umax(b0, b1);
}

// The sum over 128 inputs of the products of 16 matrix rows (a) and 16 tokens (b): lane l holds, of
// both, row l % 16 and the same 32 of the inputs, in the same order; result: token l % 16, rows
// 4 (l / 16) .. + 3.
//
// The matrix core's e4m3 instructions cut the products of each run of 8 consecutive inputs off towards zero, below
// 2^(E - 13), where 2^E is the largest product of two operands' powers of two in the run (2^-6 for a subnormal; zeros
// do not count), and add the runs in binary32.  448 * 448 - 448 * 448 + 6 * 4 gives 0: E = 16, what lies below 8 is gone
// (measured, the 32- and the 128-input forms alike).  A run of 8 is off by less than 2^(E - 10), so a sum of normal
// operands by less than 2^-10 of the sum of its products' magnitudes; on bell-shaped operands by 1.5e-5 of the result.
// mfma_fp8 is that, at twice the bf16 rate: taken where the sum is rounded to bf16 (half a step is 2^-8) and stored.
// mfma_fp8_exact widens both operands to bf16 (exact) and uses the bf16 instruction, whose sums are binary32 (5e-7
// measured): where the weights' bytes bound the product anyway, where the caller wants a binary32 result, and for
// h, which is rounded to 8 bits and multiplied again.
__device__ __forceinline__ f32x4_t mfma_fp8(i32x8_t a, i32x8_t b) {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

typedef __bf16 bf16v2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16v8_t __attribute__((ext_vector_type(8)));

// two values rounded to bf16 (nearest even) by the hardware's conversion, the first in the low half
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16v2_t));
}

struct Wide8 {  // a lane's 32 inputs as bf16
    bf16v8_t v[4];
};

__device__ __forceinline__ Wide8 widen(i32x8_t p) {
    Wide8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bf16v2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)p[i], 1.0f, false);
        const bf16v2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)p[i], 1.0f, true);
        o.v[i / 2][4 * (i & 1)] = lo[0];
        o.v[i / 2][4 * (i & 1) + 1] = lo[1];
        o.v[i / 2][4 * (i & 1) + 2] = hi[0];
        o.v[i / 2][4 * (i & 1) + 3] = hi[1];
    }
    return o;
}

__device__ __forceinline__ f32x4_t mfma_fp8_exact(const Wide8& a, const Wide8& b) {
    f32x4_t c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ i32x8_t join8(u32x4_t lo, u32x4_t hi) {
    return i32x8_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

}  // namespace moe
