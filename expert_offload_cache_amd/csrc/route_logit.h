// The router's logits for a few tokens: the part of the fixed summation order that one lane does.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_common.h"

namespace moe {

// acc + a*b with two roundings (a*b exact for bf16 inputs, so a fused form gives the same bits)
template <bool kBf16>
__device__ __forceinline__ float madd(float acc, float a, float b) {
    if constexpr (kBf16) {
        return __builtin_fmaf(a, b, acc);
    } else {
#pragma clang fp contract(off)
        float p = a * b;
        return acc + p;
    }
}

template <bool kBf16>
__device__ __forceinline__ float load_elem(const void* base, size_t i) {
    if constexpr (kBf16) return bf16_to_f32(((const uint16_t*)base)[i]);
    else return ((const float*)base)[i];
}

// acc[i] = segment `lane` (d / 64 inputs, in ascending order from +0) of the product of row t0 + i of x
// and row e of w; tokens past the last repeat it.  wave_tree_sum joins the 64 segments.
template <bool kBf16, int TB>
__device__ __forceinline__ void logit_segments(const void* __restrict__ x, const void* __restrict__ w, int T, int d, int t0,
                                               int e, int lane, float (&acc)[TB]) {
    const int S = d / 64;
    const size_t seg = (size_t)lane * S;
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i] = 0.f;
    if (kBf16 && S % 8 == 0) {
        const uint4* wr = (const uint4*)((const uint16_t*)w + (size_t)e * d + seg);
        const uint4* xr[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i) xr[i] = (const uint4*)((const uint16_t*)x + (size_t)min(t0 + i, T - 1) * d + seg);
        const int nv = S / 8;
        constexpr int CG = TB == 1 ? 8 : 4;  // chunks whose loads are issued together
        for (int c0 = 0; c0 < nv; c0 += CG) {
            uint4 wv[CG], xv[CG][TB];
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                const int cc = min(c0 + c, nv - 1);
                wv[c] = wr[cc];
#pragma unroll
                for (int i = 0; i < TB; ++i) xv[c][i] = xr[i][cc];
            }
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                if (c0 + c < nv) {
                    const uint32_t ws[4] = {wv[c].x, wv[c].y, wv[c].z, wv[c].w};
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int i = 0; i < TB; ++i) {
                            const uint32_t xs = h == 0 ? xv[c][i].x : h == 1 ? xv[c][i].y : h == 2 ? xv[c][i].z : xv[c][i].w;
                            acc[i] = madd<true>(acc[i], bf16_lo(xs), bf16_lo(ws[h]));
                            acc[i] = madd<true>(acc[i], bf16_hi(xs), bf16_hi(ws[h]));
                        }
                }
            }
        }
    } else {
        for (int j = 0; j < S; ++j) {
            const float wj = load_elem<kBf16>(w, (size_t)e * d + seg + j);
#pragma unroll
            for (int i = 0; i < TB; ++i)
                acc[i] = madd<kBf16>(acc[i], load_elem<kBf16>(x, (size_t)min(t0 + i, T - 1) * d + seg + j), wj);
        }
    }
}

}  // namespace moe
