// Internal interface of the 8-bit matrix products: the dense one (moe_gemm_fp8) and the routed
// experts' two projections over 8-bit slots.
#pragma once

#include "ffn.h"
#include "fp8.h"

namespace moe {

// c[m, n] = sum over 128-input groups g of a_scale[m, g] w_scale[n / 128, g] sum_{k in g} a[m, k] w[n, k]
struct GemmFp8 {
    const uint8_t* a;
    size_t lda;
    const float* a_scale;  // [M, G]
    const uint8_t* w;
    size_t ldw;
    const float* w_scale;  // [ceil(N / 128), G]
    void* c;
    size_t ldc;
    int M, N, K, G;
    int c_bf16;  // c elements: bf16 (each sum rounded once), else binary32
    int c_vec;   // four consecutive elements of c may be stored at once
};

// A grouped call: FfnArgs with x either bf16 rows (x_scale NULL, quantised as they are loaded) or
// e4m3 rows with their scales; h holds the intermediate rows in binary32.
struct FfnFp8 {
    FfnArgs a;
    const float* x_scale;
};

moe_status gemm_fp8_stream(const GemmFp8& g, hipStream_t st);
moe_status ffn_fp8_stream(const FfnFp8& f, int mode, hipStream_t st);
// both projections of a grouped call with 8-bit weights
moe_status ffn_fp8_run(const FfnFp8& f, hipStream_t st);
size_t ffn_fp8_workspace(int T, int d, int f, int k, int has_shared);

}  // namespace moe
