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
    int c_vec;   // rows of c start on 16 bytes
};

inline int64_t blocks_of(int64_t n, int block) { return (n + block - 1) / block; }

// four consecutive columns n .. of row m of c
__device__ __forceinline__ void store_c4(const GemmFp8& g, int m, int n, f32x4_t v) {
    if (g.c_vec && n + 3 < g.N) {
        if (g.c_bf16) {
            uint2 o;
            o.x = bf16_pair(v[0], v[1]);
            o.y = bf16_pair(v[2], v[3]);
            *(uint2*)((uint16_t*)g.c + (size_t)m * g.ldc + n) = o;
        } else {
            *(float4*)((float*)g.c + (size_t)m * g.ldc + n) = make_float4(v[0], v[1], v[2], v[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < g.N) {
            if (g.c_bf16) ((uint16_t*)g.c)[(size_t)m * g.ldc + n + i] = f32_to_bf16(v[i]);
            else ((float*)g.c)[(size_t)m * g.ldc + n + i] = v[i];
        }
}

// A grouped call: FfnArgs with x either bf16 rows (x_scale NULL) or e4m3 rows with their scales.
// The streaming kernels (calls of up to kFp8Stream tokens) keep the intermediate rows of h in binary32 (a.h)
// and quantise them, and bf16 rows of x where x8 is NULL, as they load them; the tiles read x8 / x_scale
// and keep h8 / h_scale.
struct FfnFp8 {
    FfnArgs a;
    const float* x_scale;
    const uint8_t* x8 = nullptr;
    uint8_t* h8 = nullptr;
    float* h_scale = nullptr;
};
// Up to 16 tokens a streamed call is one token block an expert.  16 tokens on 50 of 256 experts of 4096 x 2048 and the
// shared one take 234 us streamed, 17 on 51 256 us in tiles; where all choose the same 6 experts, which is rare, 85 and 58.
constexpr int kFp8Stream = 16;

// bf16 rows [T, d], back to back, into e4m3 rows and scales (norm.hip)
moe_status quant_rows_bf16(const void* x, int T, int d, uint8_t* q, float* scale, hipStream_t st);

// few rows (fp8_stream.hip): the weights are streamed once
moe_status gemm_fp8_stream(const GemmFp8& g, hipStream_t st);
float gemm_fp8_stream_us(const GemmFp8& g);
moe_status ffn_fp8_stream(const FfnFp8& f, int mode, hipStream_t st);
// many rows (fp8_tile.hip): the tile with the least estimated time (us; NULL: none applies), its launch
const void* gemm_fp8_best_tile(const GemmFp8& g, float& us);
moe_status gemm_fp8_tile(const GemmFp8& g, const void* tile, hipStream_t st);
moe_status ffn_fp8_tile(const FfnFp8& f, int mode, hipStream_t st);
// both projections of a grouped call with 8-bit weights
moe_status ffn_fp8_run(const FfnFp8& f, hipStream_t st);
size_t ffn_fp8_workspace(int T, int d, int f, int k, int has_shared);

}  // namespace moe
