// Internal interface between moe_lora_linear and its kernels.
#pragma once

#include "moe_common.h"

namespace moe {

struct LoraArgs {
    const uint16_t* x;  // [M, K] bf16
    size_t ldx;
    int M, K;
    const uint16_t* w;  // [N, K] bf16 or nullptr
    size_t ldw;
    int N;
    const void* base;  // [M, N] or nullptr
    size_t ldb;
    const uint16_t* a;  // [n, r, K]
    const uint16_t* b;  // [n, N, r]
    int r, n;
    const float* scale;      // [n]
    const int32_t* rank;     // [n] or nullptr
    const int32_t* adapter;  // [M]
    void* y;                 // [M, N]
    size_t ldy;
    float* v;  // workspace [M, r]
    float* part;  // workspace [splits, M, N]: sums of x W^T over runs of the inputs
    int splits;   // 0: launch 2 forms x W^T
    bool wide;  // the rows of y and base start on 16 bytes
};

// an element of base or y
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return f32_to_bf16(v); }

// runs of the inputs whose sums launch 1 leaves
constexpr size_t kLoraPartBytes = (size_t)1 << 20;
int lora_splits(const LoraArgs& p);
// one row, a low rank and a workgroup a compute unit: v is formed by the launch that uses it
bool lora_alone(const LoraArgs& p);
// v = scale A x for the rows that have an adapter
moe_status lora_shrink(const LoraArgs& p, hipStream_t st);
// y = x W^T + base + v B^T, any shape
moe_status lora_rows(const LoraArgs& p, moe_dtype base, moe_dtype out, hipStream_t st);

}  // namespace moe
