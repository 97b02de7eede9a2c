// moe_lora_linear: a projection with a low-rank adapter for each row.
//
//   y[m,:] = x[m,:] W^T + base[m,:] + scale_a (x[m,:] A_a^T) B_a^T,   a = adapter[m]
//
// Launch 1 (lora_shrink_kernel): v[m,:] = scale_a A_a x[m,:] for the rows that have an adapter, in binary32.
// Launch 2: the projection, with the adapters' second product at its end.
//
// v is binary32 and the matrix instructions take bf16, so v enters as a sum of bf16 parts: v1 = bf16(v),
// v2 = bf16(v - v1), v3 = bf16(v - v1 - v2); two parts hold 16 bits of it, which is beyond what a bf16
// result shows, three all 24.  r is small beside K, so the parts cost little.
//
// Rows of several adapters share a tile: each adapter's product is formed for the whole tile and taken over
// for its own rows only, by selection, so that an adapter with infinities or NaN touches no other
// request's rows.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp8.h"
#include "lora.h"

namespace moe {
namespace {

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4_t zero4() { return u32x4_t{0u, 0u, 0u, 0u}; }
__device__ __forceinline__ f32x4_t zerof() { return f32x4_t{0.f, 0.f, 0.f, 0.f}; }

// a row's adapter, or -1
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int m) {
    const int a = m < p.M ? p.adapter[m] : -1;
    return a >= 0 && a < p.n ? a : -1;
}
__device__ __forceinline__ int rank_of(const LoraArgs& p, int a) { return p.rank ? min(max(p.rank[a], 0), p.r) : p.r; }

// ---- launch 1 ---------------------------------------------------------------------------------------
// A workgroup takes 16 * NM rows and NR blocks of 16 ranks; its 8 waves split the inputs.  The adapters of
// its rows are taken one after the other (blockIdx.z, gridDim.z apart).
constexpr int kShrinkWaves = 8;

template <int NM, int NR>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(LoraArgs p) {
    __shared__ float red[kShrinkWaves * NM * 256];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x * 16 * NM, r0 = blockIdx.y * 16 * NR;
    // every wave: lane i holds row i's adapter (NM <= 4), `first` marks the rows whose adapter has not come before
    const int mine = lane < 16 * NM ? adapter_of(p, m0 + lane) : -1;
    uint64_t left = __ballot(mine >= 0);
    int turn = 0;
    const int nst = (p.K + 31) / 32, s0 = wv * nst / kShrinkWaves, s1 = (wv + 1) * nst / kShrinkWaves;
    while (left) {
        const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(left), 64));
        const uint64_t rows = __ballot(mine == a);
        left &= ~rows;
        if (turn++ % (int)gridDim.z != (int)blockIdx.z) continue;
        const int rank = rank_of(p, a);
        if (r0 >= rank) continue;
        const uint16_t* A = p.a + (size_t)a * p.r * p.K;
        f32x4_t acc[NM][NR];
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) acc[i][j] = zerof();
        const uint16_t *xr[NM], *ar[NR];
#pragma unroll
        for (int i = 0; i < NM; ++i) xr[i] = p.x + (size_t)min(m0 + 16 * i + r16, p.M - 1) * p.ldx + 8 * q;
#pragma unroll
        for (int j = 0; j < NR; ++j) ar[j] = A + (size_t)min(r0 + 16 * j + r16, p.r - 1) * p.K + 8 * q;
        constexpr int C = NM * NR <= 2 ? 8 : NM * NR <= 8 ? 4 : 2;  // steps whose loads are issued together
        for (int s = s0; s < s1; s += C) {
            u32x4_t vx[C][NM], va[C][NR];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bool in = s + c < s1 && (s + c) * 32 + 8 * q < p.K;
#pragma unroll
                for (int i = 0; i < NM; ++i) vx[c][i] = in ? *(const u32x4_t*)(xr[i] + (size_t)(s + c) * 32) : zero4();
#pragma unroll
                for (int j = 0; j < NR; ++j) va[c][j] = in ? *(const u32x4_t*)(ar[j] + (size_t)(s + c) * 32) : zero4();
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int i = 0; i < NM; ++i) acc[i][j] = mfma_bf16(va[c][j], vx[c][i], acc[i][j]);
        }
        const float scale = p.scale[a];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NM; ++i) *(f32x4_t*)&red[(wv * NM + i) * 256 + r16 * 16 + 4 * q] = acc[i][j];
            __syncthreads();
            for (int o = tid; o < NM * 256; o += 64 * kShrinkWaves) {
                const int i = o >> 8, t = (o >> 4) & 15, c = r0 + 16 * j + (o & 15);
                float s = red[o];
#pragma unroll
                for (int w = 1; w < kShrinkWaves; ++w) s += red[w * NM * 256 + o];
                if (((rows >> (16 * i + t)) & 1) && c < rank) p.v[(size_t)(m0 + 16 * i + t) * p.r + c] = scale * s;
            }
        }
        __syncthreads();
    }
}

// ---- launch 2 ---------------------------------------------------------------------------------------
// 8 values of v as bf16 parts
template <int PARTS>
__device__ __forceinline__ void split_v(const float (&v)[8], u32x4_t (&part)[PARTS]) {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
    for (int n = 0; n < PARTS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = bf16_pair(rest[2 * i], rest[2 * i + 1]);
            part[n][i] = w;
            // an infinite part leaves nothing (not infinity minus infinity)
            const float lo = bf16_lo(w), hi = bf16_hi(w);
            rest[2 * i] = fabsf(lo) < INFINITY ? rest[2 * i] - lo : 0.f;
            rest[2 * i + 1] = fabsf(hi) < INFINITY ? rest[2 * i + 1] - hi : 0.f;
        }
}

// the elements of a 16-byte chunk from element `n` on cleared
__device__ __forceinline__ u32x4_t keep_first(u32x4_t v, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i >= n) v[i] = 0;
        else if (2 * i + 1 >= n) v[i] &= 0xFFFFu;
    }
    return v;
}

// A wave takes 16 rows x 64 columns: 4 operand blocks of weight rows.  Row i of block b is column
// 16 (i / 4) + 4 b + i % 4, so that a lane's results are 16 neighbouring columns of one row.
template <typename OutT, typename BaseT, int PARTS>
__global__ __launch_bounds__(256) void lora_rows_kernel(LoraArgs p) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 64, m0 = (blockIdx.y * 4 + wv) * 16;
    if (m0 >= p.M) return;  // the whole wave
    const int m = m0 + r16;
    int col[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) col[b] = min(n0 + 16 * (r16 >> 2) + 4 * b + (r16 & 3), p.N - 1);
    f32x4_t acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[b] = zerof();
    if (p.w) {
        const uint16_t* xr = p.x + (size_t)min(m, p.M - 1) * p.ldx;
        for (int k = 8 * q; k < (p.K + 31) / 32 * 32; k += 32) {
            const bool in = k < p.K;
            const u32x4_t x = in ? *(const u32x4_t*)(xr + k) : zero4();
#pragma unroll
            for (int b = 0; b < 4; ++b)
                acc[b] = mfma_bf16(in ? *(const u32x4_t*)(p.w + (size_t)col[b] * p.ldw + k) : zero4(), x, acc[b]);
        }
    }
    const int mine = adapter_of(p, m);
    uint64_t left = __ballot(mine >= 0);
    while (left) {
        const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(left), 64));
        left &= ~__ballot(mine == a);
        const int rank = rank_of(p, a);
        const bool on = mine == a;
        f32x4_t d[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) d[b] = zerof();
        for (int k = 8 * q; k < (rank + 31) / 32 * 32; k += 32) {
            float v[8];
            const float4* vr = (const float4*)(p.v + (size_t)m * p.r + k);
            const float4 lo = on && k < rank ? vr[0] : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 hi = on && k < rank ? vr[1] : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + i < rank ? v[i] : 0.f;
            u32x4_t part[PARTS];
            split_v<PARTS>(v, part);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                u32x4_t w = k < rank ? *(const u32x4_t*)(p.b + ((size_t)a * p.N + col[b]) * p.r + k) : zero4();
                if (k + 8 > rank) w = keep_first(w, rank - k);
#pragma unroll
                for (int n = 0; n < PARTS; ++n) d[b] = mfma_bf16(w, part[n], d[b]);
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][i] = on ? acc[b][i] + d[b][i] : acc[b][i];
    }
    if (m >= p.M) return;
    const int c0 = n0 + 16 * q;
    const size_t at = (size_t)m * p.ldy + c0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 4 * b + i;
            if (c < p.N) {
                float s = acc[b][i];
                if (p.base) s += to_f32(((const BaseT*)p.base)[(size_t)m * p.ldb + c]);
                ((OutT*)p.y)[at + 4 * b + i] = from_f32<OutT>(s);
            }
        }
}

template <int NM, int NR>
void launch_shrink(const LoraArgs& p, int turns, hipStream_t st) {
    const dim3 grid((unsigned)((p.M + 16 * NM - 1) / (16 * NM)), (unsigned)((p.r + 16 * NR - 1) / (16 * NR)), (unsigned)turns);
    lora_shrink_kernel<NM, NR><<<grid, 64 * kShrinkWaves, 0, st>>>(p);
}

}  // namespace

moe_status lora_shrink(const LoraArgs& p, hipStream_t st) {
    ProfScope ps("lora_shrink", st);
    if (p.M <= 64) launch_shrink<1, 1>(p, std::min(p.M, 16), st);
    else if (p.r <= 16) launch_shrink<2, 1>(p, 1, st);
    else if (p.r <= 32) launch_shrink<2, 2>(p, 1, st);
    else if (p.r <= 64) launch_shrink<2, 4>(p, 1, st);
    else launch_shrink<2, 8>(p, 1, st);
    return check_launch("lora_shrink");
}

moe_status lora_rows(const LoraArgs& p, moe_dtype base, moe_dtype out, hipStream_t st) {
    const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)((p.M + 63) / 64));
    ProfScope ps("lora_rows", st);
    if (out == MOE_BF16) {
        if (base == MOE_BF16) lora_rows_kernel<uint16_t, uint16_t, 2><<<grid, 256, 0, st>>>(p);
        else lora_rows_kernel<uint16_t, float, 2><<<grid, 256, 0, st>>>(p);
    } else {
        if (base == MOE_BF16) lora_rows_kernel<float, uint16_t, 3><<<grid, 256, 0, st>>>(p);
        else lora_rows_kernel<float, float, 3><<<grid, 256, 0, st>>>(p);
    }
    return check_launch("lora_rows");
}

}  // namespace moe
