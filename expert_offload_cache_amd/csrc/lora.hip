// moe_lora_linear: a projection with a low-rank adapter for each row.
//
//   y[m,:] = x[m,:] W^T + base[m,:] + scale_a (x[m,:] A_a^T) B_a^T,   a = adapter[m]
//
// Launch 1: v[m,:] = scale_a A_a x[m,:] for the rows that have an adapter, in binary32 (for few rows also the sums of
// x W^T over runs of the inputs).  Launch 2: the projection, with the adapters' second product at its end.
//
// v is binary32 and the matrix instructions take bf16, so v enters as the sum of kParts = 3 bf16 parts: v1 = bf16(v),
// v2 = bf16(v - v1), v3 = bf16(v - v1 - v2), 24 bits together.  Two parts hold 16, which is beyond what a bf16 result
// shows unless the adapters' sum and the rest nearly cancel; then a result from 65 rows on would be worse than one up
// to 64, where v stays as it is.  The third part takes 1 us of 88 (8192 rows of adapters alone, 4096 wide, rank 64) and
// 0.4 of 27.5 (1000 x 1001 x 2000, rank 24).
//
// Rows of several adapters share a tile: each adapter's product is formed for the whole tile and taken over
// for its own rows only, by selection, so that an adapter with infinities or NaN touches no other
// request's rows.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

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

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* gbl_ptr_t;
__device__ __align__(16) const uint8_t g_no_inputs[16] = {};

// lane l's 16 bytes at `from` to 16 l bytes past `to` in LDS
__device__ __forceinline__ void load_to_lds(const void* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((gbl_ptr_t)from, (lds_ptr_t)to, 16, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_and_meet() {  // at most N of this wave's loads in flight, its LDS reads done; then the others
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// for every adapter of the rows' list (LDS, `rows` of them, -1: none), in order of appearance; uniform over the workgroup
template <typename Body>
__device__ __forceinline__ void for_adapters(const int* list, int rows, int lane, Body&& body) {
    for (int t0 = 0; t0 < rows; t0 += 64) {
        int who = lane < rows - t0 ? list[t0 + lane] : -1;
        for (int i = 0; i < t0; ++i)
            if (list[i] == who) who = -1;
        uint64_t left = __ballot(who >= 0);
        while (left) {
            const int a = __builtin_amdgcn_readfirstlane(__shfl(who, __builtin_ctzll(left), 64));
            left &= ~__ballot(who == a);
            body(a);
        }
    }
}

// acc[j][i] += the products of 16 rows, block j of NA, with 16 rows of x, block i of NX, over the inputs of the steps
// s0 .. s1 - 1 of 32.  The rows' loads run C steps ahead, those of x (which many workgroups read, from L2) G.
// row(j), xrow(i): this lane's row of a block, nullptr a row of zeros.
template <int NX, int NA, int C, int G, typename Row, typename XRow>
__device__ __forceinline__ void stream_steps(int s0, int s1, int K, int q, Row&& row, XRow&& xrow, f32x4_t (&acc)[NA][NX]) {
    static_assert(C % G == 0, "rings");
    if (s0 >= s1) return;
    const uint16_t *ar[NA], *xr[NX];
    int xm[NX];  // 0: no row, the zeros again and again
#pragma unroll
    for (int i = 0; i < NA; ++i) ar[i] = row(i);
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        xr[i] = xrow(i);
        xm[i] = xr[i] ? -1 : 0;
        xr[i] = xr[i] ? xr[i] : (const uint16_t*)g_no_inputs;
    }
    u32x4_t a[C][NA], x[G][NX];
    // a step past the last repeats it, inputs past the last one repeat its chunk: neither is multiplied
    auto at = [&](int s) __attribute__((always_inline)) { return min(min(s, s1 - 1) * 32 + 8 * q, K - 8); };
    auto load_a = [&](int s, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NA; ++i) a[c][i] = *(const u32x4_t*)(ar[i] + at(s));
    };
    auto load_x = [&](int s, int g) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NX; ++i) x[g][i] = *(const u32x4_t*)(xr[i] + (at(s) & xm[i]));
    };
    auto multiply = [&](int s, int c) __attribute__((always_inline)) {
        const bool in = s * 32 + 8 * q < K;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const u32x4_t v = in ? x[c % G][i] : zero4();
#pragma unroll
            for (int j = 0; j < NA; ++j) acc[j][i] = mfma_bf16(in ? a[c][j] : zero4(), v, acc[j][i]);
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) load_a(s0 + c, c);
#pragma unroll
    for (int c = 0; c < G; ++c) load_x(s0 + c, c);
    int s = s0;
    for (; s + C < s1; s += C)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            multiply(s + c, c);
            load_a(s + c + C, c);
            load_x(s + c + G, c % G);
        }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (s + c < s1) multiply(s + c, c);
        if (c + G < C) load_x(s + c + G, c % G);
    }
}

// ---- launch 1 ---------------------------------------------------------------------------------------
// A workgroup takes 16 * NM rows and NR blocks of 16 ranks; its NW waves split the inputs, each with the loads of C
// steps on their way.  So x is read once for every 16 NR ranks and A once for every 16 NM rows: 8192 rows of 4096, rank 32, 33
// us, rank 64, which reads x twice, 47.  A workgroup takes 512 KB there, 10 us at the most that a compute unit takes from its L2
// (55 B/ns), and x alone 14 us from memory: with 16 steps a wave and 4 on their way it is latency that counts.
// Of its rows' adapters a workgroup takes every Z-th.
// red: NW * NM * NR KB of LDS.
template <int NM, int NR, int NW, int C>
__device__ __forceinline__ void shrink_tile(const LoraArgs& p, int m0, int r0, int z, int Z, float* red) {
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    // every wave: lane i holds row i's adapter (NM <= 4)
    const int mine = lane < 16 * NM ? adapter_of(p, m0 + lane) : -1;
    uint64_t left = __ballot(mine >= 0);
    int turn = 0;
    const int nst = (p.K + 31) / 32, s0 = wv * nst / NW, s1 = (wv + 1) * nst / NW;
    while (left) {
        const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(left), 64));
        const uint64_t rows = __ballot(mine == a);
        left &= ~rows;
        if (turn++ % Z != z) continue;
        const int rank = rank_of(p, a);
        if (r0 >= rank) continue;
        const float scale = p.scale[a];
        f32x4_t acc[NR][NM];
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int i = 0; i < NM; ++i) acc[j][i] = zerof();
        stream_steps<NM, NR, C, C>(s0, s1, p.K, q,
            [&](int j) __attribute__((always_inline)) { return p.a + ((size_t)a * p.r + min(r0 + 16 * j + r16, p.r - 1)) * p.K; },
            [&](int i) __attribute__((always_inline)) {  // (other adapters' rows would be read for nothing)
                const int m = 16 * i + r16;
                return (rows >> m) & 1 ? p.x + (size_t)(m0 + m) * p.ldx : (const uint16_t*)nullptr;
            }, acc);
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) *(f32x4_t*)&red[((wv * NM + i) * 16 + r16) * NR * 16 + j * 16 + 4 * q] = acc[j][i];
        __syncthreads();
        for (int o = tid; o < NM * NR * 256; o += 64 * NW) {
            const int m = o / (NR * 16), c = r0 + o % (NR * 16);
            float s = red[o];
#pragma unroll
            for (int w = 1; w < NW; ++w) s += red[w * NM * NR * 256 + o];
            if (((rows >> m) & 1) && c < rank) p.v[(size_t)(m0 + m) * p.r + c] = scale * s;
        }
        if (left) __syncthreads();
    }
}

template <int NM, int NR, int NW, int C>
__global__ __launch_bounds__(64 * NW, 4) void lora_shrink_kernel(LoraArgs p) {
    __shared__ float red[NW * NM * NR * 256];
    // the first adapters' workgroups start last: beside those few that take a tile's second, not before them
    shrink_tile<NM, NR, NW, C>(p, blockIdx.x * 16 * NM, blockIdx.y * 16 * NR, gridDim.z - 1 - blockIdx.z, gridDim.z, red);
}

// A few rows and a narrow matrix: x W^T needs nothing of v, so one launch forms both.  After the workgroups of the form above
// come those of the product, 16 columns and a run of inputs each (`splits` of them, so that every compute unit
// has work); launch 2 adds their sums up.
constexpr int kBothWaves = 8;

template <int MB>
__global__ __launch_bounds__(64 * kBothWaves, 4) void lora_both_kernel(LoraArgs p, int rank_blocks, int Z) {
    constexpr int NW = kBothWaves;
    __shared__ float red[NW * MB * 256];
    const int tiles = (p.M + 15) / 16, shrink = tiles * rank_blocks * Z;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int id = blockIdx.x;
    if (id < shrink) {
        shrink_tile<1, 1, NW, 8>(p, id % tiles * 16, id / tiles % rank_blocks * 16, id / (tiles * rank_blocks), Z, red);
        return;
    }
    id -= shrink;
    const int cols = (p.N + 15) / 16, n0 = id % cols * 16, split = id / cols, nst = (p.K + 31) / 32;
    const int s0 = (int)((int64_t)split * nst / p.splits), n = (int)((int64_t)(split + 1) * nst / p.splits) - s0;
    f32x4_t acc[1][MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[0][i] = zerof();
    stream_steps<MB, 1, 8, MB <= 3 ? 4 : 2>(s0 + wv * n / NW, s0 + (wv + 1) * n / NW, p.K, q,
        [&](int) __attribute__((always_inline)) { return p.w + (size_t)min(n0 + r16, p.N - 1) * p.ldw; },
        [&](int i) __attribute__((always_inline)) { return p.x + (size_t)min(16 * i + r16, p.M - 1) * p.ldx; }, acc);
#pragma unroll
    for (int i = 0; i < MB; ++i) *(f32x4_t*)&red[(wv * MB + i) * 256 + r16 * 16 + 4 * q] = acc[0][i];
    __syncthreads();
    for (int o = tid; o < p.M * 16; o += 64 * NW) {
        if (n0 + (o & 15) >= p.N) continue;
        float s = red[o];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w * MB * 256 + o];
        p.part[((size_t)split * p.M + (o >> 4)) * p.N + n0 + (o & 15)] = s;
    }
}

// ---- launch 2 ---------------------------------------------------------------------------------------
// 8 values of v from input k on, those beyond the rank zero
__device__ __forceinline__ void load_v(const LoraArgs& p, int m, int k, int rank, float (&v)[8]) {
    const float4* from = (const float4*)(p.v + (size_t)m * p.r + k);
    const float4 lo = from[0], hi = from[1];
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < rank ? v[e] : 0.f;
}

// 8 values of v as bf16 parts
constexpr int kParts = 3;
__device__ __forceinline__ void split_v(const float (&v)[8], u32x4_t (&part)[kParts]) {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
    for (int n = 0; n < kParts; ++n)
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

// 16 neighbouring columns of a row: base is asked for at once, added at the store
template <typename OutT, typename BaseT>
struct Columns {
    const LoraArgs& p;
    const int m, c0;
    const bool whole;
    u32x4_t base[sizeof(BaseT)];
    __device__ __forceinline__ Columns(const LoraArgs& p, int m, int c0)
        : p(p), m(m), c0(c0), whole(p.wide && m < p.M && c0 + 16 <= p.N) {
        if (!p.base) return;
        const u32x4_t* from = (const u32x4_t*)((const BaseT*)p.base + (size_t)m * p.ldb + c0);
#pragma unroll
        for (int e = 0; e < (int)sizeof(BaseT); ++e) base[e] = whole ? from[e] : zero4();
    }
    __device__ __forceinline__ void store(float (&s)[16]) const {
        OutT* y = (OutT*)p.y + (size_t)m * p.ldy + c0;
        if (whole) {
            if (p.base)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if constexpr (sizeof(BaseT) == 4) s[e] += as_f32(base[e / 4][e % 4]);
                    else s[e] += e & 1 ? bf16_hi(base[e / 8][e % 8 / 2]) : bf16_lo(base[e / 8][e % 8 / 2]);
                }
            if constexpr (sizeof(OutT) == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ((float4*)y)[e] = make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    ((u32x4_t*)y)[e] = u32x4_t{bf16_pair(s[8 * e], s[8 * e + 1]), bf16_pair(s[8 * e + 2], s[8 * e + 3]),
                                               bf16_pair(s[8 * e + 4], s[8 * e + 5]), bf16_pair(s[8 * e + 6], s[8 * e + 7])};
            }
        } else if (m < p.M) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c0 + e < p.N) {
                    const float b = p.base ? to_f32(((const BaseT*)p.base)[(size_t)m * p.ldb + c0 + e]) : 0.f;
                    y[e] = from_f32<OutT>(s[e] + b);
                }
        }
    }
};

// ---- launch 2, few rows: the matrix streamed once -------------------------------------------------------
// A workgroup takes 16 columns and all rows (16 MB of them).  8 of its 16 waves split the inputs of x W^T, the loads of
// 8 steps of W on their way; meanwhile the other 8 (all 16 without W) form the adapters' second product on
// the vector units, a row at a time: 16 columns x r inputs, a wave reads them as they lie, and v stays binary32.
// ALONE: one row whose v is formed here too, by every workgroup for itself (A is small and in L2: one launch less), by the
// other 8 waves; NA blocks of 16 ranks.
constexpr int kStreamWaves = 16;
// Up to 64 rows (4 operand blocks, an element a thread at the end): 64 rows of 2048 x 4096, rank 64, take 25.5 us, in tiles
// 94; of 4096 x 2048, rank 16, 20.6 and 72.  So there is a step at 65 rows: nothing cuts the inputs of a 64 x 64 tile.
constexpr int kStreamRows = 64;

template <typename OutT, typename BaseT, int MB, int NA>
__global__ __launch_bounds__(64 * kStreamWaves) void lora_stream_kernel(LoraArgs p) {
    constexpr bool kAlone = NA > 0;
    constexpr int H = kStreamWaves / 2;
    __shared__ float red[H][MB * 256];
    __shared__ float delta[MB * 256];
    __shared__ __align__(16) float vs[kAlone ? H + 1 : 1][kAlone ? NA * 16 : 1];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16, nst = (p.K + 31) / 32;
    const int only = kAlone ? __builtin_amdgcn_readfirstlane(adapter_of(p, 0)) : -1;
    auto x_row = [&](int i) __attribute__((always_inline)) { return p.x + (size_t)min(16 * i + r16, p.M - 1) * p.ldx; };
    const bool product = p.w && !p.splits;
    // (a thread has one element of the result at most)
    const int row = tid >> 4, col = n0 + (tid & 15);
    const bool mine = row < p.M && col < p.N;
    float sum0 = 0.f, base = 0.f;
    if (mine) {
        for (int i = 0; i < p.splits; ++i) sum0 += p.part[((size_t)i * p.M + row) * p.N + col];
        if (p.base) base = to_f32(((const BaseT*)p.base)[(size_t)row * p.ldb + col]);
    }
    if (wv < H && product) {
        f32x4_t acc[1][MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[0][i] = zerof();
        stream_steps<MB, 1, 8, MB <= 2 ? 8 : MB == 3 ? 4 : 2>(wv * nst / H, (wv + 1) * nst / H, p.K, q,
            [&](int) __attribute__((always_inline)) { return p.w + (size_t)min(n0 + r16, p.N - 1) * p.ldw; }, x_row, acc);
#pragma unroll
        for (int i = 0; i < MB; ++i) *(f32x4_t*)&red[wv][i * 256 + r16 * 16 + 4 * q] = acc[0][i];
    }
    if constexpr (kAlone) {
        if (wv >= H && only >= 0) {
            f32x4_t acc[NA][1];
#pragma unroll
            for (int i = 0; i < NA; ++i) acc[i][0] = zerof();
            stream_steps<1, NA, 8, 8>((wv - H) * nst / H, (wv - H + 1) * nst / H, p.K, q,
                [&](int i) __attribute__((always_inline)) { return p.a + ((size_t)only * p.r + min(16 * i + r16, p.r - 1)) * p.K; }, x_row, acc);
            if (r16 == 0)
#pragma unroll
                for (int i = 0; i < NA; ++i) *(f32x4_t*)&vs[wv - H][i * 16 + 4 * q] = acc[i][0];
        }
        __syncthreads();
        if (tid < NA * 16 && only >= 0) {
            float s = vs[0][tid];
#pragma unroll
            for (int w = 1; w < H; ++w) s += vs[w][tid];
            vs[H][tid] = p.scale[only] * s;
        }
        __syncthreads();
    }
    // rows first, first + step, ...: lane l takes column l / 4 and inputs 8 (l % 4) .. + 7 of each 32
    constexpr int F = MB >= 3 ? 4 : MB;  // rows whose operands are read together
    const int first = product && !kAlone ? wv - H : wv, step = product && !kAlone ? H : kStreamWaves;
    const int n = min(n0 + (lane >> 2), p.N - 1);
    for (int m0 = first; m0 >= 0 && m0 < p.M; m0 += step * F) {
        int ad[F], rank[F];
        float sum[F];
#pragma unroll
        for (int f = 0; f < F; ++f) ad[f] = adapter_of(p, m0 + f * step);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            ad[f] = __builtin_amdgcn_readfirstlane(ad[f]);
            rank[f] = ad[f] >= 0 ? rank_of(p, ad[f]) : 0;
            sum[f] = 0.f;
        }
        int most = 0;
#pragma unroll
        for (int f = 0; f < F; ++f) most = max(most, rank[f]);
        for (int k = 8 * (lane & 3); k < (most + 31) / 32 * 32; k += 32) {
            u32x4_t b[F];
            float4 lo[F], hi[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const bool in = k < rank[f];
                const int m = m0 + f * step;
                b[f] = in ? *(const u32x4_t*)(p.b + ((size_t)ad[f] * p.N + n) * p.r + k) : zero4();
                const float4* v = kAlone ? (const float4*)&vs[kAlone ? H : 0][kAlone ? k : 0] : (const float4*)(p.v + (size_t)m * p.r + k);
                lo[f] = in ? v[0] : make_float4(0.f, 0.f, 0.f, 0.f);
                hi[f] = in ? v[1] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const float v[8] = {lo[f].x, lo[f].y, lo[f].z, lo[f].w, hi[f].x, hi[f].y, hi[f].z, hi[f].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // (places beyond the rank hold anything)
                    sum[f] = k + 2 * i < rank[f] ? __builtin_fmaf(v[2 * i], bf16_lo(b[f][i]), sum[f]) : sum[f];
                    sum[f] = k + 2 * i + 1 < rank[f] ? __builtin_fmaf(v[2 * i + 1], bf16_hi(b[f][i]), sum[f]) : sum[f];
                }
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int m = m0 + f * step;
            const float t = pair_sum2(pair_sum1(sum[f]));
            if (m < p.M && (lane & 3) == 0) delta[m * 16 + (lane >> 2)] = t;
        }
    }
    __syncthreads();
    if (mine) {
        if (product) {
            sum0 = red[0][tid];
#pragma unroll
            for (int w = 1; w < H; ++w) sum0 += red[w][tid];
        }
        ((OutT*)p.y)[(size_t)row * p.ldy + col] = from_f32<OutT>(sum0 + base + delta[tid]);
    }
}

// ---- launch 2, many rows and no matrix -------------------------------------------------------------------
// A workgroup takes 64 rows and 512 columns, its 4 waves 64 columns at a time.  The rows' v lies in LDS as bf16 parts, 64
// ranks at a time (row's chunk c at c ^ row % 8); B and base come straight to registers.  Columns in the order
// of the tiles below, so that a lane holds 16 neighbouring ones.
// 8192 rows of 4096, rank 64: 46 us, 134 MB of base and y at 2.9 TB/s.
constexpr int kAddCols = 512;

template <typename OutT, typename BaseT>
__global__ __launch_bounds__(256) void lora_add_kernel(LoraArgs p) {
    __shared__ __align__(16) uint8_t parts[kParts * 64 * 128];
    __shared__ int s_adapter[64], s_rank[64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.y * 64;
    if (tid < 64) {
        const int a = adapter_of(p, m0 + tid);
        s_adapter[tid] = a;
        s_rank[tid] = a >= 0 ? rank_of(p, a) : 0;
    }
    __syncthreads();
    auto stage = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = tid; i < 64 * 8; i += 256) {
            const int row = i >> 3, c = i & 7, k = k0 + 8 * c;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (k < s_rank[row]) load_v(p, m0 + row, k, s_rank[row], v);
            u32x4_t part[kParts];
            split_v(v, part);
#pragma unroll
            for (int n = 0; n < kParts; ++n) *(u32x4_t*)(parts + (n * 64 + row) * 128 + ((c ^ (row & 7)) << 4)) = part[n];
        }
        __syncthreads();
    };
    int mine[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[j] = s_adapter[16 * j + r16];
    stage(0);
    for (int g = wv; g < kAddCols / 64; g += 4) {
        const int n0 = blockIdx.x * kAddCols + 64 * g;  // (past the end: nothing is stored)
        const Columns<OutT, BaseT> out[4] = {{p, m0 + r16, n0 + 16 * q}, {p, m0 + 16 + r16, n0 + 16 * q},
                                             {p, m0 + 32 + r16, n0 + 16 * q}, {p, m0 + 48 + r16, n0 + 16 * q}};
        f32x4_t acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = zerof();
        for (int k0 = 0; k0 < p.r; k0 += 64) {
            if (p.r > 64) {
                __syncthreads();
                stage(k0);
            }
            for_adapters(s_adapter, 64, lane, [&](int a) __attribute__((always_inline)) {
                const int rank = p.rank ? rank_of(p, a) : p.r;
                if (k0 >= rank) return;
                u32x4_t b[4][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = k0 + 32 * h + 8 * q;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = min(n0 + 16 * (r16 >> 2) + 4 * i + (r16 & 3), p.N - 1);
                        b[i][h] = *(const u32x4_t*)(p.b + ((size_t)a * p.N + n) * p.r + min(k, p.r - 8));
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i][h] = keep_first(b[i][h], rank - (k0 + 32 * h + 8 * q));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool on = mine[j] == a;
                    if (!__ballot(on)) continue;
                    f32x4_t d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = zerof();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (k0 + 32 * h >= rank) break;
#pragma unroll
                        for (int n = 0; n < kParts; ++n) {
                            const u32x4_t v = *(const u32x4_t*)(parts + (n * 64 + 16 * j + r16) * 128 + (((4 * h + q) ^ (r16 & 7)) << 4));
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[i] = mfma_bf16(b[i][h], v, d[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][i][e] = on ? acc[j][i][e] + d[i][e] : acc[j][i][e];
                }
            });
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = acc[j][e / 4][e % 4];
            out[j].store(s);
        }
    }
}

// ---- launch 2, many rows: tiles ---------------------------------------------------------------------------
// A workgroup computes BN columns x BM rows; its WN x WM waves take equal parts.  Inputs advance 64 at a time
// through a ring of R steps in LDS filled by direct-to-LDS loads: one barrier a step, after which the slot that the step
// before has left is filled for step + R - 1.  A row's eight 16-byte chunks of a step lie on 128 bytes, chunk c at
// position c ^ turn(row), so that no operand read meets a bank twice.
// Operand row i of a wave's column block 4 g + b is column 64 g + 16 (i / 4) + 4 b + i % 4, so that a lane's results are
// 16 neighbouring columns of a row, and four lanes' whole lines.
// 8192 x 4096 x 4096: 255 us (1.08 PFLOP/s), the LDS reads take as long as the products; 1000 x 1001 x 2000: 21 us, latency.
// The adapters come last: each adapter of the tile's rows, 64 ranks at a time, with B and the parts of v in LDS in the
// same layout, multiplied 32 ranks at a time: the registers hold one step's parts beside the tile's sums (both steps'
// spill at 256 x 256: 308 us a call of 8192 x 4096 x 4096, rank 32, against 288).
__device__ __forceinline__ int turn_n(int row) { return ((row >> 1) & 1) | ((row >> 4) & 3) << 1; }
__device__ __forceinline__ int turn_m(int row) { return (row >> 1) & 7; }

template <typename OutT, typename BaseT, int BN, int BM, int WN, int WM, int R>
__global__ __launch_bounds__(64 * WN * WM, 2) void lora_tile_kernel(LoraArgs p) {
    constexpr int NW = WN * WM, RA = BN / WN / 16, CB = BM / WM / 16;
    constexpr int kStep = (BN + BM) * 128, kLoads = kStep / 1024 / NW;  // bytes of a step; a wave's 1 KB loads
    static_assert(RA % 4 == 0 && kLoads * NW * 1024 == kStep, "tile shape");
    static_assert(BN * 128 + kParts * BM * 128 <= R * kStep, "B and the parts of v fit the ring");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_adapter[BM];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wv % WN, wm = wv / WN;
    // consecutive workgroups go to the XCDs in turn: each XCD takes a run of tiles, neighbours in n first
    const int gx = (p.N + BN - 1) / BN, total = gx * ((p.M + BM - 1) / BM);
    const int per = (total + 7) / 8, tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= total || (int)(blockIdx.x >> 3) >= per) return;
    const int n0 = tile % gx * BN, m0 = tile / gx * BM;
    for (int i = tid; i < BM; i += 64 * NW) s_adapter[i] = adapter_of(p, m0 + i);

    f32x4_t acc[RA][CB];
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[i][j] = zerof();
    // LDS byte of chunk q of a lane's operand row; chunk 4 + q is at ^ 64
    int at_n[4], at_m[CB];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int row = 16 * (r16 >> 2) + 4 * b + (r16 & 3);  // of a wave's first 64 columns
        at_n[b] = (wn * RA * 16 + row) * 128 + ((q ^ turn_n(row)) << 4);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
        const int row = (wm * CB + j) * 16 + r16;
        at_m[j] = (BN + row) * 128 + ((q ^ turn_m(row)) << 4);
    }
    // the products of what lies in `buf` over 32 of its inputs (half h) added to acc
    auto multiply = [&](const uint8_t* buf, int h) __attribute__((always_inline)) {
        u32x4_t b[CB];
#pragma unroll
        for (int j = 0; j < CB; ++j) b[j] = *(const u32x4_t*)(buf + (at_m[j] ^ (64 * h)));
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const u32x4_t a = *(const u32x4_t*)(buf + (i / 4) * 64 * 128 + (at_n[i % 4] ^ (64 * h)));
#pragma unroll
            for (int j = 0; j < CB; ++j) acc[i][j] = mfma_bf16(a, b[j], acc[i][j]);
        }
    };
    if (p.w) {
        const int nst = (p.K + 63) / 64;
        const uint16_t* src[kLoads];
        int first[kLoads];  // this lane's first input of a step
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int row = (wv * kLoads + u) * 8 + (lane >> 3);  // of the step's BN + BM
            const bool is_n = row < BN;
            const int r = is_n ? row : row - BN, c = (lane & 7) ^ (is_n ? turn_n(r) : turn_m(r));
            first[u] = 8 * c;
            src[u] = (is_n ? p.w + (size_t)min(n0 + r, p.N - 1) * p.ldw : p.x + (size_t)min(m0 + r, p.M - 1) * p.ldx) + 8 * c;
        }
        auto issue = [&](int ks, int slot) __attribute__((always_inline)) {
            const int st = min(ks, nst - 1);  // past the end: the last step again, into a slot nobody reads
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const void* from = st * 64 + first[u] < p.K ? (const void*)(src[u] + (size_t)st * 64) : (const void*)g_no_inputs;
                load_to_lds(from, smem + slot * kStep + (wv * kLoads + u) * 1024);
            }
        };
#pragma unroll
        for (int s = 0; s < R - 1; ++s) issue(s, s);
        int slot = 0;
        for (int ks = 0; ks < nst; ++ks) {
            wait_and_meet<(R - 2) * kLoads>();  // step ks is there, and every wave has left step ks - 1
            issue(ks + R - 1, slot == 0 ? R - 1 : slot - 1);
            const uint8_t* buf = smem + slot * kStep;
            multiply(buf, 0);
            multiply(buf, 1);
            slot = slot + 1 < R ? slot + 1 : 0;
        }
    }
    wait_and_meet<0>();  // the ring is free, s_adapter is written
    int mine[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) mine[j] = s_adapter[(wm * CB + j) * 16 + r16];
    for_adapters(s_adapter, BM, lane, [&](int a) __attribute__((always_inline)) {
            const int rank = rank_of(p, a);
            for (int k0 = 0; k0 < rank; k0 += 64) {
                const int halves = rank - k0 > 32 ? 2 : 1;
                // B [BN, 64] and the parts of v [BM, 64]; places beyond the rank, and other adapters' rows, zero
                for (int i = tid; i < BN * 8; i += 64 * NW) {
                    const int row = i >> 3, c = i & 7, k = k0 + 8 * c;
                    u32x4_t w = k < rank ? *(const u32x4_t*)(p.b + ((size_t)a * p.N + min(n0 + row, p.N - 1)) * p.r + k) : zero4();
                    if (k + 8 > rank) w = keep_first(w, rank - k);
                    *(u32x4_t*)(smem + row * 128 + ((c ^ turn_n(row)) << 4)) = w;
                }
                for (int i = tid; i < BM * 8; i += 64 * NW) {
                    const int row = i >> 3, c = i & 7, k = k0 + 8 * c;
                    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (k < rank && s_adapter[row] == a) load_v(p, m0 + row, k, rank, v);
                    u32x4_t part[kParts];
                    split_v(v, part);
#pragma unroll
                    for (int n = 0; n < kParts; ++n)
                        *(u32x4_t*)(smem + (BN + n * BM + row) * 128 + ((c ^ turn_m(row)) << 4)) = part[n];
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    const bool on = mine[j] == a;
#pragma unroll 1
                    for (int h = 0; h < halves; ++h) {
                        u32x4_t b[kParts];
#pragma unroll
                        for (int n = 0; n < kParts; ++n) b[n] = *(const u32x4_t*)(smem + n * BM * 128 + (at_m[j] ^ (64 * h)));
#pragma unroll
                        for (int i = 0; i < RA; ++i) {
                            const u32x4_t w = *(const u32x4_t*)(smem + (i / 4) * 64 * 128 + (at_n[i % 4] ^ (64 * h)));
                            f32x4_t d = zerof();
#pragma unroll
                            for (int n = 0; n < kParts; ++n) d = mfma_bf16(w, b[n], d);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][e] = on ? acc[i][j][e] + d[e] : acc[i][j][e];
                        }
                    }
                }
                __syncthreads();
            }
    });
#pragma unroll
    for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int g = 0; g < RA / 4; ++g) {
            const Columns<OutT, BaseT> out(p, m0 + (wm * CB + j) * 16 + r16, n0 + (wn * RA + 4 * g) * 16 + 16 * q);
            float s[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = acc[4 * g + e / 4][j][e % 4];
            out.store(s);
        }
}

template <int NM, int NR, int NW, int C>
void launch_shrink(const LoraArgs& p, int z, hipStream_t st) {
    const dim3 grid((unsigned)((p.M + 16 * NM - 1) / (16 * NM)), (unsigned)((p.r + 16 * NR - 1) / (16 * NR)), (unsigned)z);
    lora_shrink_kernel<NM, NR, NW, C><<<grid, 64 * NW, 0, st>>>(p);
}

template <typename OutT, typename BaseT>
moe_status launch_stream(const LoraArgs& p, hipStream_t st) {
    const unsigned grid = (unsigned)((p.N + 15) / 16);
    ProfScope ps(lora_alone(p) ? "lora_alone" : "lora_stream", st);
    if (lora_alone(p)) {
        lora_stream_kernel<OutT, BaseT, 1, 1><<<grid, 64 * kStreamWaves, 0, st>>>(p);
    } else if (p.M <= 16) lora_stream_kernel<OutT, BaseT, 1, 0><<<grid, 64 * kStreamWaves, 0, st>>>(p);
    else if (p.M <= 32) lora_stream_kernel<OutT, BaseT, 2, 0><<<grid, 64 * kStreamWaves, 0, st>>>(p);
    else if (p.M <= 48) lora_stream_kernel<OutT, BaseT, 3, 0><<<grid, 64 * kStreamWaves, 0, st>>>(p);
    else lora_stream_kernel<OutT, BaseT, 4, 0><<<grid, 64 * kStreamWaves, 0, st>>>(p);
    return MOE_OK;
}

int64_t tiles_of(const LoraArgs& p, int bn, int bm) { return ((int64_t)p.N + bn - 1) / bn * ((p.M + bm - 1) / bm); }

template <typename OutT, typename BaseT, int BN, int BM, int WN, int WM, int R>
moe_status launch_tile(const LoraArgs& p, hipStream_t st) {
    constexpr int lds = R * (BN + BM) * 128;
    auto kern = lora_tile_kernel<OutT, BaseT, BN, BM, WN, WM, R>;
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    // columns x rows, steps of the ring: a profile tells the tiles apart
    static const std::string name = "lora_tile_" + std::to_string(BN) + "x" + std::to_string(BM) + "_" + std::to_string(R);
    ProfScope ps(name.c_str(), st);
    kern<<<(unsigned)((tiles_of(p, BN, BM) + 7) / 8 * 8), 64 * WN * WM, lds, st>>>(p);
    return MOE_OK;
}

template <typename OutT, typename BaseT>
moe_status launch_tiles(const LoraArgs& p, hipStream_t st) {
    if (!p.w) {
        ProfScope ps("lora_add", st);
        lora_add_kernel<OutT, BaseT><<<dim3((unsigned)((p.N + kAddCols - 1) / kAddCols), (unsigned)((p.M + 63) / 64)), 256, 0, st>>>(p);
        return MOE_OK;
    }
    // The largest tile that gives three quarters of the compute units one (us a call, outputs' columns x rows x inputs in
    // tiles of 256 x 256, 128 x 128, 64 x 64): 4096 x 8192 x 4096, rank 32, 287, 435, 766; 4096 x 2944 x 4096 (192 of 256 x
    // 256) 146, 173, 296; 4096 x 2048 x 4096 144, 130, 208; 2048 x 1536 x 4096 (192 of 128 x 128) 132, 69, 90; 1001 x 1000
    // x 2000 (64 of 128 x 128) 101, 51, 27.  Below 192 of 128 x 128 the border depends on the inputs' length: 176 of
    // them, 2048 x 1400 x 4096, 65 against 83 in 64 x 64.
    if (tiles_of(p, 256, 256) >= 192) return launch_tile<OutT, BaseT, 256, 256, 2, 4, 2>(p, st);
    if (tiles_of(p, 128, 128) >= 192) return launch_tile<OutT, BaseT, 128, 128, 2, 2, 3>(p, st);
    return launch_tile<OutT, BaseT, 64, 64, 1, 4, 6>(p, st);
}

template <typename OutT>
moe_status launch_rows(const LoraArgs& p, moe_dtype base, hipStream_t st) {
    if (p.M <= kStreamRows) return base == MOE_BF16 ? launch_stream<OutT, uint16_t>(p, st) : launch_stream<OutT, float>(p, st);
    return base == MOE_BF16 ? launch_tiles<OutT, uint16_t>(p, st) : launch_tiles<OutT, float>(p, st);
}

}  // namespace

// Where the sums fit their place, as many runs as give each of the 256 compute units a workgroup: 37 rows of 2048 x 4096,
// rank 64, 20 us against 26 with the product in launch 2.
int lora_splits(const LoraArgs& p) {
    if (!p.w || p.M > kStreamRows || lora_alone(p)) return 0;
    const int splits = std::min(std::max(256 / ((p.N + 15) / 16), 1), (p.K + 511) / 512);
    return (int)std::min<size_t>(splits, kLoraPartBytes / ((size_t)p.M * p.N * 4));
}

// One launch or two for one row (us, N x K, one against two):
//  - every workgroup of the one reads A for itself: rank 16, 4096 x 2048 9.6 against 11.5, 4096 x 4096 13.9 against 16.1; rank 32
//    11.9 against 11.7, 18.1 against 16.1; rank 64 28 against 12;
//  - so it has to be one workgroup a compute unit, 16 columns each: rank 16, 4096 x 2048 as above, 4112 x 2048 15.3 against 12.1,
//    8192 x 2048 17.3 against 15.1, without W 4096 x 4096 8.5 against 9.2, 4608 x 4096 15.2 against 10.1;
//  - a narrow W of long rows is better cut into runs of the inputs, which launch 1 of two does (lora_splits): rank 16,
//    K = 4 N 1024 x 4096 13.1 against 13.4, 6 N 1024 x 6144 17.9 against 15.5, 8 N 1024 x 8192 21.8 against 18.2; without W
//    1024 x 6144 10.4 against 11.4.
bool lora_alone(const LoraArgs& p) { return p.M == 1 && p.r <= 16 && p.N <= 4096 && (!p.w || p.K <= (int64_t)4 * p.N); }

moe_status lora_shrink(const LoraArgs& p, hipStream_t st) {
    if (lora_alone(p)) return MOE_OK;
    ProfScope ps(p.splits ? "lora_both" : "lora_shrink", st);
    const int blocks = (p.M + 15) / 16 * ((p.r + 15) / 16), few = std::min(std::min(p.M, 16), p.n);
    if (p.splits) {
        const unsigned grid = (unsigned)(blocks * few + (p.N + 15) / 16 * p.splits);
        if (p.M <= 16) lora_both_kernel<1><<<grid, 64 * kBothWaves, 0, st>>>(p, (p.r + 15) / 16, few);
        else if (p.M <= 32) lora_both_kernel<2><<<grid, 64 * kBothWaves, 0, st>>>(p, (p.r + 15) / 16, few);
        else if (p.M <= 48) lora_both_kernel<3><<<grid, 64 * kBothWaves, 0, st>>>(p, (p.r + 15) / 16, few);
        else lora_both_kernel<4><<<grid, 64 * kBothWaves, 0, st>>>(p, (p.r + 15) / 16, few);
    } else if (p.M <= kStreamRows) launch_shrink<1, 1, 16, 4>(p, few, st);
    // small tiles until they fill the compute units: 1000 x 2000, rank 24: 27 us the whole call, 30 with the large ones
    else if (blocks < 256) launch_shrink<1, 1, 16, 4>(p, std::min(p.n, 2), st);
    else launch_shrink<2, 2, 8, 4>(p, std::min(p.n, 2), st);
    return check_launch("lora_shrink");
}

moe_status lora_rows(const LoraArgs& p, moe_dtype base, moe_dtype out, hipStream_t st) {
    const moe_status e = out == MOE_BF16 ? launch_rows<uint16_t>(p, base, st) : launch_rows<float>(p, base, st);
    return e == MOE_OK ? check_launch("lora_rows") : e;
}

}  // namespace moe
