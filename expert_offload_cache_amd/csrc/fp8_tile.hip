// Products of 8-bit operands with many rows of activations (prefill): tiles on the matrix cores.
//
// A workgroup of NW waves computes MT = NW * RA * 16 weight rows x NT = 16 * NTB tokens; each wave owns RA
// blocks of 16 rows for all of the tile's tokens.  Inputs advance 128 at a time, one scale group: a
// step is one mfma_fp8 (fp8.h; mfma_fp8_exact where the caller wants binary32) per (row block, token
// block), whose sum is added to binary32 accumulators times the token's scale and the row block's.
//
// Each wave loads its own weight rows straight into registers, one step ahead (two register sets take
// turns); only the tokens go through LDS, in a ring of three stages filled by direct-to-LDS
// loads, two steps ahead, in the lane order in which every wave reads them back without conflicts.
// The scales of the whole tile are put into LDS once, before the first step.
//
// Gate/up: a wave's row blocks are gate and up blocks in turn, so SwiGLU happens in registers; the
// 16 / RA waves that share a 128-column group of h join their largest magnitudes through LDS, and h is
// written in 8 bits with its scale.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ffn_common.h"
#include "fp8_ops.h"
#include "slot_layout.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* gbl_ptr_t;

enum { kDense = 2 };  // beside kGateUp and kDown

__device__ __align__(16) const uint8_t g_zeros[16] = {};

__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* lds_wave_base) {
    // 16 bytes per lane; lane i's bytes land at lds_wave_base + 16 i whatever its source address
    __builtin_amdgcn_global_load_lds((gbl_ptr_t)src, (lds_ptr_t)lds_wave_base, 16, 0, 0);
}

// At most N of this wave's loads still in flight and its LDS reads done, then meet the other waves.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int RA, int NTB, int NW>
struct Tile8 {
    static constexpr int kMT = NW * RA * 16, kNT = NTB * 16;
    static constexpr int kStage = NTB * kFp8Frag;
    static constexpr int kUnits = 2 * NTB / NW;  // 1 KB halves of a token block each wave loads a step
    static constexpr int kRing = 3;
    static constexpr int kWScales = kMT >= 128 ? kMT / 128 : 1;  // weight scales a step
    static_assert(kUnits * NW == 2 * NTB, "token blocks must divide over the waves");
    // scales of step g: the tokens' at g * (kNT + 1), then (after G steps) the weights'
    static constexpr int lds(int G) { return kRing * kStage + 4 * G * (kNT + 1 + kWScales); }
    static_assert(kNT * NW * 4 <= kRing * kStage, "the magnitudes reuse the ring");
};

// What a wave's loop needs: lane l's weight bytes of row block i start at w + w_off[i] (second half w_half
// on, the next step w_step on); lane l's token bytes of its u-th unit at x[u] (the next step 128 on).
template <int RA, int UN>
struct Feed {
    const uint8_t* w;
    uint32_t w_off[RA];
    int w_step, w_half;
    const uint8_t* x[UN];
};

// acc = the tile's products over all steps.  MODE decides which scale a row block takes.
template <int MODE, int RA, int NTB, int NW, bool EXACT, bool TAIL>
__device__ __forceinline__ void tile_loop(const Feed<RA, Tile8<RA, NTB, NW>::kUnits>& fd, uint8_t* smem, int nst, int K,
                                          int wv, int lane, f32x4_t (&acc)[RA][NTB]) {
    using TL = Tile8<RA, NTB, NW>;
    constexpr int UN = TL::kUnits;
    const float* xs = (const float*)(smem + TL::kRing * TL::kStage);
    const float* ws = xs + (size_t)nst * (TL::kNT + 1);
    const int q = lane >> 4;
    auto issue_x = [&](int ks, int slot) __attribute__((always_inline)) {
        ks = min(ks, nst - 1);
        uint8_t* buf = smem + slot * TL::kStage;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint8_t* p = fd.x[u] + (size_t)ks * 128;
            if constexpr (TAIL) {
                const int h = (wv * UN + u) & 1;
                if (ks * 128 + 64 * h + 16 * q >= K) p = g_zeros;
            }
            load_to_lds(p, buf + (wv * UN + u) * 1024);
        }
    };
    auto load_w = [&](int ks, u32x4_t (&a)[RA][2]) __attribute__((always_inline)) {
        ks = min(ks, nst - 1);
        const uint8_t* base = fd.w + (size_t)ks * fd.w_step;
        const bool in0 = !TAIL || ks * 128 + 16 * q < K, in1 = !TAIL || ks * 128 + 64 + 16 * q < K;
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const uint8_t* p = base + fd.w_off[i];
            a[i][0] = *(const u32x4_t*)(in0 ? p : g_zeros);
            a[i][1] = *(const u32x4_t*)(in1 ? p + fd.w_half : g_zeros);
        }
    };
    // step ks in ring slot `slot`: its operands have landed; loads of step ks + 1 (weights) and ks + 2
    // (tokens, into the slot that step ks - 1 has left) go out first
    auto step = [&](int ks, int slot, const u32x4_t (&cur)[RA][2], u32x4_t (&nxt)[RA][2]) __attribute__((always_inline)) {
        stage_barrier<UN>();
        load_w(ks + 1, nxt);
        issue_x(ks + 2, slot >= 1 ? slot - 1 : TL::kRing - 1);
        const uint8_t* sb = smem + slot * TL::kStage + lane * 16;
        const float* xrow = xs + ks * (TL::kNT + 1) + (lane & 15);
        float s0, s1;  // this wave's weight scales: its rows' block, or its gate and its up block
        if constexpr (MODE == kGateUp) {
            s0 = ws[ks * TL::kWScales + 2 * (wv * RA / 16)];
            s1 = ws[ks * TL::kWScales + 2 * (wv * RA / 16) + 1];
        } else {
            s0 = s1 = ws[ks * TL::kWScales + wv * RA / 8];
        }
#pragma unroll
        for (int j = 0; j < NTB; ++j) {
            const i32x8_t b = join8(*(const u32x4_t*)(sb + (2 * j) * 1024), *(const u32x4_t*)(sb + (2 * j + 1) * 1024));
            const float sx = xrow[16 * j];
            const float f0 = sx * s0, f1 = MODE == kGateUp ? sx * s1 : f0;
#pragma unroll
            for (int i = 0; i < RA; ++i) {
                f32x4_t p;
                if constexpr (EXACT) p = mfma_fp8_exact(widen(join8(cur[i][0], cur[i][1])), widen(b));
                else p = mfma_fp8(join8(cur[i][0], cur[i][1]), b);
                const float f = (i & 1) ? f1 : f0;
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(p[c], f, acc[i][j][c]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < NTB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    u32x4_t a0[RA][2], a1[RA][2];
    issue_x(0, 0);
    load_w(0, a0);
    issue_x(1, 1);
    int ks = 0;
    for (; ks + 6 <= nst; ks += 6) {
        step(ks, 0, a0, a1);
        step(ks + 1, 1, a1, a0);
        step(ks + 2, 2, a0, a1);
        step(ks + 3, 0, a1, a0);
        step(ks + 4, 1, a0, a1);
        step(ks + 5, 2, a1, a0);
    }
    if (ks < nst) step(ks, 0, a0, a1);
    if (ks + 1 < nst) step(ks + 1, 1, a1, a0);
    if (ks + 2 < nst) step(ks + 2, 2, a0, a1);
    if (ks + 3 < nst) step(ks + 3, 0, a1, a0);
    if (ks + 4 < nst) step(ks + 4, 1, a0, a1);
    stage_barrier<0>();  // the tail's repeated loads have landed, every wave has left the ring
}

// ---- the dense product ------------------------------------------------------------------------------
template <int RA, int NTB, int NW, bool EXACT, bool TAIL>
__global__ __launch_bounds__(NW * 64, 2) void gemm_fp8_tile_kernel(GemmFp8 g) {
    using TL = Tile8<RA, NTB, NW>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * TL::kMT, m0 = blockIdx.y * TL::kNT;
    const int nrow = n0 + wv * RA * 16;  // this wave's first weight row
    Feed<RA, TL::kUnits> fd;
    fd.w = g.w + (size_t)n0 * g.ldw;
    fd.w_step = 128;
    fd.w_half = 64;
#pragma unroll
    for (int i = 0; i < RA; ++i)  // rows past the end repeat the last one and are not stored
        fd.w_off[i] = (uint32_t)(min(nrow + 16 * i + (lane & 15), g.N - 1) - n0) * (uint32_t)g.ldw + 16 * (lane >> 4);
#pragma unroll
    for (int u = 0; u < TL::kUnits; ++u) {
        const int unit = wv * TL::kUnits + u;
        const int m = min(m0 + 16 * (unit >> 1) + (lane & 15), g.M - 1);
        fd.x[u] = g.a + (size_t)m * g.lda + 64 * (unit & 1) + 16 * (lane >> 4);
    }
    float* xs = (float*)(smem + TL::kRing * TL::kStage);
    float* ws = xs + (size_t)g.G * (TL::kNT + 1);
    for (int i = threadIdx.x; i < g.G * TL::kNT; i += NW * 64) {
        const int t = i / g.G, k = i - t * g.G;
        xs[k * (TL::kNT + 1) + t] = g.a_scale[(size_t)min(m0 + t, g.M - 1) * g.G + k];
    }
    for (int i = threadIdx.x; i < g.G * TL::kWScales; i += NW * 64) {
        const int b = i / g.G, k = i - b * g.G;
        ws[k * TL::kWScales + b] = g.w_scale[(size_t)(min(n0 + 128 * b, g.N - 1) / 128) * g.G + k];
    }
    f32x4_t acc[RA][NTB];
    tile_loop<kDense, RA, NTB, NW, EXACT, TAIL>(fd, smem, g.G, g.K, wv, lane, acc);
#pragma unroll
    for (int j = 0; j < NTB; ++j) {
        const int m = m0 + 16 * j + (lane & 15);
        if (m >= g.M) continue;
#pragma unroll
        for (int i = 0; i < RA; ++i) store_c4(g, m, nrow + 16 * i + 4 * (lane >> 4), acc[i][j]);
    }
}

template <int RA, int NTB, int NW, bool EXACT>
moe_status launch_gemm(const GemmFp8& g, hipStream_t st) {
    using TL = Tile8<RA, NTB, NW>;
    const bool tail = g.K % 128 != 0;
    auto kern = tail ? gemm_fp8_tile_kernel<RA, NTB, NW, EXACT, true> : gemm_fp8_tile_kernel<RA, NTB, NW, EXACT, false>;
    const int lds = TL::lds(g.G);
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    const dim3 grid((unsigned)((g.N + TL::kMT - 1) / TL::kMT), (unsigned)((g.M + TL::kNT - 1) / TL::kNT));
    ProfScope p("gemm_fp8_tile", st);
    kern<<<grid, NW * 64, lds, st>>>(g);
    return check_launch("gemm_fp8_tile");
}

// ---- the routed experts' projections ------------------------------------------------------------------
template <int MODE, int RA, int NTB, int NW>
__global__ __launch_bounds__(NW * 64, 2) void ffn_fp8_tile_kernel(FfnFp8 p) {
    using TL = Tile8<RA, NTB, NW>;
    static_assert(MODE != kGateUp || (RA % 2 == 0 && TL::kMT % 256 == 0), "gate/up tiles hold whole groups of h");
    extern __shared__ __align__(16) uint8_t smem[];
    const FfnArgs& a = p.a;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = MODE == kGateUp ? a.d : a.f, G = K / 128;
    int e, chunk;
    if (!find_work(a.counts, a.E, a.T, TL::kNT, a.shared_w != nullptr, blockIdx.y, e, chunk, a.n_lo, a.n_hi)) return;
    const bool shared = e == -1;
    const int n_all = __builtin_amdgcn_readfirstlane(shared ? a.T : a.counts[e]);
    const int t0 = chunk * TL::kNT;
    const int nt = __builtin_amdgcn_readfirstlane(min(TL::kNT, n_all - t0));
    const int p0 = __builtin_amdgcn_readfirstlane(shared ? a.T * a.k : a.offsets[e]) + t0;  // first row of the tile
    const uint8_t* base;
    if (shared) {
        base = a.shared_w;
    } else {
        const int slot = __builtin_amdgcn_readfirstlane(a.slot_of_expert[e]);
        if (slot == MOE_SLOT_ELSEWHERE) return;  // rows produced elsewhere: leave them
        if (slot < 0 || slot >= a.n_slots) {     // absent: flagged, zero rows (h is not read then)
            if (threadIdx.x == 0) *a.status = 1;
            if (MODE == kDown)
                for (int i = threadIdx.x; i < nt * TL::kMT; i += NW * 64) {
                    const int c = blockIdx.x * TL::kMT + i % TL::kMT;
                    if (c < a.d) store_y(a, (size_t)(p0 + i / TL::kMT), c, 0.f);
                }
            return;
        }
        base = a.pool + (size_t)slot * a.stride;
    }
    // d and f are multiples of 128, a wave's rows of 64 at most: all of them exist, or none (then the
    // wave repeats the last block's loads and stores nothing)
    const int nblk = MODE == kGateUp ? 2 * (a.f / 16) : a.d / 16;
    const int b0 = (blockIdx.x * NW + wv) * RA;
    const size_t rbb = rowblock_bytes(K, MOE_FP8_B128);
    Feed<RA, TL::kUnits> fd;
    const int bw = blockIdx.x * NW * RA;
    fd.w = base + (MODE == kGateUp ? 0 : down_block_offset(0, a.d, a.f, MOE_FP8_B128)) + (size_t)bw * rbb;
    fd.w_step = kFp8Frag;
    fd.w_half = kFp8Frag / 2;
#pragma unroll
    for (int i = 0; i < RA; ++i) fd.w_off[i] = (uint32_t)(min(b0 + i, nblk - 1) - bw) * (uint32_t)rbb + lane * 16;
    // tokens past the tile's end repeat its first; their columns are not stored
    auto source = [&](int t) __attribute__((always_inline)) {
        const int row = p0 + (t < nt ? t : 0);
        if (MODE != kGateUp) return row;
        return shared ? row - a.T * a.k : a.perm[row] / a.k;
    };
    const uint8_t* x = MODE == kGateUp ? p.x8 : p.h8;
    const float* x_scale = MODE == kGateUp ? p.x_scale : p.h_scale;
#pragma unroll
    for (int u = 0; u < TL::kUnits; ++u) {
        const int unit = wv * TL::kUnits + u;
        fd.x[u] = x + (size_t)source(16 * (unit >> 1) + (lane & 15)) * K + 64 * (unit & 1) + 16 * (lane >> 4);
    }
    float* xs = (float*)(smem + TL::kRing * TL::kStage);
    float* ws = xs + (size_t)G * (TL::kNT + 1);
    for (int i = threadIdx.x; i < G * TL::kNT; i += NW * 64) {
        const int t = i / G, k = i - t * G;
        xs[k * (TL::kNT + 1) + t] = x_scale[(size_t)source(t) * G + k];
    }
    for (int i = threadIdx.x; i < G * TL::kWScales; i += NW * 64) {
        const int s = i / G, k = i - s * G;
        // gate/up: the gate and the up scale of each 128 columns of h (16 blocks); down: of 8 blocks
        const int b = min(bw + (MODE == kGateUp ? 16 * (s >> 1) + (s & 1) : 8 * s), nblk - 2 + (MODE == kGateUp ? (s & 1) : 1));
        const uint8_t* blk = base + (MODE == kGateUp ? 0 : down_block_offset(0, a.d, a.f, MOE_FP8_B128)) + (size_t)b * rbb;
        ws[k * TL::kWScales + s] = ((const float*)(blk + (size_t)16 * K))[k];
    }
    f32x4_t acc[RA][NTB];
    tile_loop<MODE, RA, NTB, NW, false, false>(fd, smem, G, K, wv, lane, acc);
    const int quad = lane >> 4;
    if constexpr (MODE == kGateUp) {
        constexpr int GW = 16 / RA;  // waves that share a 128-column group of h
        uint32_t* mags = (uint32_t*)smem;  // [wave][token]
#pragma unroll
        for (int j = 0; j < NTB; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < RA / 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float h = silu_mul(acc[2 * i][j][c], acc[2 * i + 1][j][c]);
                    acc[2 * i][j][c] = h;
                    m = umax(m, abs_bits(h));
                }
            m = quarter_max(m);
            if (quad == 0) mags[wv * TL::kNT + 16 * j + lane] = m;
        }
        __syncthreads();
        if (b0 >= nblk) return;
        const int col0 = b0 / 2 * 16;
#pragma unroll
        for (int j = 0; j < NTB; ++j) {
            const int t = 16 * j + (lane & 15);
            if (t >= nt) continue;
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < GW; ++w) m = umax(m, mags[(wv / GW * GW + w) * TL::kNT + t]);
            const float s = fp8_scale(m), r = 1.0f / s;
            const size_t row = (size_t)(p0 + t);
#pragma unroll
            for (int i = 0; i < RA / 2; ++i)
                *(uint32_t*)(p.h8 + row * a.f + col0 + 16 * i + 4 * quad) =
                    fp8_pack4(acc[2 * i][j][0], acc[2 * i][j][1], acc[2 * i][j][2], acc[2 * i][j][3], r);
            if (wv % GW == 0 && quad == 0) p.h_scale[row * (a.f / 128) + col0 / 128] = s;
        }
    } else {
        if (b0 >= nblk) return;
#pragma unroll
        for (int j = 0; j < NTB; ++j) {
            const int t = 16 * j + (lane & 15);
            if (t >= nt) continue;
#pragma unroll
            for (int i = 0; i < RA; ++i)
                store_y4(a, (size_t)(p0 + t), (b0 + i) * 16 + 4 * quad, acc[i][j][0], acc[i][j][1], acc[i][j][2],
                         acc[i][j][3]);
        }
    }
}

template <int MODE, int RA, int NTB, int NW>
moe_status launch_ffn(const FfnFp8& p, hipStream_t st, const char* name) {
    using TL = Tile8<RA, NTB, NW>;
    const int64_t items = work_items(p.a, TL::kNT);
    if (items > 65535) return set_error(MOE_ESHAPE, "%s: %lld token tiles exceed one launch", name, (long long)items);
    if (items <= 0) return MOE_OK;
    const int nblk = MODE == kGateUp ? 2 * (p.a.f / 16) : p.a.d / 16;
    auto kern = ffn_fp8_tile_kernel<MODE, RA, NTB, NW>;
    const int lds = TL::lds((MODE == kGateUp ? p.a.d : p.a.f) / 128);
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    ProfScope sc(name, st);
    kern<<<dim3((unsigned)((nblk + NW * RA - 1) / (NW * RA)), (unsigned)items), NW * 64, lds, st>>>(p);
    return check_launch(name);
}

}  // namespace

// MOE_EDTYPE where the tiles do not apply
moe_status gemm_fp8_tile(const GemmFp8& g, hipStream_t st) {
    if (g.G > 192 || g.ldw > (1u << 22) || g.M > 65535 * 32) return MOE_EDTYPE;  // scales fit LDS, offsets 32 bits
    // fewer tiles than half the compute units: the streaming kernel splits the work finer
    if ((int64_t)((g.N + 511) / 512) * ((g.M + 127) / 128) < 128) return MOE_EDTYPE;
    if (!g.c_bf16) return launch_gemm<2, 8, 8, true>(g, st);
    return launch_gemm<4, 8, 8, false>(g, st);
}

moe_status ffn_fp8_tile(const FfnFp8& p, int mode, hipStream_t st) {
    FfnFp8 heavy = p, light = p;
    heavy.a.n_lo = 33;
    light.a.n_hi = 32;
    if (mode == kGateUp) {
        moe_status r = launch_ffn<kGateUp, 4, 8, 8>(heavy, st, "ffn_fp8_gateup_tile");
        return r != MOE_OK ? r : launch_ffn<kGateUp, 2, 4, 8>(light, st, "ffn_fp8_gateup_tile_light");
    }
    moe_status r = launch_ffn<kDown, 4, 8, 8>(heavy, st, "ffn_fp8_down_tile");
    return r != MOE_OK ? r : launch_ffn<kDown, 2, 4, 8>(light, st, "ffn_fp8_down_tile_light");
}

}  // namespace moe
