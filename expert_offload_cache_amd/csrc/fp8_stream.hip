// Products of 8-bit operands with few rows of activations (decode): the weights are streamed once.
//
// A workgroup owns RB blocks of 16 weight rows and up to TB blocks of 16 tokens; its S waves split
// the inputs, wave w taking the 128-input steps w, w + S, w + 2 S, ...  A step is one matrix-core
// product per (row block, token block), mfma_fp8_exact (fp8.h), lane l holding 32 inputs of row
// l % 16 and of token l % 16.  Which 32 is free as long as both operands agree:
// here 16 (l / 16) .. + 15 of each 64-input half, so a wave's 16-byte loads cover 64 consecutive
// bytes of each row of a row-major matrix.  The step's sum is added to binary32 accumulators times
// the product of the token's and the row block's scale of that 128-input group.  The S partial sums
// are joined through LDS in wave order.
//
// Nothing is staged: a wave keeps D steps of operands in flight in registers (bound by the weights'
// bytes; the activations are small and come from the caches).  Activations that are not yet in 8 bits
// (bf16 x of a layer, the binary32 h between the projections) are quantised as they are loaded: the
// four lanes l, l ^ 16, l ^ 32, l ^ 48 hold the 128 inputs of a token's group between them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ffn_common.h"
#include "fp8_ops.h"
#include "slot_layout.h"

namespace moe {
namespace {

enum { kSrcFp8 = 0, kSrcBf16 = 1, kSrcF32 = 2 };  // the activations' type

template <int SRC>
struct SrcOf;
template <>
struct SrcOf<kSrcFp8> {
    static constexpr int kBytes = 1;
};
template <>
struct SrcOf<kSrcBf16> {
    static constexpr int kBytes = 2;
};
template <>
struct SrcOf<kSrcF32> {
    static constexpr int kBytes = 4;
};

__device__ __align__(16) const uint8_t g_zero16[16] = {};

// One step's operands of a wave.
template <int SRC, int RB, int TB>
struct Step {
    static constexpr int NX = 2 * SrcOf<SRC>::kBytes;  // 16-byte loads of a token's 32 inputs
    u32x4_t w[RB][2];
    float ws[RB];
    u32x4_t x[TB][NX];
    float xs[TB];
};

// 32 inputs of a token as the matrix core takes them, and the group's scale
template <int SRC>
__device__ __forceinline__ i32x8_t token_operand(const u32x4_t (&x)[2 * SrcOf<SRC>::kBytes], float& scale) {
    if constexpr (SRC == kSrcFp8) {
        return join8(x[0], x[1]);
    } else {
        float v[32];
#pragma unroll
        for (int i = 0; i < 2 * SrcOf<SRC>::kBytes; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (SRC == kSrcBf16) {
                    v[8 * i + 2 * j] = bf16_lo(x[i][j]);
                    v[8 * i + 2 * j + 1] = bf16_hi(x[i][j]);
                } else {
                    v[4 * i + j] = as_f32(x[i][j]);
                }
            }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = umax(m, abs_bits(v[i]));
        scale = fp8_scale(quarter_max(m));
        const float r = 1.0f / scale;
        i32x8_t o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (int)fp8_pack4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], r);
        return o;
    }
}

// Where a wave finds its operands: wp[i] is lane l's first 16 bytes of row block i (the second half
// `whalf` bytes on, the next step `wstep` bytes on), wsc[i] the block's scales by step; xp[j] the row of
// lane l's token of block j, xsc[j] its scales.
template <int RB, int TB>
struct Operands {
    const uint8_t* wp[RB];
    const float* wsc[RB];
    const uint8_t* xp[TB];
    const float* xsc[TB];
    int wstep, whalf;
};

template <int SRC, int RB, int TB, bool TAIL>
__device__ __forceinline__ void load_step(const Operands<RB, TB>& o, int ks, int K, Step<SRC, RB, TB>& st) {
    constexpr int EB = SrcOf<SRC>::kBytes;
    const int q = (threadIdx.x & 63) >> 4;
    // TAIL: the last step may end inside its 128 inputs; 16-byte pieces past the end are zeros
    const bool in0 = !TAIL || ks * 128 + 16 * q < K, in1 = !TAIL || ks * 128 + 64 + 16 * q < K;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const uint8_t* p = o.wp[i] + (size_t)ks * o.wstep;
        st.w[i][0] = *(const u32x4_t*)(in0 ? p : g_zero16);
        st.w[i][1] = *(const u32x4_t*)(in1 ? p + o.whalf : g_zero16);
        st.ws[i] = o.wsc[i][ks];
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const uint8_t* p = o.xp[j] + ((size_t)ks * 128 + 16 * q) * EB;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < EB; ++c)
                st.x[j][h * EB + c] = *(const u32x4_t*)((h ? in1 : in0) ? p + h * 64 * EB + 16 * c : g_zero16);
        if constexpr (SRC == kSrcFp8) st.xs[j] = o.xsc[j][ks];
    }
}

// acc += the products of steps w, w + S, ... below nst
template <int SRC, int RB, int TB, int D, bool TAIL>
__device__ __forceinline__ void stream(const Operands<RB, TB>& o, int nst, int w, int S, int K,
                                       f32x4_t (&acc)[RB][TB]) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int n = w < nst ? (nst - w + S - 1) / S : 0;  // this wave's steps
    if (n == 0) return;
    Step<SRC, RB, TB> ring[D];
#pragma unroll
    for (int u = 0; u < D; ++u)
        if (u < n) load_step<SRC, RB, TB, TAIL>(o, w + u * S, K, ring[u]);
    for (int i0 = 0; i0 < n; i0 += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            if (i0 + u >= n) break;
            Step<SRC, RB, TB>& st = ring[u];
            Wide8 a[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) a[i] = widen(join8(st.w[i][0], st.w[i][1]));
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                float xs = st.xs[j];
                const Wide8 b = widen(token_operand<SRC>(st.x[j], xs));
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const f32x4_t p = mfma_fp8_exact(a[i], b);
                    const float s = st.ws[i] * xs;
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(p[c], s, acc[i][j][c]);
                }
            }
            if (i0 + u + D < n) load_step<SRC, RB, TB, TAIL>(o, w + (i0 + u + D) * S, K, st);
        }
    }
}

// The S waves' sums of NU units (a unit: one accumulator of all 64 lanes), joined in wave order;
// wave w then holds and handles the units w, w + S, ...: f(unit, this lane's four sums).
template <int NU, typename F>
__device__ __forceinline__ void join_waves(const f32x4_t (&acc)[NU], int w, int S, float4* red, F&& f) {
    const int lane = threadIdx.x & 63;
    if (S == 1) {
#pragma unroll
        for (int u = 0; u < NU; ++u) f(u, acc[u]);
        return;
    }
#pragma unroll
    for (int u = 0; u < NU; ++u)
        red[((size_t)w * NU + u) * 64 + lane] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
    __syncthreads();
    for (int u = w; u < NU; u += S) {
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < S; ++p) {
            const float4 t = red[((size_t)p * NU + u) * 64 + lane];
            v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
        }
        f(u, v);
    }
}

// ---- the dense product ----------------------------------------------------------------------------
template <int RB, int TB, int D, bool TAIL>
__global__ __launch_bounds__(512) void gemm_fp8_stream_kernel(GemmFp8 g) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), S = blockDim.x >> 6;
    const int n0 = blockIdx.x * RB * 16, m0 = blockIdx.y * TB * 16;
    Operands<RB, TB> o;
    o.wstep = 128;
    o.whalf = 64;
#pragma unroll
    for (int i = 0; i < RB; ++i) {  // rows and tokens past the end repeat the last one and are not stored
        o.wp[i] = g.w + (size_t)min(n0 + 16 * i + (lane & 15), g.N - 1) * g.ldw + 16 * (lane >> 4);
        o.wsc[i] = g.w_scale + (size_t)(min(n0 + 16 * i, g.N - 1) / 128) * g.G;
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const int m = min(m0 + 16 * j + (lane & 15), g.M - 1);
        o.xp[j] = g.a + (size_t)m * g.lda;
        o.xsc[j] = g.a_scale + (size_t)m * g.G;
    }
    f32x4_t acc[RB][TB];
    stream<kSrcFp8, RB, TB, D, TAIL>(o, g.G, w, S, g.K, acc);
    join_waves(*(const f32x4_t(*)[RB * TB])&acc, w, S, (float4*)smem, [&](int u, f32x4_t v) {
        const int m = m0 + 16 * (u % TB) + (lane & 15), n = n0 + 16 * (u / TB) + 4 * (lane >> 4);
        if (m < g.M) store_c4(g, m, n, v);
    });
}

template <int RB, int TB, int D>
moe_status launch_gemm(const GemmFp8& g, int S, hipStream_t st) {
    const int64_t gx = (g.N + 16 * RB - 1) / (16 * RB), gy = (g.M + 16 * TB - 1) / (16 * TB);
    MOE_CHECK(gy <= 65535, MOE_ESHAPE, "moe_gemm_fp8: M=%d rows exceed one launch", g.M);
    const int lds = S > 1 ? S * RB * TB * 1024 : 0;
    const bool tail = g.K % 128 != 0;
    auto kern = tail ? gemm_fp8_stream_kernel<RB, TB, D, true> : gemm_fp8_stream_kernel<RB, TB, D, false>;
    if (lds > 65536) MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    ProfScope p("gemm_fp8_stream", st);
    kern<<<dim3((unsigned)gx, (unsigned)gy), 64 * S, lds, st>>>(g);
    return check_launch("gemm_fp8_stream");
}

// ---- the routed experts' projections ----------------------------------------------------------------
template <int MODE, int SRC, int RB, int D>
__global__ __launch_bounds__(512) void ffn_fp8_stream_kernel(FfnFp8 p) {
    static_assert(MODE == kDown || RB % 2 == 0, "gate/up rows come in gate/up pairs");
    extern __shared__ __align__(16) uint8_t smem[];
    const FfnArgs& a = p.a;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), S = blockDim.x >> 6;
    const int K = MODE == kGateUp ? a.d : a.f;
    const int b0 = blockIdx.x * RB;  // first row block
    int e, chunk, slot, n_all, p0;
    if (!find_item(a, 16, blockIdx.y, e, chunk, slot, n_all, p0)) return;
    const bool shared = e == -1;
    const int t0 = chunk * 16, nt = min(16, n_all - t0);
    const uint8_t* base;
    if (shared) {
        base = a.shared_w;
    } else {
        if (slot == MOE_SLOT_ELSEWHERE) return;  // rows produced elsewhere: leave them
        if (slot < 0 || slot >= a.n_slots) {     // absent: flagged, zero rows (h is not read then)
            if (threadIdx.x == 0) *a.status = 1;
            if (MODE == kDown)
                for (int i = threadIdx.x; i < nt * RB * 16; i += blockDim.x) {
                    const int c = b0 * 16 + i % (RB * 16);
                    if (c < a.d) store_y(a, (size_t)(p0 + t0 + i / (RB * 16)), c, 0.f);
                }
            return;
        }
        base = a.pool + (size_t)slot * a.stride;
    }
    Operands<RB, 1> o;
    o.wstep = kFp8Frag;
    o.whalf = kFp8Frag / 2;
    const int nblk = MODE == kGateUp ? 2 * (a.f / 16) : a.d / 16;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int b = min(b0 + i, nblk - 1);
        const uint8_t* blk = base + (MODE == kGateUp ? gu_block_offset(b >> 1, b & 1, a.d, MOE_FP8_B128)
                                                     : down_block_offset(b, a.d, a.f, MOE_FP8_B128));
        o.wp[i] = blk + lane * 16;
        o.wsc[i] = (const float*)(blk + (size_t)16 * K);
    }
    const int row = p0 + t0 + min(lane & 15, nt - 1);  // lanes past the last token repeat it
    int src = row;
    if (MODE == kGateUp) src = shared ? row - a.T * a.k : a.perm[row] / a.k;
    o.xp[0] = (const uint8_t*)(MODE == kGateUp ? a.x : a.h) + (size_t)src * K * SrcOf<SRC>::kBytes;
    o.xsc[0] = SRC == kSrcFp8 ? p.x_scale + (size_t)src * (K / 128) : nullptr;
    f32x4_t acc[RB][1];
    stream<SRC, RB, 1, D, false>(o, K / 128, w, S, K, acc);
    const bool mine = (lane & 15) < nt;
    const size_t orow = (size_t)(p0 + t0 + (lane & 15));
    if constexpr (MODE == kGateUp) {
        // a unit is a gate block and its up block: SwiGLU where their sums meet
        float4* red = (float4*)smem;
#pragma unroll
        for (int i = 0; i < RB; ++i)
            red[((size_t)w * RB + i) * 64 + lane] = make_float4(acc[i][0][0], acc[i][0][1], acc[i][0][2], acc[i][0][3]);
        __syncthreads();
        for (int u = w; u < RB / 2; u += S) {
            float4 g = make_float4(0.f, 0.f, 0.f, 0.f), v = g;
            for (int q = 0; q < S; ++q) {
                const float4 tg = red[((size_t)q * RB + 2 * u) * 64 + lane], tu = red[((size_t)q * RB + 2 * u + 1) * 64 + lane];
                g.x += tg.x, g.y += tg.y, g.z += tg.z, g.w += tg.w;
                v.x += tu.x, v.y += tu.y, v.z += tu.z, v.w += tu.w;
            }
            const int c = (b0 / 2 + u) * 16 + 4 * (lane >> 4);
            if (mine && c < a.f)
                *(float4*)((float*)a.h + orow * a.f + c) =
                    make_float4(silu_mul(g.x, v.x), silu_mul(g.y, v.y), silu_mul(g.z, v.z), silu_mul(g.w, v.w));
        }
    } else {
        join_waves(*(const f32x4_t(*)[RB])&acc, w, S, (float4*)smem, [&](int u, f32x4_t v) {
            const int c = (b0 + u) * 16 + 4 * (lane >> 4);
            if (mine && c < a.d) store_y4(a, orow, c, v[0], v[1], v[2], v[3]);
        });
    }
}

template <int MODE, int SRC, int RB, int D>
moe_status launch_ffn(const FfnFp8& p, int S, hipStream_t st, const char* name) {
    const int nblk = MODE == kGateUp ? 2 * (p.a.f / 16) : p.a.d / 16;
    const int64_t items = work_items(p.a, 16);
    if (items > 65535) return set_error(MOE_ESHAPE, "%s: %lld work items exceed one launch", name, (long long)items);
    const int lds = S * RB * 1024;
    ProfScope sc(name, st);
    ffn_fp8_stream_kernel<MODE, SRC, RB, D><<<dim3((unsigned)((nblk + RB - 1) / RB), (unsigned)items), 64 * S, lds, st>>>(p);
    return check_launch(name);
}

}  // namespace

moe_status gemm_fp8_stream(const GemmFp8& g, hipStream_t st) {
    const int S = std::min(8, g.G);
    if (g.M <= 16) return launch_gemm<1, 1, 4>(g, S, st);
    if (g.M <= 32) return launch_gemm<2, 2, 4>(g, S, st);
    return launch_gemm<2, 4, 1>(g, S, st);
}

moe_status ffn_fp8_stream(const FfnFp8& p, int mode, hipStream_t st) {
    const int S = std::min(8, (mode == kGateUp ? p.a.d : p.a.f) / 128);
    if (mode == kDown) return launch_ffn<kDown, kSrcF32, 2, 2>(p, S, st, "ffn_fp8_down");
    if (p.x_scale) return launch_ffn<kGateUp, kSrcFp8, 2, 4>(p, S, st, "ffn_fp8_gateup");
    return launch_ffn<kGateUp, kSrcBf16, 2, 4>(p, S, st, "ffn_fp8_gateup");
}

}  // namespace moe
