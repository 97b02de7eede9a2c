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
// Nothing is staged: a wave keeps operands in flight in registers (bound by the weights' bytes; the
// activations are small and come from the caches).  Activations that are not yet in 8 bits
// (bf16 x of a layer, the binary32 h between the projections) are quantised as they are loaded: the
// four lanes l, l ^ 16, l ^ 32, l ^ 48 hold the 128 inputs of a token's group between them.
//
// Experts: one token on 6 of 256 experts of 4096 x 2048 and the shared one (176 MB) 25 + 13.5 us, 4.6 TB/s; 16 tokens
// on 50 of them and the shared one 234 us, 5.5 TB/s (with the tokens prepared again for each row block: 453).
// Dense: one row against 4096 x 2048 (8.4 MB) 4.3 us, of which 3 are a launch and its first loads; 37 rows against
// 2048 x 4096 9.6 us, a wave's 4 steps one after the other: the 32 x 16 and 32 x 32 blocks hold one step in flight, so each
// step's loads wait for the step before.  Deeper rings were measured for the 16 x 16 block alone.
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
template <int RB, int TB>
struct Step {
    u32x4_t w[RB][2];
    float ws[RB];
    u32x4_t x[TB][2];
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

// Where a wave of the dense product finds its operands: wp[i] is lane l's first 16 bytes of row block i
// (the second half 64 bytes on, the next step 128 bytes on), wsc[i] the block's scales by step; xp[j] the
// row of lane l's token of block j, xsc[j] its scales.
template <int RB, int TB>
struct Operands {
    const uint8_t* wp[RB];
    const float* wsc[RB];
    const uint8_t* xp[TB];
    const float* xsc[TB];
};

template <int RB, int TB, bool TAIL>
__device__ __forceinline__ void load_step(const Operands<RB, TB>& o, int ks, int K, Step<RB, TB>& st) {
    const int q = (threadIdx.x & 63) >> 4;
    // TAIL: the last step may end inside its 128 inputs; 16-byte pieces past the end are zeros
    const bool in0 = !TAIL || ks * 128 + 16 * q < K, in1 = !TAIL || ks * 128 + 64 + 16 * q < K;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const uint8_t* p = o.wp[i] + (size_t)ks * 128;
        st.w[i][0] = *(const u32x4_t*)(in0 ? p : g_zero16);
        st.w[i][1] = *(const u32x4_t*)(in1 ? p + 64 : g_zero16);
        st.ws[i] = o.wsc[i][ks];
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const uint8_t* p = o.xp[j] + (size_t)ks * 128 + 16 * q;
        st.x[j][0] = *(const u32x4_t*)(in0 ? p : g_zero16);
        st.x[j][1] = *(const u32x4_t*)(in1 ? p + 64 : g_zero16);
        st.xs[j] = o.xsc[j][ks];
    }
}

// acc += the products of steps w, w + S, ... below nst
template <int RB, int TB, int D, bool TAIL>
__device__ __forceinline__ void stream(const Operands<RB, TB>& o, int nst, int w, int S, int K,
                                       f32x4_t (&acc)[RB][TB]) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int n = w < nst ? (nst - w + S - 1) / S : 0;  // this wave's steps
    if (n == 0) return;
    Step<RB, TB> ring[D];
#pragma unroll
    for (int u = 0; u < D; ++u)
        if (u < n) load_step<RB, TB, TAIL>(o, w + u * S, K, ring[u]);
    for (int i0 = 0; i0 < n; i0 += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            if (i0 + u >= n) break;
            Step<RB, TB>& st = ring[u];
            Wide8 a[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) a[i] = widen(join8(st.w[i][0], st.w[i][1]));
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const Wide8 b = widen(join8(st.x[j][0], st.x[j][1]));
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const f32x4_t p = mfma_fp8_exact(a[i], b);
                    const float s = st.ws[i] * st.xs[j];
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(p[c], s, acc[i][j][c]);
                }
            }
            if (i0 + u + D < n) load_step<RB, TB, TAIL>(o, w + (i0 + u + D) * S, K, st);
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

// ---- up to 16 tokens ----------------------------------------------------------------------------------
// One token block, RBW row blocks a workgroup (4: 16 KB of weights in flight a wave at a ring of 8): the wave's token operands (NS steps) are prepared once and stay
// in registers, and its RBW * NS weight fragments stream through a ring of D.  frag(i, ks): this lane's
// first 16 bytes of row block i at step ks, the second half kFp8Frag / 2 on; wscale(i): the block's scales.
// EVEN: S * NS = nst, every wave has NS steps; else wave w has those of w, w + S, ... that exist.
template <int SRC, int NS, int RBW, int D, bool EVEN, typename FP, typename SP>
__device__ __forceinline__ void stream_rows(FP&& frag, SP&& wscale, const uint8_t* xrow, const float* xscale, int nst,
                                            int w, int S, f32x4_t (&acc)[RBW]) {
    constexpr int EB = SrcOf<SRC>::kBytes;
    const int q = (threadIdx.x & 63) >> 4;
    const int n = EVEN ? NS : min(NS, max(0, (nst - w + S - 1) / S));
    u32x4_t rw[D][2];
    float rs[D];
    auto load = [&](int idx) __attribute__((always_inline)) {
        const int i = idx / NS, t = idx % NS, ks = w + t * S;
        if (!EVEN && t >= n) return;
        const uint8_t* p = frag(i, ks);
        rw[idx % D][0] = __builtin_nontemporal_load((const u32x4_t*)p);
        rw[idx % D][1] = __builtin_nontemporal_load((const u32x4_t*)(p + kFp8Frag / 2));
        rs[idx % D] = wscale(i)[ks];
    };
#pragma unroll
    for (int idx = 0; idx < (D < RBW * NS ? D : RBW * NS); ++idx) load(idx);
    constexpr bool kWide = NS <= 2;  // few steps: their tokens are kept as bf16
    Wide8 xw[kWide ? NS : 1];
    i32x8_t xr[kWide ? 1 : NS];
    float xs[NS];
#pragma unroll
    for (int t = 0; t < NS; ++t) {
        if (!EVEN && t >= n) continue;
        const int ks = w + t * S;
        const uint8_t* p = xrow + ((size_t)ks * 128 + 16 * q) * EB;
        u32x4_t x[2 * EB];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < EB; ++c) x[h * EB + c] = *(const u32x4_t*)(p + h * 64 * EB + 16 * c);
        if constexpr (SRC == kSrcFp8) xs[t] = xscale[ks];
        if constexpr (kWide) xw[t] = widen(token_operand<SRC>(x, xs[t]));
        else xr[t] = token_operand<SRC>(x, xs[t]);
    }
#pragma unroll
    for (int i = 0; i < RBW; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int idx = 0; idx < RBW * NS; ++idx) {
        const int i = idx / NS, t = idx % NS;
        if (EVEN || t < n) {
            const f32x4_t p = mfma_fp8_exact(widen(join8(rw[idx % D][0], rw[idx % D][1])), kWide ? xw[kWide ? t : 0] : widen(xr[kWide ? 0 : t]));
            const float f = rs[idx % D] * xs[t];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = __builtin_fmaf(p[c], f, acc[i][c]);
        }
        if (idx + D < RBW * NS) load(idx + D);
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
    stream<RB, TB, D, TAIL>(o, g.G, w, S, g.K, acc);
    join_waves(*(const f32x4_t(*)[RB * TB])&acc, w, S, (float4*)smem, [&](int u, f32x4_t v) {
        const int m = m0 + 16 * (u % TB) + (lane & 15), n = n0 + 16 * (u / TB) + 4 * (lane >> 4);
        if (m < g.M) store_c4(g, m, n, v);
    });
}

template <int RB, int TB, int D>
moe_status launch_gemm(const GemmFp8& g, int S, hipStream_t st) {
    const int64_t gx = blocks_of(g.N, 16 * RB), gy = blocks_of(g.M, 16 * TB);
    MOE_CHECK(gy <= 65535, MOE_ESHAPE, "moe_gemm_fp8: M=%d rows exceed one launch", g.M);
    const int lds = S > 1 ? S * RB * TB * 1024 : 0;
    const bool tail = g.K % 128 != 0;
    auto kern = tail ? gemm_fp8_stream_kernel<RB, TB, D, true> : gemm_fp8_stream_kernel<RB, TB, D, false>;
    ProfScope p("gemm_fp8_stream", st);
    kern<<<dim3((unsigned)gx, (unsigned)gy), 64 * S, lds, st>>>(g);
    return check_launch("gemm_fp8_stream");
}

// ---- the routed experts' projections ----------------------------------------------------------------
template <int MODE, int SRC, int NS, int RBW, int D, bool EVEN>
__global__ __launch_bounds__(NS == 8 ? 1024 : 512, 4) void ffn_fp8_stream_kernel(FfnFp8 p) {
    static_assert(MODE == kDown || RBW % 2 == 0, "gate/up rows come in gate/up pairs");
    extern __shared__ __align__(16) uint8_t smem[];
    const FfnArgs& a = p.a;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), S = blockDim.x >> 6;
    const int K = MODE == kGateUp ? a.d : a.f;
    const int b0 = blockIdx.x * RBW;  // first row block
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
                for (int i = threadIdx.x; i < nt * RBW * 16; i += blockDim.x) {
                    const int c = b0 * 16 + i % (RBW * 16);
                    if (c < a.d) store_y(a, (size_t)(p0 + t0 + i / (RBW * 16)), c, 0.f);
                }
            return;
        }
        base = a.pool + (size_t)slot * a.stride;
    }
    const int nblk = MODE == kGateUp ? 2 * (a.f / 16) : a.d / 16;
    const size_t rbb = rowblock_bytes(K, MOE_FP8_B128);
    if (MODE == kDown) base += down_block_offset(0, a.d, a.f, MOE_FP8_B128);
    // blocks past the end repeat the last one and are not stored
    auto block = [&](int i) __attribute__((always_inline)) { return base + (size_t)min(b0 + i, nblk - 1) * rbb; };
    auto frag = [&](int i, int ks) __attribute__((always_inline)) { return block(i) + (size_t)ks * kFp8Frag + lane * 16; };
    auto wscale = [&](int i) __attribute__((always_inline)) { return (const float*)(block(i) + (size_t)16 * K); };
    const int row = p0 + t0 + min(lane & 15, nt - 1);  // lanes past the last token repeat it
    int src = row;
    if (MODE == kGateUp) src = shared ? row - a.T * a.k : a.perm[row] / a.k;
    const uint8_t* x = MODE == kDown ? (const uint8_t*)a.h : SRC == kSrcFp8 ? p.x8 : (const uint8_t*)a.x;
    f32x4_t acc[RBW];
    stream_rows<SRC, NS, RBW, D, EVEN>(frag, wscale, x + (size_t)src * K * SrcOf<SRC>::kBytes,
                                       SRC == kSrcFp8 ? p.x_scale + (size_t)src * (K / 128) : nullptr, K / 128, w, S, acc);
    const bool mine = (lane & 15) < nt;
    const size_t orow = (size_t)(p0 + t0 + (lane & 15));
    float4* red = (float4*)smem;
#pragma unroll
    for (int i = 0; i < RBW; ++i) red[((size_t)w * RBW + i) * 64 + lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    auto joined = [&](int i) __attribute__((always_inline)) {  // the waves' sums of row block i, in wave order
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int o = 0; o < S; ++o) {
            const float4 t = red[((size_t)o * RBW + i) * 64 + lane];
            v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
        }
        return v;
    };
    if constexpr (MODE == kGateUp) {
        for (int u = w; u < RBW / 2; u += S) {  // a gate block and its up block: SwiGLU where their sums meet
            const float4 g = joined(2 * u), v = joined(2 * u + 1);
            const int c = (b0 / 2 + u) * 16 + 4 * (lane >> 4);
            if (mine && c < a.f)
                *(float4*)((float*)a.h + orow * a.f + c) =
                    make_float4(silu_mul(g.x, v.x), silu_mul(g.y, v.y), silu_mul(g.z, v.z), silu_mul(g.w, v.w));
        }
    } else {
        for (int u = w; u < RBW; u += S) {
            const float4 v = joined(u);
            const int c = (b0 + u) * 16 + 4 * (lane >> 4);
            if (mine && c < a.d) store_y4(a, orow, c, v.x, v.y, v.z, v.w);
        }
    }
}

template <int MODE, int SRC, int NS, int RBW, int D, bool EVEN>
moe_status launch_rows(const FfnFp8& p, int S, hipStream_t st, const char* name) {
    const int nblk = MODE == kGateUp ? 2 * (p.a.f / 16) : p.a.d / 16;
    const int64_t items = work_items(p.a, 16);
    if (items > 65535) return set_error(MOE_ESHAPE, "%s: %lld work items exceed one launch", name, (long long)items);
    if (items <= 0) return MOE_OK;
    const int lds = S * RBW * 1024;  // 64 KB at most (16 waves)
    auto kern = ffn_fp8_stream_kernel<MODE, SRC, NS, RBW, D, EVEN>;
    ProfScope sc(name, st);
    kern<<<dim3((unsigned)((nblk + RBW - 1) / RBW), (unsigned)items), 64 * S, lds, st>>>(p);
    return check_launch(name);
}

// S waves that split nst steps, NS each at most: 4 to 8 waves, which leaves two workgroups a compute unit, with as few
// steps each as that allows
struct Split {
    int S, NS;
    bool even;
};
Split split_steps(int nst) {
    for (int ns = 1; ns <= 4; ns *= 2)  // 4 to 8 waves without a rest
        if (nst % ns == 0 && nst / ns >= 4 && nst / ns <= 8) return {nst / ns, ns, true};
    if (nst < 4) return {nst, 1, true};
    int ns = 2;
    while ((nst + ns - 1) / ns > (ns < 8 ? 8 : 16)) ns *= 2;
    return {(nst + ns - 1) / ns, ns, false};
}

template <int MODE, int SRC>
moe_status launch_split(const FfnFp8& p, hipStream_t st, const char* name) {
    const Split sp = split_steps((MODE == kGateUp ? p.a.d : p.a.f) / 128);
    constexpr int RBW = 4;
    if (sp.even) {
        if (sp.NS == 1) return launch_rows<MODE, SRC, 1, RBW, 4, true>(p, sp.S, st, name);
        if (sp.NS == 2) return launch_rows<MODE, SRC, 2, RBW, 8, true>(p, sp.S, st, name);
        return launch_rows<MODE, SRC, 4, RBW, 8, true>(p, sp.S, st, name);
    }
    if (sp.NS == 2) return launch_rows<MODE, SRC, 2, RBW, 4, false>(p, sp.S, st, name);
    if (sp.NS == 4) return launch_rows<MODE, SRC, 4, RBW, 4, false>(p, sp.S, st, name);
    return launch_rows<MODE, SRC, 8, RBW, 4, false>(p, sp.S, st, name);
}

}  // namespace

// The dense product's workgroup: the smallest block of weight rows x tokens that leaves no compute unit a
// second workgroup, and 32 x 32 where none does.  Measured (us, 16x16 / 32x16 / 32x32, weights N x K):
// 16 x 8192 x 4096 12.7 / 10.2 / 10.7, 32 x 4096 x 2048 7.5 / 6.4 / 7.7, 16 x 2048 x 4096 7.6 / 9.3 / 9.9,
// 64 x 2048 x 4096 11.9 / 9.4 / 12.2, 64 x 8192 x 4096 38 / 28 / 22; 64 rows or 64 tokens are slower at all.
namespace {
struct StreamBlock {
    int rb, tb;
    int64_t wgs;
};
StreamBlock stream_block(const GemmFp8& g) {
    auto wgs = [&](int rb, int tb) { return blocks_of(g.N, 16 * rb) * blocks_of(g.M, 16 * tb); };
    if (wgs(1, 1) <= 256) return {1, 1, wgs(1, 1)};
    if (wgs(2, 1) <= 256) return {2, 1, wgs(2, 1)};
    return {2, 2, wgs(2, 2)};
}
}  // namespace

// Estimated time (us), where a tile may be faster: 3.5 us and, for each 128-input step of a wave and each
// round of 256 workgroups, 1, 1.5 or 2.2 us (within 6% of the figures above and of 24 more up to 128 rows).
// Up to 16 rows no tile is faster.
float gemm_fp8_stream_us(const GemmFp8& g) {
    if (g.M <= 16) return 0.f;
    const StreamBlock b = stream_block(g);
    return 3.5f + (float)blocks_of(g.G, 8) * (b.rb == 1 ? 1.0f : b.tb == 1 ? 1.5f : 2.2f) * (float)((b.wgs + 255) / 256);
}

moe_status gemm_fp8_stream(const GemmFp8& g, hipStream_t st) {
    const int S = std::min(8, g.G);
    const StreamBlock b = stream_block(g);
    if (b.rb == 1) return launch_gemm<1, 1, 2>(g, S, st);
    if (b.tb == 1) return launch_gemm<2, 1, 1>(g, S, st);
    return launch_gemm<2, 2, 1>(g, S, st);
}

moe_status ffn_fp8_stream(const FfnFp8& p, int mode, hipStream_t st) {
    if (mode == kDown) return launch_split<kDown, kSrcF32>(p, st, "ffn_fp8_down");
    if (p.x8) return launch_split<kGateUp, kSrcFp8>(p, st, "ffn_fp8_gateup");
    return launch_split<kGateUp, kSrcBf16>(p, st, "ffn_fp8_gateup");
}

}  // namespace moe
