// Products of 8-bit operands with many rows of activations (prefill): tiles on the matrix cores.
//
// A workgroup of NW waves computes MT = NW * RA * 16 weight rows x NT = 16 * NTB tokens; each wave owns RA
// blocks of 16 rows for all of the tile's tokens.  Inputs advance 128 at a time, one scale group: a
// step is one mfma_fp8 (fp8.h; mfma_fp8_exact where the caller wants binary32) per (row block, token
// block), whose sum is added to binary32 accumulators times the token's scale and the row block's.
//
// The tokens go through LDS, in a ring of three stages filled by direct-to-LDS loads.  Weights of
// slots, which lie in operand order, are loaded by each wave straight into registers, one step ahead (two
// register sets take turns); weights of a row-major matrix take an LDS area of the wave's own, because
// operand-order loads of it touch 16 rows at a time.  The scales of the whole tile are put into LDS
// once, before the first step.
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

// This wave's LDS reads done; at most N of its loads still in flight.  The empty asm statements keep the
// compiler from moving LDS accesses across.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0)
    asm volatile("" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));  // vmcnt(N)
    asm volatile("" ::: "memory");
}

template <int RA, int NTB, int NW, bool WLDS>
struct Tile8 {
    static constexpr int kMT = NW * RA * 16, kNT = NTB * 16;
    static constexpr int kStage = NTB * kFp8Frag;
    static constexpr int kUnits = 2 * NTB / NW;  // 1 KB halves of a token block each wave loads a step
    static constexpr int kRing = 3;
    static constexpr int kWBytes = WLDS ? kMT * kFp8Group : 0;  // the waves' weight rows of one step
    static constexpr int kScales = kRing * kStage + kWBytes;    // where the scales begin
    static constexpr int kWScales = kMT >= 128 ? kMT / 128 : 1;  // weight scales a step
    static_assert(kUnits * NW == 2 * NTB, "token blocks must divide over the waves");
    static_assert(NTB % 2 == 0 && RA <= 4 && (!WLDS || NTB >= 4), "pipeline shape");
    // scales of step g: the tokens' at g * (kNT + 1), then (after G steps) the weights'
    static constexpr int lds(int G) { return kScales + 4 * G * (kNT + 1 + kWScales); }
    static_assert(kNT * NW * 4 <= kRing * kStage, "the magnitudes reuse the ring");
};

// A 16-row x 128-input piece of a row-major operand in LDS: row r's eight 16-byte chunks lie at 128 r, chunk
// c at position c ^ (r & 7).  Filled by two 1 KB loads of 8 whole rows each (full cache lines: lanes
// reading 16 different rows cost the address unit four times as much, 93 -> 59 us for 32 steps of one
// workgroup), read back by lane (r, q) as chunks q and 4 + q without bank conflicts.
__device__ __forceinline__ int chunk_of_lane(int lane) { return (lane & 7) ^ (lane >> 3); }  // of row lane / 8
__device__ __forceinline__ int lds_piece(int lane) {  // byte of chunk q; chunk 4 + q is at ^ 64
    const int r = lane & 15, q = lane >> 4;
    return r * 128 + ((q ^ (r & 7)) << 4);
}

// Where a wave's loop finds its operands.
// x[u]: lane l's 16 token bytes of the wave's u-th unit (the next step 128 on).
// WLDS false (slots, fragments in operand order): w + w_off[i] is row block i (of the whole wave).  WLDS true
// (row-major matrix): w + w_off[2 i + h] is lane l's chunk of rows 8 h .. + 7 of row block i.
template <int RA, int UN, bool WLDS>
struct Feed {
    const uint8_t* w;
    uint32_t w_off[WLDS ? 2 * RA : RA];
    const uint8_t* x[UN];
};

// acc = the tile's products over all steps.  MODE decides which scale a row block takes.
//
// The products are software-pipelined by hand across the steps' ends: a product is folded into its
// accumulator RA products later, so the vector unit's four multiply-adds run while the matrix core
// works; token block j + 1 is read from LDS during block j; the next step's weight loads go out one row
// block at a time over the first half of a step; and the waves meet in the middle of a step, where
// the tokens of the next step have landed, so that its first operands are read during the last block.
// (Left to itself the compiler waits for every product before it starts the next.)
// WLDS: the weights take the way through LDS, each wave's rows in an area of its own.  During a step's last
// block the next step's rows have landed, and each row block's registers are read again as soon as
// its last product is on its way; then, in the next step's first block, the area is filled again.
template <int MODE, int RA, int NTB, int NW, bool WLDS, bool EXACT, bool TAIL>
__device__ __forceinline__ void tile_loop(const Feed<RA, Tile8<RA, NTB, NW, WLDS>::kUnits, WLDS>& fd, uint8_t* smem, int nst,
                                          int K, int wv, int lane, f32x4_t (&acc)[RA][NTB]) {
    using TL = Tile8<RA, NTB, NW, WLDS>;
    constexpr int UN = TL::kUnits, MID = NTB / 2, P = RA;
    const float* xs = (const float*)(smem + TL::kScales);
    const float* ws = xs + (size_t)nst * (TL::kNT + 1);
    const int piece = lds_piece(lane);
    uint8_t* w_area = smem + TL::kRing * TL::kStage + wv * RA * kFp8Frag;
    auto in_row = [&](int ks, int chunk) __attribute__((always_inline)) { return !TAIL || ks * 128 + 16 * chunk < K; };
    auto issue_x = [&](int ks, int slot) __attribute__((always_inline)) {
        ks = min(ks, nst - 1);  // past the end: the last stage again, into a slot nobody uses
        uint8_t* buf = smem + slot * TL::kStage;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint8_t* p = fd.x[u] + (size_t)ks * 128;
            load_to_lds(in_row(ks, chunk_of_lane(lane)) ? p : g_zeros, buf + (wv * UN + u) * 1024);
        }
    };
    auto load_w = [&](int ks, int i, u32x4_t (&a)[2]) __attribute__((always_inline)) {
        const uint8_t* p = fd.w + fd.w_off[i] + (size_t)min(ks, nst - 1) * kFp8Frag;
        a[0] = *(const u32x4_t*)(p + lane * 16);
        a[1] = *(const u32x4_t*)(p + lane * 16 + kFp8Frag / 2);
    };
    auto issue_w = [&](int ks) __attribute__((always_inline)) {
        ks = min(ks, nst - 1);
        const uint8_t* base = fd.w + (size_t)ks * 128;
#pragma unroll
        for (int u = 0; u < 2 * RA; ++u)
            load_to_lds(in_row(ks, chunk_of_lane(lane)) ? base + fd.w_off[WLDS ? u : 0] : g_zeros, w_area + u * 1024);
    };
    auto read_w = [&](int i, u32x4_t (&a)[2]) __attribute__((always_inline)) {
        a[0] = *(const u32x4_t*)(w_area + i * kFp8Frag + piece);
        a[1] = *(const u32x4_t*)(w_area + i * kFp8Frag + (piece ^ 64));
    };
    u32x4_t b[2][2];
    float sx[2], f[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, s0, s1;
    f32x4_t p[P];
    auto read_b = [&](int ks, int slot, int j) __attribute__((always_inline)) {
        const uint8_t* sb = smem + slot * TL::kStage + j * kFp8Frag;
        b[j & 1][0] = *(const u32x4_t*)(sb + piece);
        b[j & 1][1] = *(const u32x4_t*)(sb + (piece ^ 64));
        sx[j & 1] = xs[ks * (TL::kNT + 1) + 16 * j + (lane & 15)];
    };
    auto read_s = [&](int ks) __attribute__((always_inline)) {  // this wave's weight scales
        if constexpr (MODE == kGateUp) {  // of its gate and of its up blocks
            s0 = ws[ks * TL::kWScales + 2 * (wv * RA / 16)];
            s1 = ws[ks * TL::kWScales + 2 * (wv * RA / 16) + 1];
        } else {
            s0 = s1 = ws[ks * TL::kWScales + wv * RA / 8];
        }
    };
    auto fold = [&](int t) __attribute__((always_inline)) {
        const int i = t % RA, j = t / RA;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[i][j][c] = __builtin_fmaf(p[i][c], f[j & 1][MODE == kGateUp ? i & 1 : 0], acc[i][j][c]);
    };
    int slot = 0;
    // nxt: the other register set, or (WLDS) cur itself
    auto step = [&](int ks, u32x4_t (&cur)[RA][2], u32x4_t (&nxt)[RA][2]) __attribute__((always_inline)) {
        const int next = slot + 1 < TL::kRing ? slot + 1 : 0, prev = slot >= 1 ? slot - 1 : TL::kRing - 1;
        Wide8 wide[EXACT ? RA : 1];
        if constexpr (EXACT)
#pragma unroll
            for (int i = 0; i < RA; ++i) wide[i] = widen(join8(cur[i][0], cur[i][1]));
#pragma unroll
        for (int t = 0; t < RA * NTB; ++t) {
            const int i = t % RA, j = t / RA;
            // the first block folds what the last block of the step before has left (nothing, scaled by 0, at first)
            fold(t >= P ? t - P : RA * NTB - P + t);
            if (i == 0) {
                f[j & 1][0] = sx[j & 1] * s0;
                f[j & 1][1] = sx[j & 1] * s1;
            }
            const i32x8_t bj = join8(b[j & 1][0], b[j & 1][1]);
            if constexpr (EXACT) p[i] = mfma_fp8_exact(wide[i], widen(bj));
            else p[i] = mfma_fp8(join8(cur[i][0], cur[i][1]), bj);
            __builtin_amdgcn_sched_barrier(0);
            if (i == 0) {
                if (j + 1 < NTB) {
                    read_b(ks, slot, j + 1);
                } else {
                    const int kn = min(ks + 1, nst - 1);
                    read_b(kn, next, 0);
                    read_s(kn);
                }
            }
            if constexpr (!WLDS) {
                if (i == RA - 1 && j < MID) {
#pragma unroll
                    for (int o = 0; o < RA; ++o)
                        if (o * MID / RA == j) load_w(ks + 1, o, nxt[o]);
                }
            }
            if (i == RA - 1 && j == MID - 1) {
                // the tokens of step ks + 1 have landed (younger: weights of step ks + 1), every wave is past step ks - 1
                stage_barrier<2 * RA>();
                issue_x(ks + 2, prev);
            }
            if constexpr (WLDS) {
                if (i == RA - 1 && j == 0) {
                    wait_lds();  // this step's rows are in registers
                    issue_w(ks + 1);
                }
                if (j == NTB - 1) {
                    if (i == 0) wait_loads<UN>();  // the rows of step ks + 1 have landed (younger: tokens of step ks + 2)
                    read_w(i, nxt[i]);
                }
            }
        }
        slot = next;
    };
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        p[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NTB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    u32x4_t a0[RA][2], a1[RA][2];
    issue_x(0, 0);
    if constexpr (WLDS) {
        issue_w(0);
    } else {
#pragma unroll
        for (int i = 0; i < RA; ++i) load_w(0, i, a0[i]);
    }
    issue_x(1, 1);
    stage_barrier<UN>();
    read_b(0, 0, 0);
    read_s(0);
    if constexpr (WLDS) {
#pragma unroll
        for (int i = 0; i < RA; ++i) read_w(i, a0[i]);
        for (int ks = 0; ks < nst; ++ks) step(ks, a0, a0);
    } else {
        int ks = 0;
        for (; ks + 2 <= nst; ks += 2) {
            step(ks, a0, a1);
            step(ks + 1, a1, a0);
        }
        if (ks < nst) step(ks, a0, a1);
    }
#pragma unroll
    for (int t = RA * NTB - P; t < RA * NTB; ++t) fold(t);
    stage_barrier<0>();  // the tail's repeated loads have landed, every wave has left the ring
}

// ---- the dense product ------------------------------------------------------------------------------
template <int RA, int NTB, int NW, bool EXACT, bool TAIL>
__global__ __launch_bounds__(NW * 64, 2) void gemm_fp8_tile_kernel(GemmFp8 g) {
    constexpr bool WLDS = true;
    using TL = Tile8<RA, NTB, NW, WLDS>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * TL::kMT, m0 = blockIdx.y * TL::kNT;
    const int nrow = n0 + wv * RA * 16;  // this wave's first weight row
    Feed<RA, TL::kUnits, WLDS> fd;
    fd.w = g.w + (size_t)n0 * g.ldw;
#pragma unroll
    for (int u = 0; u < 2 * RA; ++u)  // rows past the end repeat the last one and are not stored
        fd.w_off[u] = (uint32_t)(min(nrow + 8 * u + (lane >> 3), g.N - 1) - n0) * (uint32_t)g.ldw + 16 * chunk_of_lane(lane);
#pragma unroll
    for (int u = 0; u < TL::kUnits; ++u) {
        const int m = min(m0 + 8 * (wv * TL::kUnits + u) + (lane >> 3), g.M - 1);
        fd.x[u] = g.a + (size_t)m * g.lda + 16 * chunk_of_lane(lane);
    }
    float* xs = (float*)(smem + TL::kScales);
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
    tile_loop<kDense, RA, NTB, NW, WLDS, EXACT, TAIL>(fd, smem, g.G, g.K, wv, lane, acc);
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
    using TL = Tile8<RA, NTB, NW, true>;
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
    constexpr bool WLDS = false;
    using TL = Tile8<RA, NTB, NW, WLDS>;
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
    Feed<RA, TL::kUnits, WLDS> fd;
    const int bw = blockIdx.x * NW * RA;
    fd.w = base + (MODE == kGateUp ? 0 : down_block_offset(0, a.d, a.f, MOE_FP8_B128)) + (size_t)bw * rbb;
#pragma unroll
    for (int i = 0; i < RA; ++i) fd.w_off[i] = (uint32_t)(min(b0 + i, nblk - 1) - bw) * (uint32_t)rbb;
    // tokens past the tile's end repeat its first; their columns are not stored
    auto source = [&](int t) __attribute__((always_inline)) {
        const int row = p0 + (t < nt ? t : 0);
        if (MODE != kGateUp) return row;
        return shared ? row - a.T * a.k : a.perm[row] / a.k;
    };
    const uint8_t* x = MODE == kGateUp ? p.x8 : p.h8;
    const float* x_scale = MODE == kGateUp ? p.x_scale : p.h_scale;
#pragma unroll
    for (int u = 0; u < TL::kUnits; ++u)
        fd.x[u] = x + (size_t)source(8 * (wv * TL::kUnits + u) + (lane >> 3)) * K + 16 * chunk_of_lane(lane);
    float* xs = (float*)(smem + TL::kScales);
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
    tile_loop<MODE, RA, NTB, NW, WLDS, false, false>(fd, smem, G, K, wv, lane, acc);
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
    using TL = Tile8<RA, NTB, NW, false>;
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
