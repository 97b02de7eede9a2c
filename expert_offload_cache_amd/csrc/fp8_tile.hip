// Products of 8-bit operands with many rows of activations (prefill): tiles on the matrix cores.
//
// A workgroup of NW waves computes MT = NW * RA * 16 weight rows x NT = 16 * NTB tokens; each wave owns RA
// blocks of 16 rows for all of the tile's tokens.  Inputs advance 128 at a time, one scale group: a
// step is one mfma_fp8 (fp8.h; mfma_fp8_exact where the result is binary32 or h) per (row block, token
// block), whose sum is added to binary32 accumulators times the token's scale and the row block's.
//
// Both operands go through LDS by direct-to-LDS loads: the tokens, which every wave reads, in a ring of
// RX steps; each wave's weight rows in a ring of RW steps of its own.  (Weights straight into
// registers take two register sets, which does not leave room for the products in flight: experts of
// 8192 tokens 1.69 ms against 1.61, both with e4m3 sums; and operand-order loads of a row-major matrix
// touch 16 rows at a time.)  The scales of the whole tile are put into LDS once, before the first step.
//
// Gate/up: a wave's row blocks are gate and up blocks in turn, so SwiGLU happens in registers; the
// 16 / RA waves that share a 128-column group of h join their largest magnitudes through LDS, and h is
// written in 8 bits with its scale.
//
// Measured: 8192 x 4096 x 4096 in 125 to 131 us, 2.1 to 2.2 PFLOP/s.  Counters: the matrix cores are busy 60 % of the
// units' cycles, the vector units about as much (four multiply-adds a product and one instruction more), LDS 29 %, bank
// conflicts 3 % of that; the loop holds 32 products in 285 instructions.  What is left is two waves a SIMD that both wait
// at a step's barrier and for operands one block ahead: the accumulators, 128 registers, leave no room for a third
// wave or a longer lead (reading two token blocks ahead, 32 x 32 products and buffer loads to LDS gained nothing).
// 8192 tokens on 6 of 256 experts of 4096 x 2048 and the shared one, the six the same: gate/up 1750 to 1890 us,
// 1.0 to 1.1 PFLOP/s (the library's bf16 product of 8192^3 reaches 1.63), the bf16 rows of the down projection 490 to 505,
// 1.9 PFLOP/s.  Gate/up: the matrix cores 50 % busy, LDS 16 %; four vector instructions beside each matrix instruction,
// two of them widenings, since every wave widens the tokens' operands for itself.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "ffn_common.h"
#include "fp8_ops.h"
#include "slot_layout.h"

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* gbl_ptr_t;

constexpr int kLds = 160 << 10;  // LDS of a compute unit
constexpr int kXCDs = 8;         // workgroup i runs on XCD i mod 8
constexpr int kCUs = 256;        // compute units (a multiple of the 8 XCDs)

enum { kDense = 2 };  // beside kGateUp and kDown
enum { kWFrags = 0, kWRows = 1 };  // the weights: a slot's fragments, or the rows of a matrix

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

template <int RA, int NTB, int NW, int RW, int RX>
struct Tile8 {
    static constexpr int kMT = NW * RA * 16, kNT = NTB * 16;
    static constexpr int kStage = NTB * kFp8Frag;
    static constexpr int kUnits = 2 * NTB / NW;  // 1 KB halves of a token block each wave loads a step
    static constexpr int kWBytes = kMT * kFp8Group;             // the waves' weight rows of one step
    static constexpr int kScales = RX * kStage + RW * kWBytes;  // where the scales begin
    static constexpr int kWScales = kMT >= 128 ? kMT / 128 : 1;  // weight scales a step
    static_assert(kUnits * NW == 2 * NTB, "token blocks must divide over the waves");
    static_assert(NTB % 2 == 0 && NTB >= 4 && RA <= 4, "pipeline shape");
    static_assert(RX >= 3 && RX >= RW && RX <= RW + 3, "the waits count on loads of both operands between two of one");
    // scales of step g: the tokens' at g * (kNT + 1), then (after G steps) the weights'
    static constexpr int lds(int G) { return kScales + 4 * G * (kNT + 1 + kWScales); }
    static_assert(kNT * NW * 4 <= RX * kStage, "the magnitudes reuse the ring");
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
// Slots (fragments in operand order): w + w_off[i] is row block i (of the whole wave).  kWRows: w + w_off[2 i + h]
// is lane l's chunk of rows 8 h .. + 7 of row block i.
template <int RA, int UN, int W>
struct Feed {
    const uint8_t* w;
    uint32_t w_off[W == kWRows ? 2 * RA : RA];
    const uint8_t* x[UN];
};

// acc = the tile's products over its nst steps, of which the first `given` exist (TAIL: the rest are
// scaled by 0 and load nothing of the rows).  MODE decides which scale a row block takes.
//
// The products are software-pipelined by hand across the steps' ends: a product is folded into its
// accumulator four products later, so the vector unit's four multiply-adds run while the matrix core
// works; token blocks are read from LDS one or two blocks ahead; and the waves meet in the middle of a step,
// where the tokens of the next step have landed, so that its first operands are read during the last block.
// (Left to itself the compiler waits for every product before it starts the next.)
// The weights of a wave's rows take the way through an LDS ring of its own of RW steps: during a step's
// last block the next step's rows have landed, and each row block's registers are read again as soon as
// its last product is on its way; in the next step's first block the slot they left is filled again.
template <int MODE, int RA, int NTB, int NW, int RW, int RX, int W, bool EXACT, bool TAIL, typename SX, typename SW>
__device__ __forceinline__ void tile_loop(const Feed<RA, Tile8<RA, NTB, NW, RW, RX>::kUnits, W>& fd, uint8_t* smem, int nst,
                                          int given, int K, int wv, int lane, int tid, SX&& x_scales, SW&& w_scales,
                                          f32x4_t (&acc)[RA][NTB]) {
    using TL = Tile8<RA, NTB, NW, RW, RX>;
    constexpr int UN = TL::kUnits, WN = 2 * RA;  // token and weight loads of a step
    constexpr int MID = NTB / 2;
    constexpr int P = 4;                    // products in flight
    constexpr int BA = RA == 4 ? 1 : 2;     // token blocks read ahead: four products or more before they are needed
    constexpr int BN = 2 * BA, BM = BN - 1;  // their registers take turns
    // the last block's weights for the next step: read over themselves, or (few products a block) one
    // block earlier into the other of two sets
    constexpr bool kTwoSets = RA < 4;
    constexpr int WJ = kTwoSets ? NTB - 2 : NTB - 1;
    static_assert(NTB % BN == 0 && (RA * NTB) % P == 0, "registers take turns across steps");
    const float* xs = (const float*)(smem + TL::kScales);
    const float* ws = xs + (size_t)nst * (TL::kNT + 1);
    const int piece = lds_piece(lane);
    uint8_t* w_area = smem + RX * TL::kStage + wv * RA * kFp8Frag;
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
    auto issue_w = [&](int ks, int wslot) __attribute__((always_inline)) {
        uint8_t* area = w_area + wslot * TL::kWBytes;
        ks = min(ks, nst - 1);
#pragma unroll
        for (int u = 0; u < 2 * RA; ++u) {
            const uint8_t* p;
            if constexpr (W == kWRows) p = in_row(ks, chunk_of_lane(lane)) ? fd.w + fd.w_off[u] + (size_t)ks * 128 : g_zeros;
            else p = fd.w + fd.w_off[u / 2] + (size_t)ks * kFp8Frag + (u & 1) * 1024 + lane * 16;
            load_to_lds(p, area + u * 1024);
        }
    };
    auto read_w = [&](int wslot, int i, u32x4_t (&a)[2]) __attribute__((always_inline)) {
        const uint8_t* p = w_area + wslot * TL::kWBytes + i * kFp8Frag;
        a[0] = *(const u32x4_t*)(p + (W == kWRows ? piece : lane * 16));
        a[1] = *(const u32x4_t*)(p + (W == kWRows ? piece ^ 64 : lane * 16 + kFp8Frag / 2));
    };
    u32x4_t b[BN][2];
    float sx[BN], f[BN][2], s0, s1;
    f32x4_t p[P];
    auto read_b = [&](int ks, int slot, int j) __attribute__((always_inline)) {
        const uint8_t* sb = smem + slot * TL::kStage + j * kFp8Frag;
        b[j & BM][0] = *(const u32x4_t*)(sb + piece);
        b[j & BM][1] = *(const u32x4_t*)(sb + (piece ^ 64));
        sx[j & BM] = xs[ks * (TL::kNT + 1) + 16 * j + (lane & 15)];
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
            acc[i][j][c] = __builtin_fmaf(p[t % P][c], f[j & BM][MODE == kGateUp ? i & 1 : 0], acc[i][j][c]);
    };
    int slot = 0, wslot = 0;
    auto step = [&](int ks, u32x4_t (&a)[RA][2], u32x4_t (&nxt)[RA][2]) __attribute__((always_inline)) {
        const int next = slot + 1 < RX ? slot + 1 : 0, prev = slot >= 1 ? slot - 1 : RX - 1;  // the slots of steps ks + 1 and ks - 1
        const int wnext = wslot + 1 < RW ? wslot + 1 : 0;
        Wide8 wide[EXACT ? RA : 1];
        if constexpr (EXACT)
#pragma unroll
            for (int i = 0; i < RA; ++i) wide[i] = widen(join8(a[i][0], a[i][1]));
#pragma unroll
        for (int t = 0; t < RA * NTB; ++t) {
            const int i = t % RA, j = t / RA;
            // first the products that the step before has left are folded (none, scaled by 0, at first)
            fold(t >= P ? t - P : RA * NTB - P + t);
            if (i == 0) {
                f[j & BM][0] = sx[j & BM] * s0;
                f[j & BM][1] = sx[j & BM] * s1;
            }
            const i32x8_t bj = join8(b[j & BM][0], b[j & BM][1]);
            if constexpr (EXACT) p[t % P] = mfma_fp8_exact(wide[i], widen(bj));
            else p[t % P] = mfma_fp8(join8(a[i][0], a[i][1]), bj);
            __builtin_amdgcn_sched_barrier(0);
            if (i == 0) {
                const int kn = min(ks + 1, nst - 1);
                if (j + BA < NTB) read_b(ks, slot, j + BA);
                else read_b(kn, next, j + BA - NTB);
                if (j == NTB - 1) read_s(kn);
            }
            if (i == RA - 1 && j == 0) {
                wait_lds();  // this step's weights are in registers: their slot can be filled again
                issue_w(ks + RW, wslot);
            }
            if (i == RA - 1 && j == MID - 1) {
                // the tokens of step ks + 1 have landed (younger: the weights asked for since, and the tokens of
                // the steps ks + 2 ..), every wave is past step ks - 1
                stage_barrier<(RX - 2) * WN + (RX - 3) * UN>();
                issue_x(ks + RX - 1, prev);
            }
            if (j == WJ) {
                // the weights of step ks + 1 have landed (younger: those of ks + 2 .. ks + RW, and the tokens between)
                if (i == 0) wait_loads<(RW - 1) * (WN + UN) + UN>();
                read_w(wnext, i, nxt[i]);
            }
        }
        slot = next;
        wslot = wnext;
    };
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < BN; ++i) f[i][0] = f[i][1] = 0.f;
#pragma unroll
    for (int i = 0; i < RA; ++i) {
#pragma unroll
        for (int j = 0; j < NTB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // the loads in the order in which steps before the first would have issued them, so that the waits' counts hold
    constexpr int kBefore = RW > RX - 1 ? RW : RX - 1;
#pragma unroll
    for (int o = -kBefore; o < 0; ++o) {
        if (o + RW >= 0) issue_w(o + RW, o + RW);
        if (o + RX - 1 >= 0) issue_x(o + RX - 1, o + RX - 1);
    }
    // Meanwhile the scales of the whole tile: the tokens' (x_scales(token): its row of scales), then
    // those of the weights' 128-row blocks (w_scales(block)).
    {
        float* to = (float*)(smem + TL::kScales);
        // a thread takes one token, and 4 of its scales at a time
        const int t = tid % TL::kNT;
        const float* from = x_scales(t);
        const bool whole = (uintptr_t)from % 16 == 0;
#pragma unroll 2
        for (int k = 4 * (tid / TL::kNT); k < nst; k += 4 * (NW * 64 / TL::kNT)) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (whole && k + 4 <= given) {
                v = *(const float4*)(from + k);
            } else {
                if (k < given) v.x = from[k];
                if (k + 1 < given) v.y = from[k + 1];
                if (k + 2 < given) v.z = from[k + 2];
                if (k + 3 < given) v.w = from[k + 3];
            }
            to[k * (TL::kNT + 1) + t] = v.x;
            if (k + 1 < nst) to[(k + 1) * (TL::kNT + 1) + t] = v.y;
            if (k + 2 < nst) to[(k + 2) * (TL::kNT + 1) + t] = v.z;
            if (k + 3 < nst) to[(k + 3) * (TL::kNT + 1) + t] = v.w;
        }
        to += (size_t)nst * (TL::kNT + 1);
        for (int i = tid; i < nst * TL::kWScales; i += NW * 64) {
            const int b = i / nst, k = i - b * nst;
            to[k * TL::kWScales + b] = !TAIL || k < given ? w_scales(b)[k] : 0.f;
        }
    }
    // weights and tokens of step 0 have landed
    constexpr int kAfterW = (RW - 1) * WN + (RW < RX - 1 ? RW : RX - 1) * UN;
    constexpr int kAfterX = (RX - 2) * UN + (RW < RX - 2 ? RW : RX - 2) * WN;
    stage_barrier<(kAfterW < kAfterX ? kAfterW : kAfterX)>();
#pragma unroll
    for (int j = 0; j < BA; ++j) read_b(0, 0, j);
    read_s(0);
    u32x4_t a[RA][2], a2[RA][2];
#pragma unroll
    for (int i = 0; i < RA; ++i) read_w(0, i, a[i]);
    if constexpr (kTwoSets) {
        int ks = 0;
        for (; ks + 2 <= nst; ks += 2) {
            step(ks, a, a2);
            step(ks + 1, a2, a);
        }
        if (ks < nst) step(ks, a, a2);
    } else {
        for (int ks = 0; ks < nst; ++ks) step(ks, a, a);
    }
#pragma unroll
    for (int t = RA * NTB - P; t < RA * NTB; ++t) fold(t);
    stage_barrier<0>();  // the tail's repeated loads have landed, every wave has left the ring
}

// A wave's sums (RA * 16 columns x NTB * 16 tokens) to rows of E (bf16 or binary32), through LDS so that a
// store takes whole pieces of rows: 1 KB of 16-byte chunks a wave instead of 16 rows x 32 bytes.  area: 8 KB of
// the wave's own.  row(t): where token t's columns begin, nullptr to leave them; cols of them exist; wide:
// rows start on 16 bytes.  Chunk c of token t lies at position c ^ (t mod chunks of a row).
template <typename E, int RA, int NTB, typename Row>
__device__ __forceinline__ void store_rows(const f32x4_t (&acc)[RA][NTB], uint8_t* area, int lane, int cols, bool wide,
                                           Row&& row) {
    constexpr int BYTES = RA * 16 * sizeof(E), CH = BYTES / 16, PER = 16 / sizeof(E);  // of a token; elements a chunk
    constexpr int JP = 8192 / (16 * BYTES) < NTB ? 8192 / (16 * BYTES) : NTB;            // token blocks a pass
    const int q = lane >> 4;
#pragma unroll
    for (int j0 = 0; j0 < NTB; j0 += JP) {
        wait_lds();  // the pass before has been read
#pragma unroll
        for (int j = j0; j < j0 + JP; ++j) {
            const int t = 16 * (j - j0) + (lane & 15);
#pragma unroll
            for (int i = 0; i < RA; ++i) {
                const f32x4_t v = acc[i][j];
                if constexpr (sizeof(E) == 2) {
                    uint2 o;
                    o.x = bf16_pair(v[0], v[1]);
                    o.y = bf16_pair(v[2], v[3]);
                    *(uint2*)(area + t * BYTES + (((2 * i + (q >> 1)) ^ (t & (CH - 1))) << 4) + 8 * (q & 1)) = o;
                } else {
                    *(float4*)(area + t * BYTES + (((4 * i + q) ^ (t & (CH - 1))) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        wait_lds();
        if (wide && cols >= RA * 16) {
            for (int i = lane; i < JP * 16 * CH; i += 64) {
                const int t = i / CH, c = i % CH;
                E* to = row(16 * j0 + t);
                if (to) *(u32x4_t*)(to + c * PER) = *(const u32x4_t*)(area + t * BYTES + ((c ^ (t & (CH - 1))) << 4));
            }
        } else {  // element by element, neighbouring lanes neighbouring columns
            for (int i = lane; i < JP * 16 * RA * 16; i += 64) {
                const int t = i / (RA * 16), c = i % (RA * 16);
                E* to = row(16 * j0 + t);
                if (to && c < cols)
                    to[c] = *(const E*)(area + t * BYTES + (((c / PER) ^ (t & (CH - 1))) << 4) + (c % PER) * sizeof(E));
            }
        }
    }
}

// ---- the dense product ------------------------------------------------------------------------------
// KG groups of NW waves each take a run of steps of the same tile, in an LDS area of their own, and join their sums
// in group order: where there are fewer tiles than compute units, half the steps one after the other.
template <int RA, int NTB, int NW, int RW, int RX, int KG>
struct GemmTile : Tile8<RA, NTB, NW, RW, RX> {
    using TL = Tile8<RA, NTB, NW, RW, RX>;
    static constexpr int group_lds(int G) { return (TL::lds((G + KG - 1) / KG) + 15) / 16 * 16; }
    static constexpr int gemm_lds(int G) { return KG * group_lds(G); }
};

template <int RA, int NTB, int NW, int RW, int RX, int KG, bool EXACT, bool TAIL>
__global__ __launch_bounds__(NW * KG * 64, 2) void gemm_fp8_tile_kernel(GemmFp8 g) {
    using TL = GemmTile<RA, NTB, NW, RW, RX, KG>;
    typedef std::conditional_t<EXACT, float, uint16_t> OutT;  // binary32 results are the exact ones
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = KG > 1 ? wave / NW : 0, wv = wave - kg * NW;
    const int n0 = blockIdx.x * TL::kMT, m0 = blockIdx.y * TL::kNT;
    const int nrow = n0 + wv * RA * 16;  // this wave's first weight row
    const int nst = (g.G + KG - 1) / KG, s0 = kg * nst;  // this group's steps
    uint8_t* mine = smem + kg * TL::group_lds(g.G);
    Feed<RA, TL::kUnits, kWRows> fd;
    fd.w = g.w + (size_t)n0 * g.ldw + (size_t)s0 * kFp8Group;
#pragma unroll
    for (int u = 0; u < 2 * RA; ++u)  // rows past the end repeat the last one and are not stored
        fd.w_off[u] = (uint32_t)(min(nrow + 8 * u + (lane >> 3), g.N - 1) - n0) * (uint32_t)g.ldw + 16 * chunk_of_lane(lane);
#pragma unroll
    for (int u = 0; u < TL::kUnits; ++u) {
        const int m = min(m0 + 8 * (wv * TL::kUnits + u) + (lane >> 3), g.M - 1);
        fd.x[u] = g.a + (size_t)m * g.lda + (size_t)s0 * kFp8Group + 16 * chunk_of_lane(lane);
    }
    f32x4_t acc[RA][NTB];
    tile_loop<kDense, RA, NTB, NW, RW, RX, kWRows, EXACT, TAIL>(
        fd, mine, nst, min(nst, g.G - s0), g.K - s0 * kFp8Group, wv, lane, KG > 1 ? wv * 64 + lane : threadIdx.x,
        [&](int t) { return g.a_scale + (size_t)min(m0 + t, g.M - 1) * g.G + s0; },
        [&](int b) { return g.w_scale + (size_t)(min(n0 + 128 * b, g.N - 1) / 128) * g.G + s0; }, acc);
    // the rings are free: every wave has left them
    if constexpr (KG > 1) {
        static_assert(KG == 2 && NW * RA * NTB * 1024 <= RX * TL::kStage + RW * TL::kWBytes, "the second group's sums");
        float4* sums = (float4*)(smem + TL::group_lds(g.G)) + (size_t)wv * RA * NTB * 64 + lane;
        if (kg == 1) {
#pragma unroll
            for (int i = 0; i < RA; ++i)
#pragma unroll
                for (int j = 0; j < NTB; ++j)
                    sums[(i * NTB + j) * 64] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
        __syncthreads();
        if (kg == 1) return;
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int j = 0; j < NTB; ++j) {
                const float4 t = sums[(i * NTB + j) * 64];
                acc[i][j][0] += t.x, acc[i][j][1] += t.y, acc[i][j][2] += t.z, acc[i][j][3] += t.w;
            }
    }
    static_assert(NW * 8192 <= RX * TL::kStage + RW * TL::kWBytes, "the waves' 8 KB");
    uint8_t* area = smem + wv * 8192;
    auto row = [&](int t) __attribute__((always_inline)) {
        return m0 + t < g.M ? (OutT*)g.c + (size_t)(m0 + t) * g.ldc + nrow : nullptr;
    };
    store_rows<OutT>(acc, area, lane, g.N - nrow, g.c_vec, row);
}

template <int RA, int NTB, int NW, int RW, int RX, int KG, bool EXACT>
moe_status launch_gemm(const GemmFp8& g, hipStream_t st) {
    using TL = GemmTile<RA, NTB, NW, RW, RX, KG>;
    const bool tail = g.K % 128 != 0 || g.G % KG != 0;
    auto kern = tail ? gemm_fp8_tile_kernel<RA, NTB, NW, RW, RX, KG, EXACT, true>
                     : gemm_fp8_tile_kernel<RA, NTB, NW, RW, RX, KG, EXACT, false>;
    const int lds = TL::gemm_lds(g.G);
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    const dim3 grid((unsigned)blocks_of(g.N, TL::kMT), (unsigned)blocks_of(g.M, TL::kNT));
    // weight rows x tokens x groups of waves, steps that the weights are ahead: a profile tells the tiles apart
    static const std::string name = "gemm_fp8_tile_" + std::to_string(TL::kMT) + "x" + std::to_string(TL::kNT) + "x" +
                                    std::to_string(KG) + "_" + std::to_string(RW);
    ProfScope p(name.c_str(), st);
    kern<<<grid, NW * KG * 64, lds, st>>>(g);
    return check_launch(name.c_str());
}

// ---- the routed experts' projections ------------------------------------------------------------------
__device__ __forceinline__ int64_t ceil_of(int64_t n, int block) { return (n + block - 1) / block; }

// The call's experts in LDS, for up to kTableExperts (more are read from memory): a tile's item is then found in some
// hundred cycles, where loads wait behind the stores of the tile before and a scan over the counts takes 1.4 us.
constexpr int kTableExperts = 256;
struct Table {
    int32_t count[kTableExperts], slot[kTableExperts], row[kTableExperts];  // row: the first sorted one
    int32_t end[kTableExperts];  // chunks of the pass's experts up to and with this one
};

// every lane: inclusive sum over the lanes up to it
__device__ __forceinline__ int lanes_sum(int v, int lane) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const int o = __shfl_up(v, s, 64);
        if (lane >= s) v += o;
    }
    return v;
}

__device__ __forceinline__ void fill_table(const FfnArgs& a, Table& tb) {
    if (a.E > kTableExperts) return;
    for (int e = threadIdx.x; e < kTableExperts; e += blockDim.x) {
        tb.count[e] = e < a.E ? a.counts[e] : 0;
        tb.slot[e] = e < a.E ? a.slot_of_expert[e] : 0;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int e = 4 * threadIdx.x;
        const int4 c = *(const int4*)&tb.count[e];
        const int first = lanes_sum(c.x + c.y + c.z + c.w, threadIdx.x) - (c.x + c.y + c.z + c.w);
        *(int4*)&tb.row[e] = make_int4(first, first + c.x, first + c.x + c.y, first + c.x + c.y + c.z);
    }
    __syncthreads();
}

// The chunks of nt tokens of the experts that hold n_lo to n_hi, the shared one's last (every lane gets the sum); with
// `pass`, the table's ends for them too.
__device__ __forceinline__ int count_chunks(const FfnArgs& a, Table& tb, int nt, int n_lo, int n_hi, bool pass) {
    auto chunks = [&](int n) { return n >= n_lo && n <= n_hi ? (n + nt - 1) / nt : 0; };
    const int lane = threadIdx.x & 63, shared = a.shared_w ? chunks(a.T) : 0;
    if (a.E > kTableExperts) {
        int c = 0;
        for (int e = lane; e < a.E; e += 64) c += chunks(a.counts[e]);
        return __shfl(lanes_sum(c, lane), 63, 64) + shared;
    }
    const int4 n = *(const int4*)&tb.count[4 * lane];
    const int c0 = chunks(n.x), c1 = c0 + chunks(n.y), c2 = c1 + chunks(n.z), c3 = c2 + chunks(n.w);
    const int last = lanes_sum(c3, lane), first = last - c3;
    if (pass) {
        __syncthreads();  // nobody reads the ends of the pass before any more
        if (threadIdx.x < 64) *(int4*)&tb.end[4 * lane] = make_int4(first + c0, first + c1, first + c2, last);
        __syncthreads();
    }
    return __builtin_amdgcn_readfirstlane(__shfl(last, 63, 64)) + shared;
}

// Work item `item` of the pass (it exists): as find_item
__device__ __forceinline__ void find_in_table(const FfnArgs& a, const Table& tb, int nt, int item, int& e, int& chunk,
                                              int& slot, int& n, int& p0) {
    const int4 end = *(const int4*)&tb.end[4 * (threadIdx.x & 63)];
    // the ends do not fall: as many experts end before the item as come before its own
    const int at = __popcll(__ballot(end.x <= item)) + __popcll(__ballot(end.y <= item)) +
                   __popcll(__ballot(end.z <= item)) + __popcll(__ballot(end.w <= item));
    if (at >= kTableExperts) {
        e = slot = -1;
        n = a.T;
        p0 = a.T * a.k;
        chunk = item - __builtin_amdgcn_readfirstlane(tb.end[kTableExperts - 1]);
        return;
    }
    e = at;
    slot = __builtin_amdgcn_readfirstlane(tb.slot[at]);
    n = __builtin_amdgcn_readfirstlane(tb.count[at]);
    p0 = __builtin_amdgcn_readfirstlane(tb.row[at]);
    chunk = item - (__builtin_amdgcn_readfirstlane(tb.end[at]) - (n + nt - 1) / nt);
}

// This workgroup's tiles of the experts that hold n_lo to n_hi tokens (chunks: their chunks of kNT).  Workgroup
// i runs on XCD i mod 8; each XCD takes a run of consecutive tiles, so that the tiles that read the same
// weights or the same tokens share an L2 (both projections with e4m3 sums, 2048 tokens, 8 of 128 experts of 2048 x 768:
// 254 -> 236 us against tiles dealt out in turn, 8192 on 7 of 4096 x 2048: 1597 -> 1526).
template <int MODE, bool EXACT, int RA, int NTB, int NW, int RW, int RX>
__device__ __forceinline__ void ffn_tiles(Tile8<RA, NTB, NW, RW, RX>, const FfnFp8& p, const Table& tb, uint8_t* smem, int n_lo, int n_hi, int chunks, int first) {
    using TL = Tile8<RA, NTB, NW, RW, RX>;
    static_assert(MODE != kGateUp || (RA % 2 == 0 && TL::kMT % 256 == 0), "gate/up tiles hold whole groups of h");
    static_assert(MODE != kGateUp || EXACT, "h from binary32 sums");
    const FfnArgs& a = p.a;
    const int nblk = MODE == kGateUp ? 2 * (a.f / 16) : a.d / 16;
    const int gx = (nblk + NW * RA - 1) / (NW * RA);  // tiles over the weight rows
    const int64_t n = (int64_t)chunks * gx, per = ceil_of(n, kXCDs);
    for (int64_t at = first / kXCDs; at < per; at += gridDim.x / kXCDs) {
        const int64_t id = (first % kXCDs) * per + at;
        if (id >= n) return;
        // The empty asm statements make these values new in each pass: otherwise everything that depends on
        // them alone is computed before the loop and held in registers across it, which spills.
        int tid = threadIdx.x, K = MODE == kGateUp ? a.d : a.f;
        asm volatile("" : "+v"(tid), "+s"(K));
        const int lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), G = K / 128;
        const int bx = (int)(id % gx);
        int e, chunk, slot, n_all, p0;
        if (a.E <= kTableExperts) find_in_table(a, tb, TL::kNT, (int)(id / gx), e, chunk, slot, n_all, p0);
        else if (!find_item(a, TL::kNT, (int)(id / gx), e, chunk, slot, n_all, p0, n_lo, n_hi)) return;
        const bool shared = e == -1;
        const int nt = min(TL::kNT, n_all - chunk * TL::kNT);
        p0 += chunk * TL::kNT;  // first row of the tile
        const uint8_t* base;
        if (shared) {
            base = a.shared_w;
        } else {
            if (slot == MOE_SLOT_ELSEWHERE) continue;  // rows produced elsewhere: leave them
            if (slot < 0 || slot >= a.n_slots) {     // absent: flagged, zero rows (h is not read then)
                if (tid == 0) *a.status = 1;
                if (MODE == kDown)
                    for (int i = tid; i < nt * TL::kMT; i += NW * 64) {
                        const int c = bx * TL::kMT + i % TL::kMT;
                        if (c < a.d) store_y(a, (size_t)(p0 + i / TL::kMT), c, 0.f);
                    }
                continue;
            }
            base = a.pool + (size_t)slot * a.stride;
        }
        // d and f are multiples of 128, a wave's rows of 64 at most: all of them exist, or none (then the
        // wave repeats the last block's loads and stores nothing)
        const int b0 = (bx * NW + wv) * RA;
        const size_t rbb = rowblock_bytes(K, MOE_FP8_B128);
        Feed<RA, TL::kUnits, kWFrags> fd;
        const int bw = bx * NW * RA;
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
        f32x4_t acc[RA][NTB];
        tile_loop<MODE, RA, NTB, NW, RW, RX, kWFrags, EXACT, false>(
            fd, smem, G, G, K, wv, lane, tid, [&](int t) { return x_scale + (size_t)source(t) * G; },
            [&](int s) {
                // gate/up: the gate and the up scale of each 128 columns of h (16 blocks); down: of 8 blocks
                const int b = min(bw + (MODE == kGateUp ? 16 * (s >> 1) + (s & 1) : 8 * s),
                                  nblk - 2 + (MODE == kGateUp ? (s & 1) : 1));
                return (const float*)(fd.w + (size_t)(b - bw) * rbb + (size_t)16 * K);
            },
            acc);
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
            // h in 8 bits, all of the tile's columns of a token side by side in LDS (16-byte chunk c at c ^ (t mod 16)),
            // then out in whole pieces of rows
            constexpr int COLS = TL::kMT / 2, CH = COLS / 16;
            static_assert((NW + COLS / 4) * TL::kNT * 4 <= RX * TL::kStage + RW * TL::kWBytes, "magnitudes and h");
            uint8_t* tile = smem + NW * TL::kNT * 4;
            const int cw = wv * RA * 8;  // this wave's first column of the tile
#pragma unroll
            for (int j = 0; j < NTB; ++j) {
                const int t = 16 * j + (lane & 15);
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < GW; ++w) m = umax(m, mags[(wv / GW * GW + w) * TL::kNT + t]);
                const float s = fp8_scale(m), r = 1.0f / s;
#pragma unroll
                for (int i = 0; i < RA / 2; ++i)
                    *(uint32_t*)(tile + t * COLS + ((((cw >> 4) + i) ^ (t & (CH - 1))) << 4) + 4 * quad) =
                        fp8_pack4(acc[2 * i][j][0], acc[2 * i][j][1], acc[2 * i][j][2], acc[2 * i][j][3], r);
                const int c = bx * COLS + cw;
                if (wv % GW == 0 && quad == 0 && t < nt && c < a.f) p.h_scale[(size_t)(p0 + t) * (a.f / 128) + c / 128] = s;
            }
            __syncthreads();
            for (int i = tid; i < nt * CH; i += NW * 64) {
                const int t = i / CH, c = i % CH, col = bx * COLS + 16 * c;
                if (col < a.f)
                    *(u32x4_t*)(p.h8 + (size_t)(p0 + t) * a.f + col) = *(const u32x4_t*)(tile + t * COLS + ((c ^ (t & (CH - 1))) << 4));
            }
        } else if (b0 < nblk) {
            static_assert(NW * 8192 <= RX * TL::kStage + RW * TL::kWBytes, "the waves' 8 KB");
            uint8_t* area = smem + wv * 8192;
            auto rows = [&](auto* y) __attribute__((always_inline)) {
                typedef std::remove_pointer_t<decltype(y)> E;
                auto row = [&](int t) __attribute__((always_inline)) {
                    return t < nt ? y + (size_t)(p0 + t) * a.d + b0 * 16 : nullptr;
                };
                store_rows<E>(acc, area, lane, RA * 16, true, row);
            };
            if constexpr (EXACT) rows((float*)a.y_perm);
            else rows((uint16_t*)a.y_perm);
        }
        __syncthreads();  // the next tile's scales and magnitudes take the same LDS
    }
}

// The tiles of a call.  The gate and up sums are binary32 (EXACT): h is rounded to 8 bits next, and what the e4m3
// instruction drops would move elements across borders between two e4m3 values, whole rows by 1.3e-3 of their norm.
// So are the down projection's where its rows are binary32; bf16 rows take the e4m3 instruction, as the dense product.
//
// EXACT: 512 x 64 or 256 x 64, whichever needs the less time for its rounds over the compute units at a cost of 7 to
// 4.  Measured (us of the gate/up projection, before its exact quotient, which adds 1 to 2 us a tile; 512 x 64 / 256 x 64 /
// 256 x 128): 64 tokens on each of 8 experts of 2048 x 768 34 / 25 / 36, 517 38 / 47 / 40; 4096 x 2048, 128 on each of 7
// 60 / 44 / 63, 8192 1712 / 2162 / 1770; popularity as 1 / rank^1.1, 6 of 256 of 4096 x 2048 and the shared one, 64
// tokens 338 / 367 / 573, 2048 997 / 1164 / 1442, 8192 2196 / 2713 / 2631.  (512 x 128 does not fit the registers: 64 of
// them hold the weights as bf16.)
//
// Else (bf16 rows of the down projection):
// - All experts 256 rows x 64 tokens where each such tile has a compute unit of its own.
// - Else experts with up to kLight tokens take 256 x 64, with the weights two steps ahead (their weights' bytes
//   bound them), and the others 512 x 128 or 256 x 128, whichever needs the less time for its rounds over the
//   compute units at 2.1 and 1.27 us a step (the dense product's costs).  Measured (us, 512 x 128 / 256 x 128 /
//   256 x 64 alone): 128 tokens on each of 7 experts of 4096 x 2048 30 / 22 / 22, 517 62 / 64 / 64, 4096 251 / 313 / 422;
//   8192 by popularity on 6 of 256 725 / 887 / 1080 (750 as chosen), on 8 of 128 of 2048 x 768 178 / 226 / 289 (183).
// HEAVY false: no expert of the call can hold more than kLight, or the larger tiles' scales exceed the LDS
// (inputs beyond 10752).
constexpr int kLight = 64, kMost = 1 << 30, kWaves = 8;
typedef Tile8<4, 8, kWaves, 1, 3> TileLarge;
typedef Tile8<2, 8, kWaves, 2, 3> TileMid;
typedef Tile8<2, 4, kWaves, 2, 4> TileLight;
typedef Tile8<4, 4, kWaves, 1, 3> TileWide;

// The grid is at most one workgroup a compute unit; each takes every gridDim.x-th tile until the work that
// the counts give is through (a launch for the most there could be took 19 to 58 us to find nothing).
template <int MODE, bool EXACT, bool HEAVY>
__global__ __launch_bounds__(kWaves * 64, 2) void ffn_fp8_tile_kernel(FfnFp8 p) {
    extern __shared__ __align__(16) uint8_t lds[];
    Table& tb = *(Table*)lds;
    uint8_t* smem = lds + sizeof(Table);
    fill_table(p.a, tb);
    const int rows = MODE == kGateUp ? 2 * p.a.f : p.a.d;
    if constexpr (EXACT) {
        static_assert(TileWide::kNT == TileLight::kNT, "the same chunks");
        const int chunks = count_chunks(p.a, tb, TileWide::kNT, 0, kMost, true);
        const int64_t wide = ceil_of(chunks * ceil_of(rows, TileWide::kMT), kCUs);
        const int64_t light = ceil_of(chunks * ceil_of(rows, TileLight::kMT), kCUs);
        if (7 * wide < 4 * light) ffn_tiles<MODE, true>(TileWide{}, p, tb, smem, 0, kMost, chunks, blockIdx.x);
        else ffn_tiles<MODE, true>(TileLight{}, p, tb, smem, 0, kMost, chunks, blockIdx.x);
    } else {
        int first = blockIdx.x, light = kMost;  // the 256 x 64 tiles take experts with up to `light` tokens
        if (HEAVY && (int64_t)count_chunks(p.a, tb, TileLight::kNT, 0, kMost, false) * ceil_of(rows, TileLight::kMT) > kCUs) {
            light = kLight;
            const int chunks = count_chunks(p.a, tb, TileLarge::kNT, kLight + 1, kMost, true);
            int64_t tiles = (int64_t)chunks * ceil_of(rows, TileLarge::kMT);
            const int64_t mid = (int64_t)chunks * ceil_of(rows, TileMid::kMT);
            if ((float)ceil_of(tiles, kCUs) * 2.1f < (float)ceil_of(mid, kCUs) * 1.27f) {
                ffn_tiles<MODE, false>(TileLarge{}, p, tb, smem, kLight + 1, kMost, chunks, first);
            } else {
                ffn_tiles<MODE, false>(TileMid{}, p, tb, smem, kLight + 1, kMost, chunks, first);
                tiles = mid;
            }
            // the light tiles begin with the workgroup, of the same XCD, that the heavy ones' last round did not reach
            first = (int)((blockIdx.x + gridDim.x - (int64_t)ceil_of(tiles, kXCDs) * kXCDs % gridDim.x) % gridDim.x);
        }
        const int chunks = count_chunks(p.a, tb, TileLight::kNT, 0, light, true);
        ffn_tiles<MODE, false>(TileLight{}, p, tb, smem, 0, light, chunks, first);
    }
}

template <int MODE, bool EXACT, bool HEAVY>
moe_status launch_ffn(const FfnFp8& p, hipStream_t st, const char* name) {
    const int G = (MODE == kGateUp ? p.a.d : p.a.f) / 128, rows = MODE == kGateUp ? 2 * p.a.f : p.a.d;
    int lds = TileLight::lds(G);
    if (EXACT) lds = std::max(lds, TileWide::lds(G));
    if (HEAVY) lds = std::max(lds, std::max(TileLarge::lds(G), TileMid::lds(G)));
    lds += (int)sizeof(Table);
    auto kern = ffn_fp8_tile_kernel<MODE, EXACT, HEAVY>;
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    const int64_t tiles = work_items(p.a, TileLight::kNT) * ((rows + TileLight::kMT - 1) / TileLight::kMT);
    ProfScope sc(name, st);
    kern<<<(unsigned)std::min<int64_t>(blocks_of(tiles, kXCDs) * kXCDs, kCUs), kWaves * 64, lds, st>>>(p);
    return check_launch(name);
}

}  // namespace

// The tiles, and what a 128-input step of one costs (us): alone on a compute unit, and where every unit
// has a full share of them.  A product's time follows as 3 us + steps * max(alone, rounds * full), to within 15 %
// over 64 to 8192 rows and 512 to 8192 columns of row-major matrices whose rows are whole cache lines.
// Large tiles read less from LDS a product, small ones fill the chip with fewer rows, and two groups that share
// a tile's steps fill it with fewer still.  Measured, us, rows x N x K, one tile against the next:
// 512 x 2048 x 4096 64x64 in two groups 12.7, in one 16.0; 1000 x 2048 x 4096 128x64 in two groups 17.2, in one
// 19.6, 64x64 in two groups 19.1 (one step ahead: two workgroups a unit) or 23.0; 1000 x 4096 x 2048 256x64 15.8,
// 128x64 17.1; 2048 x 4096 x 2048 256x128 25.3, 256x64 28.2; 8192 x 4096 x 4096 512x128 131, 256x128 164.
namespace {
struct TileCost {
    int mt, nt, groups;
    float alone, full;
    int (*lds)(int G);
    moe_status (*launch)(const GemmFp8&, hipStream_t);
};
template <int RA, int NTB, int NW, int RW, int RX, int KG, bool EXACT>
constexpr TileCost cost(float alone, float full) {
    using TL = GemmTile<RA, NTB, NW, RW, RX, KG>;
    return {TL::kMT, TL::kNT, KG, alone, full, TL::gemm_lds, launch_gemm<RA, NTB, NW, RW, RX, KG, EXACT>};
}
constexpr TileCost kTiles[] = {
    cost<4, 8, 8, 1, 3, 1, false>(1.70f, 2.10f), cost<2, 8, 8, 2, 3, 1, false>(0.95f, 1.27f),
    cost<2, 4, 8, 2, 4, 1, false>(0.66f, 0.77f), cost<2, 4, 4, 2, 4, 1, false>(0.49f, 0.40f),
    cost<1, 4, 4, 2, 4, 1, false>(0.39f, 0.27f), cost<2, 4, 4, 2, 4, 2, false>(0.82f, 0.90f),
    cost<1, 4, 4, 2, 4, 2, false>(0.57f, 0.65f), cost<1, 4, 4, 1, 3, 2, false>(0.68f, 0.50f)};
// (binary32 results of 8192 x 4096 x 4096 278 to 325 us: every wave widens every token block of its tile for itself)
constexpr TileCost kExactTiles[] = {
    cost<2, 8, 8, 1, 4, 1, true>(1.70f, 2.10f), cost<2, 4, 4, 3, 5, 1, true>(0.72f, 0.78f),
    cost<1, 4, 4, 3, 5, 1, true>(0.61f, 0.45f), cost<1, 4, 4, 2, 4, 2, true>(0.88f, 0.95f)};
}  // namespace

const void* gemm_fp8_best_tile(const GemmFp8& g, float& us) {
    const TileCost* best = nullptr;
    us = 0.f;
    if (g.ldw > (1u << 22)) return nullptr;  // a tile's weight offsets have 32 bits
    auto look = [&](const TileCost& t) {
        const int64_t rows = blocks_of(g.M, t.nt), tiles = blocks_of(g.N, t.mt) * rows;
        if (t.lds(g.G) > kLds || rows > 65535) return;
        const float rounds = (float)((tiles + kCUs - 1) / kCUs);
        const float e = 3.0f + (float)blocks_of(g.G, t.groups) * std::max(t.alone, rounds * t.full);
        if (!best || e < us) best = &t, us = e;
    };
    if (g.c_bf16)
        for (const TileCost& t : kTiles) look(t);
    else
        for (const TileCost& t : kExactTiles) look(t);
    return best;
}

moe_status gemm_fp8_tile(const GemmFp8& g, const void* tile, hipStream_t st) {
    return ((const TileCost*)tile)->launch(g, st);
}

moe_status ffn_fp8_tile(const FfnFp8& p, int mode, hipStream_t st) {
    if (mode == kGateUp) return launch_ffn<kGateUp, true, false>(p, st, "ffn_fp8_gateup_tile");
    if (!p.a.y_bf16) return launch_ffn<kDown, true, false>(p, st, "ffn_fp8_down_tile");
    const int G = p.a.f / 128;
    const bool heavy = p.a.T > kLight && (int)sizeof(Table) + TileLarge::lds(G) <= kLds && (int)sizeof(Table) + TileMid::lds(G) <= kLds;
    return heavy ? launch_ffn<kDown, false, true>(p, st, "ffn_fp8_down_tile")
                 : launch_ffn<kDown, false, false>(p, st, "ffn_fp8_down_tile");
}

}  // namespace moe
