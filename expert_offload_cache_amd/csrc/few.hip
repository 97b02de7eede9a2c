// moe_layer_few: a whole MoE layer for at most kFewTok tokens in two launches.
//
//   logits = x Wr^T + bias;  S = the k largest;  g = softmax over S;
//   h_e = silu(x Wg_e^T) * (x Wu_e^T);  y = sum_{e in S} g_e (h_e Wd_e^T)  (+ the shared expert)
//
// Launch 1 (few_prepare_kernel): the logits in the fixed order of moe_route, for 8-bit weights the
// quantised rows of x, and the marks and counters that launch 2 starts from.
// Launch 2 (few_layer_kernel): every workgroup selects the experts for itself from the logits (T * E
// numbers), then the workgroups take work items in order: first all gate/up items (one expert, 16
// columns of h, all of its tokens), then the down items (16 or 64 columns of y over a run of the call's experts,
// all tokens; the last run's workgroup adds the others' sums).
// With at most 16 tokens the tokens are one operand block of the matrix instructions, so an expert's
// weights are read once and its tokens need no gathering: columns of tokens that did not choose it are left out of
// the sums.  A down item holds binary32 sums, so the gates are applied in registers and no rows are written between.
//
// What bounds it: the weights' bytes from 16 tokens on (2048 x 768, 8 of 128, bf16: 355 MB in 74 us, 4.8 TB/s; 4 bits,
// 4096 x 2048, 6 of 256 + shared: 570 MB in 138 us); for one token latency (76 MB in 29 us: launch 1 takes 5, the selection
// 3.5, the first weights land 15 after the start, the join of y takes 2).
//
// The hand-over of h.  A down item needs h of every expert, which other workgroups write in the same
// launch.  Launch 1 fills h with a mark (all bits set, which is a NaN that h never holds: a NaN
// result of those bits is stored as another NaN).  h is written and read with device-scope accesses of
// whole words, and a reader that finds the mark reads again: each word is its own flag.
// Why every wait ends.  There are two: for h, and of the workgroup of run 0 of a row block for the other runs' sums
// of y (store_y).  Items are handed out by counters to workgroups that run, each when it asks; nobody waits for an item
// that is not handed out:
//  - Gate/up items wait for nothing, and a workgroup gets a down item only after all of them have been handed out.  So
//    every wait for h ends.
//  - The runs of a row block lie in one list, run 0 last (few_order.h), so run 0 waits for items handed out before it.  A
//    workgroup asks for its next item before it has finished the one at hand, so an item may be held by a workgroup that
//    waits first: then with a run 0 that was handed out to it before the item.  Whoever follows such a chain of waits
//    goes back in the order of hand-out at each step, so the chain closes no circle and ends with somebody who works.
// Neither needs all workgroups to be resident, nor any order among those that are.  (A second call that uses the same
// workspace at the same time breaks both; then a wait ends at its limit and the status word is set to 2.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "few_order.h"
#include "ffn_common.h"
#include "fp8.h"
#include "route_logit.h"
#include "select_permute.h"
#include "slot_layout.h"

namespace moe {
namespace {

constexpr int kFewTok = MOE_FEW_TOKENS;    // most tokens: one operand block of the matrix instructions
constexpr int kFewK = MOE_FEW_TOPK;        // most experts a token
constexpr int kFewRows = kFewTok * kFewK;  // most (token, expert) pairs
constexpr int kWaves = kFewWaves;
constexpr int kThreads = 64 * kWaves;
constexpr int kListStride = 64;            // words from a counter to the next
constexpr uint32_t kMark = 0xFFFFFFFFu;    // a word of h that is not written yet
constexpr int kEarlyGates = 4;             // most tokens whose gates are formed before the first products
constexpr int kSpinLimit = 1 << 20;        // reads of a word that stays marked, some 300 ns each

struct FewArgs {
    const void* x;  // [T, d]
    int T, d, f, E, k;
    const void* w_router;
    const float* bias;
    const int32_t* forced;
    const int32_t* slot_of_expert;
    int n_slots;
    const uint8_t* pool;
    size_t stride;
    const uint8_t* shared_w;
    int32_t* topk_idx;
    float* topk_w;
    void* y;
    // workspace
    int32_t* status;
    uint32_t* lists;  // [2][kLists][kListStride]: gate/up and down items handed out
    float* logits;    // [T, E]
    uint16_t* xq;     // fp8: the e4m3 values of the rows of x as bf16 [T, d] (exact)
    float* xs;        // their scales [T, d / 128]
    uint32_t* h;      // [T * k (+ T), f] bf16 (binary32 for F32 and fp8)
    uint32_t* part;   // [splits - 1][T, d] binary32: y's sums over the runs but the first
    size_t h_bytes, marks;  // bytes of h; words of h and part
    int splits;
    int piece, rows_fit, h_area;  // chunks of a row of h in LDS at a time, rows that fit, bytes they take
    int items_most, choice_area;  // most items a call of this shape may have; bytes of their Choice
};

// ---- launch 1 ---------------------------------------------------------------------------------------
// A wave takes one expert and TB tokens; lane j owns segment j of the rows (route_logit.h).
template <bool kBf16, int TB>
__global__ __launch_bounds__(256) void few_prepare_kernel(FewArgs a, int logit_blocks, int quant_blocks) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    if ((int)blockIdx.x < logit_blocks) {
        const int ntt = (a.T + TB - 1) / TB;
        const int g = blockIdx.x * 4 + wv;
        if (g >= ntt * a.E) return;
        const int t0 = g / a.E * TB, e = g - g / a.E * a.E;
        float acc[TB];
        logit_segments<kBf16, TB>(a.x, a.w_router, a.T, a.d, t0, e, lane, acc);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const float v = wave_tree_sum(acc[i]);
            if (lane == 0 && t0 + i < a.T) a.logits[(size_t)(t0 + i) * a.E + e] = a.bias ? v + a.bias[e] : v;
        }
        return;
    }
    const int b = blockIdx.x - logit_blocks;
    if (b < quant_blocks) {  // a wave takes one group of 128 inputs of one row
        const int G = a.d / kFp8Group, g = b * 4 + wv;
        if (g >= a.T * G) return;
        const uint32_t v = ((const uint32_t*)a.x)[(size_t)g * 64 + lane];
        const float v0 = bf16_lo(v), v1 = bf16_hi(v);
        uint32_t m = quarter_max(row16_max(umax(abs_bits(v0), abs_bits(v1))));
        const float s = fp8_scale(m);
        const uint32_t q = fp8_pack4(v0, v1, 0.f, 0.f, 1.0f / s);
        const bf16v2_t w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, 1.0f, false);
        ((uint32_t*)a.xq)[(size_t)g * 64 + lane] = __builtin_bit_cast(uint32_t, w);
        if (lane == 0) a.xs[g] = s;
        return;
    }
    const size_t i0 = (size_t)(b - quant_blocks) * 256 + threadIdx.x, n = (size_t)(gridDim.x - logit_blocks - quant_blocks) * 256;
    for (size_t i = i0; i < a.marks / 4; i += n) ((u32x4_t*)a.h)[i] = u32x4_t{kMark, kMark, kMark, kMark};
    if (i0 < 2 * kLists * kListStride) a.lists[i0] = 0;
}

// ---- launch 2: operands ------------------------------------------------------------------------------
template <int W>
struct FewType;  // inputs a step; 16-byte vectors of weights and of activations a lane holds of one
template <>
struct FewType<MOE_F32> {
    static constexpr int kIn = 32, kWV = 2, kXV = 2;
};
template <>
struct FewType<MOE_BF16> {
    static constexpr int kIn = 32, kWV = 1, kXV = 1;
};
template <>
struct FewType<MOE_INT4_G128> {
    static constexpr int kIn = 128, kWV = 1, kXV = 4;
};
template <>
struct FewType<MOE_FP8_B128> {
    static constexpr int kIn = 128, kWV = 2, kXV = 4;
};

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b), c, 0, 0, 0);
}

// byte offset in a row of activations of a lane's vector v of step 0 (q = lane / 16); a step is kIn inputs on
template <int W>
__device__ __forceinline__ int act_offset(int v, int q) {
    if constexpr (W == MOE_F32) return 32 * q + 16 * v;
    if constexpr (W == MOE_BF16) return 16 * q;
    if constexpr (W == MOE_INT4_G128) return 64 * v + 16 * q;
    return 128 * (v >> 1) + 32 * q + 16 * (v & 1);
}
template <int W>
constexpr int act_step() {  // bytes of a row of activations a step takes
    return FewType<W>::kIn * (W == MOE_F32 ? 4 : 2);
}

// The sum of the activations of a step (int4 only: nibbles enter as 128 + u, the weight is u - 8)
template <int W>
__device__ __forceinline__ f32x4_t act_sum(const u32x4_t (&x)[FewType<W>::kXV]) {
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    if constexpr (W == MOE_INT4_G128) {
        const u32x4_t ones = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
        for (int v = 0; v < 4; ++v) s = mfma_bf16(x[v], ones, s);
    }
    return s;
}

// acc += 16 weight rows x 16 tokens over one step.  Result: token l % 16, rows 4 (l / 16) .. + 3; for int4
// row l % 16, tokens 4 (l / 16) .. + 3, so that a lane needs one scale.
// scale: int4: of this lane's row and group; fp8: of the step times the token's.
template <int W>
__device__ __forceinline__ void step_product(f32x4_t& acc, const u32x4_t (&w)[FewType<W>::kWV], const u32x4_t (&x)[FewType<W>::kXV],
                                             float scale, f32x4_t xsum) {
    if constexpr (W == MOE_BF16) {
        acc = mfma_bf16(w[0], x[0], acc);
    } else if constexpr (W == MOE_F32) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f32(w[v][i]), as_f32(x[v][i]), acc, 0, 0, 0);
    } else if constexpr (W == MOE_INT4_G128) {
        f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            uint32_t wb[4];
            int4_word_to_bf16(w[0][v], wb);
            p = mfma_bf16(x[v], u32x4_t{wb[0], wb[1], wb[2], wb[3]}, p);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(scale, __builtin_fmaf(-136.0f, xsum[i], p[i]), acc[i]);
    } else {
        f32x4_t p = {0.f, 0.f, 0.f, 0.f};
        const Wide8 ww = widen(join8(w[0], w[1]));
#pragma unroll
        for (int v = 0; v < 4; ++v)
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww.v[v], __builtin_bit_cast(bf16v8_t, x[v]), p, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(scale, p[i], acc[i]);
    }
}

// where (row, token) of a lane's accumulator element i lies
template <int W>
__device__ __forceinline__ int acc_row(int lane, int i) {
    return W == MOE_INT4_G128 ? lane & 15 : 4 * (lane >> 4) + i;
}
template <int W>
__device__ __forceinline__ int acc_token(int lane, int i) {
    return W == MOE_INT4_G128 ? 4 * (lane >> 4) + i : lane & 15;
}

// ---- launch 2: the call's experts, in LDS ---------------------------------------------------------------
constexpr int kMaxItems = kFewRows + 1;
struct FewTable {
    int n_items;                    // experts whose weights are read, in the order in which the pairs name them; the shared one last
    int next;                       // the workgroup's next item of work
    int taken[kWaves];              // items and (above bit 16) rows that a wave's pairs bring in
    int slot[kMaxItems];            // -1: the shared expert
    uint16_t tokens[kMaxItems];     // the tokens that chose it, a bit each
    uint16_t row0[kMaxItems + 1];   // its first row of h: a row a token, in ascending order
    uint16_t place_of[kFewRows];    // pair -> item * 16 + token, or kOff
    uint32_t chosen[kPermMaxE];     // expert -> tokens, a bit each
    int16_t item_of[kPermMaxE];     // expert -> item, or -1
    int slot_of[kPermMaxE];         // expert -> slot
    int16_t sel[kFewRows];          // [T][k]
    float val[kFewRows];            // the logits chosen
};

// Beside it, for each item and token: the token's row of h, or kOff, and its gate, or -0 where it did not choose the expert
// (gates are never -0); after the last item one that nobody chose.
constexpr uint32_t kOff = 0xFFFFu;
struct Choice {
    uint16_t* row;  // [items + 1][16]
    float* gate;    // [items + 1][16]
};
__device__ __forceinline__ bool is_off(float gate) { return as_u32(gate) == 0x80000000u; }
constexpr int choice_bytes(int items) { return (items + 1) * kFewTok * 6; }

// binary32 -> an integer of the same order; NaN below everything
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = as_u32(v == 0.f ? 0.f : v);
    if (v != v) return 1u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}
// largest value of the wave's lanes
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v))));  // as row16_max
    return umax(umax(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
                umax(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// One wave selects the experts of TT tokens (t, t + kWaves; the last one again past the end): k rounds of the
// largest logit left (equal ones: the lowest id).  NE logits a lane.
template <int NE, int TT>
__device__ __forceinline__ void few_select(const FewArgs& a, int t0, FewTable& tb) {
    const int lane = threadIdx.x & 63;
    float v[TT][NE], val[TT];
    uint32_t key[TT][NE];
    int t[TT], sel[TT];
#pragma unroll
    for (int u = 0; u < TT; ++u) {
        t[u] = min(t0 + u * kWaves, a.T - 1);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[u][i] = lane + 64 * i < a.E ? a.logits[(size_t)t[u] * a.E + lane + 64 * i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < TT; ++u) {
        sel[u] = 0;
        val[u] = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) key[u][i] = lane + 64 * i < a.E ? order_key(v[u][i]) : 0u;
    }
    for (int r = 0; r < a.k; ++r) {
        uint32_t best[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            best[u] = key[u][0];
#pragma unroll
            for (int i = 1; i < NE; ++i) best[u] = umax(best[u], key[u][i]);
        }
#pragma unroll
        for (int u = 0; u < TT; ++u) best[u] = wave_max_u32(best[u]);
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            int id = -1;
            float won = 0.f;
#pragma unroll
            for (int i = NE - 1; i >= 0; --i) {
                const uint64_t at = __ballot(key[u][i] == best[u]);
                id = at ? 64 * i + (int)__builtin_ctzll(at) : id;
                won = at ? v[u][i] : won;
            }
            won = as_f32(__builtin_amdgcn_readlane(as_u32(won), id & 63));
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 64 * i == id) key[u][i] = 0;
            sel[u] = lane == r ? id : sel[u];
            val[u] = lane == r ? won : val[u];
        }
    }
#pragma unroll
    for (int u = 0; u < TT; ++u)
        if (lane < a.k) {
            tb.sel[t[u] * a.k + lane] = (int16_t)sel[u];
            tb.val[t[u] * a.k + lane] = val[u];
        }
}
template <int NE>
__device__ __forceinline__ void few_select_all(const FewArgs& a, int wv, FewTable& tb) {
    if (wv + kWaves < a.T) few_select<NE, 2>(a, wv, tb);
    else if (wv < a.T) few_select<NE, 1>(a, wv, tb);
}

// The experts of the call.  known(n): run by every wave when their number is known, before the workgroup meets last.
template <typename Known>
__device__ __forceinline__ void few_table(const FewArgs& a, FewTable& tb, Choice ch, Known&& known) {
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.k;
    for (int e = tid; e < a.E; e += kThreads) {
        tb.chosen[e] = 0;
        tb.item_of[e] = -1;
        tb.slot_of[e] = a.slot_of_expert[e];
    }
    for (int i = tid; i < (a.items_most + 1) * kFewTok; i += kThreads) {
        ch.row[i] = (uint16_t)kOff;
        ch.gate[i] = -0.f;
    }
    if (a.forced) {
        if (tid < pairs) {
            const int e = min(max(a.forced[tid], 0), a.E - 1);
            tb.sel[tid] = (int16_t)e;
            tb.val[tid] = a.logits[(size_t)(tid / a.k) * a.E + e];
        }
    } else {
        static_assert(kFewTok <= 2 * kWaves, "two tokens a wave");
        if (a.E <= 64) few_select_all<1>(a, wv, tb);
        else if (a.E <= 128) few_select_all<2>(a, wv, tb);
        else if (a.E <= 256) few_select_all<4>(a, wv, tb);
        else few_select_all<16>(a, wv, tb);
    }
    __syncthreads();
    // one thread a pair
    const int t = tid / a.k, j = tid - t * a.k, e = tid < pairs ? tb.sel[tid] : 0;
    const int slot = tid < pairs ? tb.slot_of[e] : 0;
    if (tid < pairs) atomicOr(&tb.chosen[e], 1u << t);
    __syncthreads();
    // the first pair that names an expert brings it in (a token names an expert twice only in forced_idx)
    const uint32_t tokens = tid < pairs ? tb.chosen[e] : 0;
    bool once = tid < pairs;
    if (once && a.forced)
        for (int u = 0; u < j; ++u) once = once && tb.sel[t * a.k + u] != e;
    const bool first = once && __builtin_ctz(tokens | 0x80000000u) == t;
    // an absent expert adds nothing to y; one whose part comes from elsewhere is no error
    const bool there = slot >= 0 && slot < a.n_slots;
    if (first && !there && slot != MOE_SLOT_ELSEWHERE && blockIdx.x == 0) *a.status = 1;
    const int brings = first && there ? 1 | __popc(tokens) << 16 : 0;  // one item and its rows
    int upto = brings;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const int v = __shfl_up(upto, s, 64);
        if (lane >= s) upto += v;
    }
    if (lane == 63) tb.taken[wv] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wv) before = all;
        all += tb.taken[w];
    }
    before += upto - brings;
    if (first && there) {
        const int item = before & 0xFFFF;
        tb.slot[item] = slot;
        tb.tokens[item] = (uint16_t)tokens;
        tb.row0[item] = (uint16_t)(before >> 16);
        tb.item_of[e] = (int16_t)item;
    }
    if (tid < a.T && a.shared_w) {
        ch.row[(all & 0xFFFF) * kFewTok + tid] = (uint16_t)((all >> 16) + tid);
        ch.gate[(all & 0xFFFF) * kFewTok + tid] = 1.0f;
    }
    if (tid == 0) {
        const int n = all & 0xFFFF, rows = all >> 16;
        tb.row0[n] = (uint16_t)rows;
        if (a.shared_w) {
            tb.slot[n] = -1;
            tb.tokens[n] = (uint16_t)((1u << a.T) - 1);
            tb.row0[n + 1] = (uint16_t)(rows + a.T);
        }
        tb.n_items = n + (a.shared_w ? 1 : 0);
    }
    __syncthreads();
    if (tid < pairs) {
        const int item = tb.item_of[e];
        tb.place_of[tid] = (uint16_t)kOff;
        if (once && item >= 0) {
            tb.place_of[tid] = (uint16_t)(item * kFewTok + t);
            ch.row[item * kFewTok + t] = (uint16_t)(tb.row0[item] + __popc(tokens & ((1u << t) - 1)));
        }
    }
    known((all & 0xFFFF) + (a.shared_w ? 1 : 0));
    __syncthreads();
}

// The gates, as moe_route forms them (binary64, one rounding).  An id given twice for a token counts with the sum of
// its gates.
__device__ __forceinline__ void few_gates(const FewArgs& a, FewTable& tb, Choice ch) {
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int t = wv; t < a.T; t += kWaves) {
        const float val = lane < a.k ? tb.val[t * a.k + lane] : 0.f;
        double m = -INFINITY;
        for (int i = 0; i < a.k; ++i) m = fmax(m, (double)as_f32(__builtin_amdgcn_readlane(as_u32(val), i)));
        const double term = lane < a.k ? exp((double)val - m) : 0.0;
        double den = 0.0;
        const uint64_t bits = __builtin_bit_cast(uint64_t, term);
        for (int i = 0; i < a.k; ++i) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, i), hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), i);
            den += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        }
        float g = (float)(term / den);
        if (lane < a.k && blockIdx.x == 0) {
            a.topk_idx[(size_t)t * a.k + lane] = a.forced ? a.forced[(size_t)t * a.k + lane] : tb.sel[t * a.k + lane];
            a.topk_w[(size_t)t * a.k + lane] = g;
        }
        if (a.forced) {
            const int e = lane < a.k ? tb.sel[t * a.k + lane] : -1;
            float sum = 0.f;
            for (int i = 0; i < a.k; ++i) {
                const int ei = __shfl(e, i, 64);
                const float gi = __shfl(g, i, 64);
                if (ei == e) sum += gi;
            }
            g = sum;
        }
        const uint32_t place = lane < a.k ? tb.place_of[t * a.k + lane] : kOff;
        if (place != kOff) ch.gate[place] = g;
    }
    __syncthreads();
}

// The next work item of a kind (one wave): item c + kLists v is the v-th of list c (few_order.h: `total` things, `runs`
// items each).  A workgroup starts with the list of its number and goes on to the others; -1: every list is handed out.
__device__ __forceinline__ uint32_t few_request(uint32_t* lists, int c) {
    uint32_t v = 0;
    if ((threadIdx.x & 63) == 0) v = __hip_atomic_fetch_add(lists + c * kListStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return v;  // lane 0's
}
__device__ __forceinline__ int few_resolve(uint32_t* lists, int total, int runs, int home, uint32_t asked) {
    const int lane = threadIdx.x & 63;
    int c = home;
    for (;;) {
        const uint32_t v = __builtin_amdgcn_readfirstlane(asked);
        if ((int)v < list_items(total, runs, c)) return c + kLists * (int)v;
        // another list that is not handed out yet
        const int o = (home + lane) % kLists;
        const uint32_t seen = lane < kLists ? __hip_atomic_load(lists + o * kListStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
        const uint64_t left = __ballot(lane < kLists && (int)seen < list_items(total, runs, o));
        if (!left) return -1;
        c = (home + __builtin_ctzll(left)) % kLists;
        asked = few_request(lists, c);
    }
}

// What other workgroups of the launch write is read past the caches that they do not write to: sc1, device scope.
typedef __amdgpu_buffer_rsrc_t buffer_t;
constexpr int kDeviceScope = 16;  // cache policy bit sc1
__device__ __forceinline__ u32x4_t load_shared(buffer_t h, uint32_t byte) {
    return __builtin_amdgcn_raw_buffer_load_b128(h, (int)byte, 0, kDeviceScope);
}
__device__ __forceinline__ bool marked(u32x4_t v) { return v.x == kMark || v.y == kMark || v.z == kMark || v.w == kMark; }

// Waits (a wave; lanes with `here` unset have nothing to wait for) until the word at p is written.  False: given up.
__device__ __forceinline__ bool wait_word(const uint32_t* p, bool here) {
    // the last lane's word (the last to be written, mostly); the others are looked at again by the caller
    const uint64_t at = __ballot(here);
    if (!at) return true;
    const bool mine = (int)(threadIdx.x & 63) == 63 - (int)__builtin_clzll(at);
#pragma unroll 1
    for (int spin = 0; spin < kSpinLimit; ++spin) {
        const bool still = mine && __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == kMark;
        if (!__any(still)) return true;
        __builtin_amdgcn_s_sleep(2);
    }
    return false;
}

template <int W>
constexpr bool kWideH = W == MOE_F32 || W == MOE_FP8_B128;  // h in binary32

// 16 weight rows of one step: this lane's vectors
template <int W>
__device__ __forceinline__ void load_weights(u32x4_t (&w)[FewType<W>::kWV], const uint8_t* block, int st, int lane) {
#pragma unroll
    for (int v = 0; v < FewType<W>::kWV; ++v)
        w[v] = __builtin_nontemporal_load((const u32x4_t*)(block + (size_t)st * FewType<W>::kWV * 1024 +
                                                           (W == MOE_F32 ? lane * 32 + v * 16 : v * 1024 + lane * 16)));
}

// ---- launch 2: gate/up ---------------------------------------------------------------------------------
// One item: 16 PB columns of h of one expert, whose gate and up blocks lie one after the other.  The waves split
// the inputs.  The weights come through a ring of R steps a wave that runs on from item to item: a step's registers are
// filled for the next item as soon as its last use in this one is over.  Every path issues the same loads (steps
// past a wave's share repeat its last one, which is at hand), so that waiting for one never waits for the younger ones.
// NS: a wave's rows of x, its share of the inputs, stay in registers for all items, NS steps at most; 0: they are
// read with the weights.
template <int W, int NS, int R, int PB>
struct GateUp {
    using FT = FewType<W>;
    static constexpr bool kHold = NS > 0;
    static constexpr int kM = 2 * PB;  // operand blocks of an item
    static_assert(!kHold || (R <= NS && NS % R == 0), "the ring");
    const FewArgs& a;
    int lane, nst, s0, s1;
    const uint8_t* xrow;
    const float* xscale;
    u32x4_t w[R][kM][FT::kWV], x[kHold ? NS : R][FT::kXV];
    float sx[W == MOE_FP8_B128 ? (kHold ? NS : R) : 1], sw[R][W == MOE_FP8_B128 ? kM : 1];
    u32x4_t scales[2];  // int4: 32 bytes of an item's scales on their way to LDS

    __device__ __forceinline__ GateUp(const FewArgs& args, int wv) : a(args) {
        lane = threadIdx.x & 63;
        nst = a.d / FT::kIn;
        s0 = wv * nst / kWaves;
        s1 = (wv + 1) * nst / kWaves;
        const int t = min(lane & 15, a.T - 1);
        xrow = (W == MOE_FP8_B128 ? (const uint8_t*)a.xq : (const uint8_t*)a.x) + (size_t)t * a.d * (W == MOE_F32 ? 4 : 2);
        xscale = a.xs + (size_t)t * nst;
        if constexpr (kHold)
#pragma unroll
            for (int n = 0; n < NS; ++n) load_x(n, step_of(n));
    }
    // the wave's n-th step, or its last
    __device__ __forceinline__ int step_of(int n) const { return min(min(s0 + n, max(s1 - 1, s0)), nst - 1); }
    __device__ __forceinline__ const uint8_t* blocks_of(const FewTable& tb, int item, int b) const {
        const int slot = __builtin_amdgcn_readfirstlane(tb.slot[item]);
        return (slot < 0 ? a.shared_w : a.pool + (size_t)slot * a.stride) + gu_block_offset(b * PB, 0, a.d, (moe_dtype)W);
    }
    __device__ __forceinline__ void load_x(int n, int st) {
#pragma unroll
        for (int v = 0; v < FT::kXV; ++v)
            x[n][v] = *(const u32x4_t*)(xrow + (size_t)st * act_step<W>() + act_offset<W>(v, lane >> 4));
        if constexpr (W == MOE_FP8_B128) sx[n] = xscale[st];
    }
    __device__ __forceinline__ void load(int r, const uint8_t* base, int n) {
        const int st = step_of(n);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const uint8_t* block = base + m * rowblock_bytes(a.d, (moe_dtype)W);
            load_weights<W>(w[r][m], block, st, lane);
            if constexpr (W == MOE_FP8_B128) sw[r][m] = ((const float*)(block + (size_t)nst * 2048))[st];
        }
        if constexpr (!kHold) load_x(r, st);
    }
    // int4: an item's scales, 2 nst vectors a block, to registers, and to LDS; the workgroup meets before they are read
    __device__ __forceinline__ void load_scales(const uint8_t* base) {
        if constexpr (W == MOE_INT4_G128)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = min((int)threadIdx.x + h * kThreads, kM * 2 * nst - 1), m = i / (2 * nst);
                scales[h] = *(const u32x4_t*)(base + m * rowblock_bytes(a.d, (moe_dtype)W) + (size_t)nst * 1024 + 16 * (i - m * 2 * nst));
            }
    }
    __device__ __forceinline__ void put_scales(uint8_t* area) {
        if constexpr (W == MOE_INT4_G128)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = (int)threadIdx.x + h * kThreads;
                if (i < kM * 2 * nst) *(u32x4_t*)(area + 16 * i) = scales[h];
            }
    }
    // an item's first loads go out
    __device__ __forceinline__ void begin(const uint8_t* base) {
        load_scales(base);
#pragma unroll
        for (int r = 0; r < R; ++r) load(r, base, r);
    }
    __device__ __forceinline__ void one(f32x4_t (&acc)[kM], int r, int xi, int n, const uint16_t* sc) {
        const int st = s0 + n;
        if (st >= s1) return;
        const f32x4_t sum = act_sum<W>(x[xi]);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            float f = 1.f;
            if constexpr (W == MOE_INT4_G128) f = bf16_to_f32(sc[((lane & 15) + 16 * m) * nst + st]);
            if constexpr (W == MOE_FP8_B128) f = sw[r][m] * sx[xi];
            step_product<W>(acc[m], w[r][m], x[xi], f, sum);
        }
    }
    // the item at base; MORE: the one at next is on its way when it returns
    template <bool MORE>
    __device__ __forceinline__ void multiply(f32x4_t (&acc)[kM], const uint8_t* base, const uint8_t* next, const uint8_t* area) {
        const uint16_t* sc = (const uint16_t*)area;
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (MORE) load_scales(next);
        if constexpr (kHold) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                one(acc, n % R, n, n, sc);
                if (n + R < NS) load(n % R, base, n + R);
                else if constexpr (MORE) load(n % R, next, n % R);
            }
        } else {
            const int turns = ((nst + kWaves - 1) / kWaves + R - 1) / R;
            for (int i = 0; i < turns; ++i) {
                const bool last = i + 1 == turns;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    one(acc, r, r, i * R + r, sc);
                    if (!last) load(r, base, (i + 1) * R + r);
                    else if constexpr (MORE) load(r, next, r);
                }
            }
        }
    }
};

// The waves' sums of an item joined, and its columns of h stored.
template <int W, int PB>
__device__ __forceinline__ void store_h(const FewArgs& a, const FewTable& tb, int item, int b, const float* red) {
    const uint32_t tokens = tb.tokens[item];
    const int row0 = tb.row0[item];
    for (int o = threadIdx.x; o < PB * 256; o += kThreads) {
        const int p = o >> 8, i = o & 255, t = i >> 4, r = i & 15;
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            gs += red[((w * PB + p) * 2) * 256 + i];
            us += red[((w * PB + p) * 2 + 1) * 256 + i];
        }
        const float v = silu_mul(gs, us);
        const bool on = (tokens >> t) & 1;
        const size_t at = (size_t)(row0 + __popc(tokens & ((1u << t) - 1))) * a.f + (b * PB + p) * 16 + r;
        if constexpr (kWideH<W>) {
            uint32_t h = as_u32(v);
            if (h == kMark) h = 0x7FFFFFFFu;
            if (on) __hip_atomic_store(a.h + at, h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else {
            uint32_t h = f32_to_bf16(v);
            h |= (uint32_t)__shfl_xor((int)h, 1, 64) << 16;
            if (h == kMark) h = 0x7FFF7FFFu;
            if (on && !(r & 1)) __hip_atomic_store(a.h + at / 2, h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// ---- launch 2: down ------------------------------------------------------------------------------------
// One item: 16 RB columns of y (so that a row of h read from LDS serves RB operand blocks) over one of `splits` runs of the call's (expert, chunk of C steps) pairs.  The run is taken in batches whose rows of h fit the LDS: whole
// experts, or where one expert's rows may not fit, pieces of `piece` chunks of one expert.  The waves split each
// batch's chunks.  The weights of R chunks a wave are on their way before h is waited for, RE of them before the
// workgroup's last gate/up products (what the registers allow).
template <int W, int RB, int C, int R, int RE>
struct Down {
    using FT = FewType<W>;
    static constexpr int HB = FT::kIn * (kWideH<W> ? 4 : 2);  // bytes of a row of h a step takes in memory
    const FewArgs& a;
    const FewTable& tb;
    int lane, wv, nch, c0, c1;  // the item's run
    int b0, b1;                 // the batch's chunks
    int w0, w1;                 // this wave's
    int wn, item_n, ch_n;       // the chunk whose weights are read next: its expert and place there
    size_t block_at;
    u32x4_t w[R][C][RB][FT::kWV];
    uint32_t sw[R][W == MOE_INT4_G128 || W == MOE_FP8_B128 ? C : 1][RB];
    f32x4_t y[RB];

    __device__ __forceinline__ Down(const FewArgs& args, const FewTable& table) : a(args), tb(table) {
        lane = threadIdx.x & 63;
        wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        nch = a.f / FT::kIn / C;
    }
    // where the batch that begins with chunk c ends
    __device__ __forceinline__ int batch_end(int c) {
        if (c >= c1) return c1;
        const int item = c / nch;
        if (a.piece < nch) return min(c1, item * nch + min(nch, ((c - item * nch) / a.piece + 1) * a.piece));
        const int n = tb.n_items, last = min(item + 1 + lane, n);
        const uint64_t fit = __ballot((int)tb.row0[last] - (int)tb.row0[item] <= a.rows_fit);
        // the first expert always fits; row0 does not fall
        return min(c1, (item + (fit == ~0ull ? 64 : (int)__builtin_ctzll(~fit))) * nch);
    }
    // the weights of the next chunk; past the end the last one again
    __device__ __forceinline__ void load_w(int r) {
        const int slot = __builtin_amdgcn_readfirstlane(tb.slot[item_n]);
        const uint8_t* first = (slot < 0 ? a.shared_w : a.pool + (size_t)slot * a.stride) + block_at;
        const int st = ch_n * C, nst = nch * C;
#pragma unroll
        for (int m = 0; m < RB; ++m) {
            const uint8_t* block = first + m * rowblock_bytes(a.f, (moe_dtype)W);
#pragma unroll
            for (int c = 0; c < C; ++c) load_weights<W>(w[r][c][m], block, st + c, lane);
            if constexpr (W == MOE_INT4_G128) {  // of this lane's row, the chunk's steps (one or two)
                const uint8_t* p = block + (size_t)nst * 1024 + ((size_t)(lane & 15) * nst + st) * 2;
                sw[r][0][m] = C == 2 ? *(const uint32_t*)p : *(const uint16_t*)p;
            }
            if constexpr (W == MOE_FP8_B128)
#pragma unroll
                for (int c = 0; c < C; ++c) sw[r][c][m] = ((const uint32_t*)(block + (size_t)nst * 2048))[st + c];
        }
        const bool go = wn + 1 < w1, over = ch_n + 1 == nch;
        wn += go;
        item_n += go && over;
        ch_n = !go ? ch_n : over ? 0 : ch_n + 1;
        __builtin_amdgcn_sched_barrier(0);  // (addresses of one chunk at a time)
    }
    __device__ __forceinline__ float scale_of(int r, int c, int m) const {
        if constexpr (W == MOE_INT4_G128) return c ? bf16_hi(sw[r][0][m]) : bf16_lo(sw[r][0][m]);
        return as_f32(sw[r][c][m]);
    }
    __device__ __forceinline__ void begin_batch(int c) {
        b0 = c;
        b1 = batch_end(c);
        w0 = b0 + wv * (b1 - b0) / kWaves;
        w1 = b0 + (wv + 1) * (b1 - b0) / kWaves;
        wn = w0;
        const int from = max(min(w0, b1 - 1), 0);
        item_n = from / nch;
        ch_n = from - item_n * nch;
    }
    // chunks' weights (a wave without chunks reads one as well)
    template <int FROM, int TO>
    __device__ __forceinline__ void load() {
#pragma unroll
        for (int r = FROM; r < TO; ++r) load_w(r);
    }
    __device__ __forceinline__ void begin(DownItem it) {
        const int64_t all = (int64_t)tb.n_items * nch;
        c0 = (int)(it.run * all / a.splits);
        c1 = (int)((it.run + 1) * all / a.splits);
        block_at = down_block_offset(it.block * RB, a.d, a.f, (moe_dtype)W);
#pragma unroll
        for (int m = 0; m < RB; ++m) y[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        begin_batch(c0);
    }
    // The batch's rows of h to LDS (fp8: quantised, as bf16 values, and their scales), each as soon as it is written.
    __device__ __forceinline__ void stage(uint8_t* hs, float* hscale, bool& lost) {
        const int item0 = b0 / nch, item1 = (b1 - 1) / nch + 1;
        const int row0 = tb.row0[item0], rows = tb.row0[item1] - row0;
        // whole rows, or of one expert the piece that holds the batch
        const int st0 = a.piece < nch ? (b0 - item0 * nch) / a.piece * a.piece * C : 0;
        const int steps = min(a.piece, nch) * C, units = steps * FT::kIn / (W == MOE_F32 ? 4 : 8);
        const uint32_t recip = (uint32_t)(0x100000000ull / (uint32_t)units) + 1;  // exact quotients of numbers below 2^16
        const buffer_t hb = __builtin_amdgcn_make_buffer_rsrc(a.h, 0, (int)a.h_bytes, 0x00027000);
        const bool few = rows * units <= 2 * kThreads;
        int tries = 0;
        constexpr int G = 4, LV = W == MOE_FP8_B128 ? 2 : 1;  // units and 16-byte loads of one that are under way
        for (int base = threadIdx.x; base - lane < rows * units; base += G * kThreads) {
            u32x4_t v[G][LV];
            uint32_t at[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int i = min(base + g * kThreads, rows * units - 1);
                const int row = (int)__umulhi((uint32_t)i, recip), col = i - row * units;
                // beyond a row's end (the last piece): out of the buffer, zeros
                at[g] = st0 * HB + col * 16 * LV < a.f * (kWideH<W> ? 4 : 2)
                            ? (uint32_t)(row0 + row) * (uint32_t)(a.f * (kWideH<W> ? 4 : 2)) + st0 * HB + col * 16 * LV
                            : 0x80000000u;
#pragma unroll
                for (int l = 0; l < LV; ++l) v[g][l] = load_shared(hb, at[g] + 16 * l);
            }
            for (;;) {  // until every word is written
                bool wait = false;
                uint32_t word = 0;
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int l = 0; l < LV; ++l)
                        if (marked(v[g][l])) {
                            wait = true;
                            const u32x4_t m = v[g][l];
                            word = at[g] / 4 + 4 * l + (m.x == kMark ? 0 : m.y == kMark ? 1 : m.z == kMark ? 2 : 3);
                        }
                if (!__any(wait) || lost) break;
                // (a few rows are simply read again)
                const bool gave_up = few ? ++tries > kSpinLimit : !wait_word(a.h + word, wait);
                if (gave_up) {
                    lost = true;
                    if (lane == 0) *a.status = 2;
                }
                asm volatile("" ::: "memory");
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int l = 0; l < LV; ++l) v[g][l] = load_shared(hb, at[g] + 16 * l);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int i = base + g * kThreads;
                if (i - lane >= rows * units) break;  // the whole wave
                const int row = (int)__umulhi((uint32_t)min(i, rows * units - 1), recip), col = min(i, rows * units - 1) - row * units;
                u32x4_t o = v[g][0];
                if constexpr (W == MOE_FP8_B128) {  // 16 lanes hold a group of 128
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = umax(m, v[g][e >> 2][e & 3] & 0x7FFFFFFFu);
                    const float s = fp8_scale(row16_max(m)), inv = 1.0f / s;
                    u32x4_t pk = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        pk[l] = fp8_pack4(as_f32(v[g][l].x), as_f32(v[g][l].y), as_f32(v[g][l].z), as_f32(v[g][l].w), inv);
                    const Wide8 hw = widen(join8(pk, pk));
                    o = __builtin_bit_cast(u32x4_t, hw.v[0]);
                    if ((lane & 15) == 0 && i < rows * units) hscale[row * (units / 16) + col / 16] = s;
                }
                if (i < rows * units) *(u32x4_t*)(hs + (size_t)row * (units * 16 + 16) + col * 16) = o;
            }
        }
    }
    // y's sums of this wave over the batch, R chunks at a time; the first ones' weights are on their way
    __device__ __forceinline__ void run(Choice ch, const uint8_t* hs, const float* hscale) {
        const int q = lane >> 4, r16 = lane & 15;
        const int first = b0 / nch, row_base = tb.row0[first];
        const int st0 = a.piece < nch ? (b0 - first * nch) / a.piece * a.piece * C : 0;
        const int steps = min(a.piece, nch) * C, row_bytes = steps * act_step<W>() + 16;
        int item = w0 / nch, st = (w0 - item * nch) * C;
        struct Place {  // this lane's row of h of a chunk, and its tokens' gates
            uint32_t row;
            float gate[4];
        };
        auto look = [&](int it) __attribute__((always_inline)) {
            Place p;
            p.row = ch.row[it * kFewTok + r16];
            if constexpr (W == MOE_INT4_G128) {
                const float4 g = *(const float4*)(ch.gate + it * kFewTok + 4 * q);
                p.gate[0] = g.x, p.gate[1] = g.y, p.gate[2] = g.z, p.gate[3] = g.w;
            } else {
                p.gate[0] = p.gate[1] = p.gate[2] = p.gate[3] = ch.gate[it * kFewTok + r16];
            }
            return p;
        };
        Place next = look(w0 < w1 ? item : tb.n_items);
        auto one = [&](int c, int r) __attribute__((always_inline)) {
            const Place p = next;
            const bool in = c < w1, over = st + C == nch * C;
            // past the end: the item that nobody chose
            next = look(c + 1 < w1 ? item + over : tb.n_items);
            const int at = p.row == kOff ? 0 : (int)p.row - row_base;  // a token that did not choose the expert: any row
            const int s = in ? st - st0 : 0;
            const uint8_t* hrow = hs + (size_t)at * row_bytes + s * act_step<W>();
            f32x4_t acc[RB];
#pragma unroll
            for (int m = 0; m < RB; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C; ++i) {
                u32x4_t x[FT::kXV];
#pragma unroll
                for (int v = 0; v < FT::kXV; ++v) x[v] = *(const u32x4_t*)(hrow + i * act_step<W>() + act_offset<W>(v, q));
                float hsc = 1.f;
                if constexpr (W == MOE_FP8_B128) hsc = hscale[at * steps + s + i];
                const f32x4_t sum = act_sum<W>(x);
#pragma unroll
                for (int m = 0; m < RB; ++m)
                    step_product<W>(acc[m], w[r][i][m], x, W == MOE_INT4_G128 || W == MOE_FP8_B128 ? scale_of(r, i, m) * hsc : 1.f, sum);
            }
#pragma unroll
            for (int m = 0; m < RB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[m][i] = is_off(p.gate[i]) ? y[m][i] : __builtin_fmaf(p.gate[i], acc[m][i], y[m][i]);
            st = over ? 0 : st + C;
            item += over;
            // a few operands at a time: the registers hold the weights
            if (RB > 1 || C * FT::kXV >= 4 || r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        };
        int c = w0;
        for (; c + R < w1; c += R) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                one(c + r, r);
                load_w(r);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) one(c + r, r);
    }
};

// The waves' sums of a down item joined: the first run's workgroup adds the others' and stores y.
template <int RB>
__device__ __forceinline__ void store_y(const FewArgs& a, bool wide, DownItem it, const float* red, bool& lost) {
    const int lane = threadIdx.x & 63;
    const size_t part = (size_t)a.T * a.d;
    for (int o = threadIdx.x; o < a.T * 16 * RB; o += kThreads) {  // whole waves
        const int t = o / (16 * RB), r = o % (16 * RB);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += red[w * 256 * RB + o];
        const size_t at = (size_t)t * a.d + it.block * 16 * RB + r;
        if (it.run > 0) {
            uint32_t v = as_u32(s);
            if (v == kMark) v = 0x7FFFFFFFu;
            __hip_atomic_store(a.part + (it.run - 1) * part + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            continue;
        }
        for (int p = 1; p < a.splits; p += 4) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __hip_atomic_load(a.part + (min(p + i, a.splits - 1) - 1) * part + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (p + i >= a.splits) break;
                const uint32_t* from = a.part + (p + i - 1) * part + at;
                while (__any(v[i] == kMark) && !lost) {
                    if (!wait_word(from, v[i] == kMark)) {
                        lost = true;
                        if (lane == 0) *a.status = 2;
                    }
                    v[i] = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
                s += as_f32(v[i]);
            }
        }
        if (wide) ((float*)a.y)[at] = s;
        else ((uint16_t*)a.y)[at] = f32_to_bf16(s);
    }
}

template <int W, int NS, int RG, int PB, int RB, int CD, int RD, int RE>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
    __shared__ FewTable tb;
    // the waves' sums and the scales (int4) of a gate/up item; then rows of h and their scales, and the sums of y
    extern __shared__ __align__(16) uint8_t lds[];
    using GU = GateUp<W, NS, RG, PB>;
    const Choice ch{(uint16_t*)(lds + (a.items_most + 1) * kFewTok * 4), (float*)lds};
    uint8_t* dyn = lds + a.choice_area;
    float* red = (float*)dyn;
    uint8_t* scales = dyn + kWaves * GU::kM * 1024;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int home = blockIdx.x % kLists, nb = a.f / 16 / PB, db = a.d / 16 / RB;
    uint32_t *gu_lists = a.lists, *dn_lists = a.lists + kLists * kListStride;
    // One wave asks for the workgroup's items ahead of time: of the down items (numbered from gate_up on) when all
    // gate/up items have been handed out; -1: none is left.
    const bool asks = wv == kWaves - 1;
    uint32_t ask0 = 0, ask1 = 0;
    if (asks) ask0 = few_request(gu_lists, home);
    int gate_up = 0;
    auto resolve = [&](uint32_t asked) __attribute__((always_inline)) {
        int it = few_resolve(gu_lists, gate_up, 1, home, asked);
        if (it < 0) {
            it = few_resolve(dn_lists, db, a.splits, home, few_request(dn_lists, home));
            if (it >= 0) it += gate_up;
        }
        if (lane == 0) tb.next = it;
    };
    few_table(a, tb, ch, [&](int n_items) __attribute__((always_inline)) {
        gate_up = n_items * nb;
        if (asks) {
            resolve(ask0);
            ask1 = few_request(gu_lists, home);
        }
    });
    if (tb.n_items == 0) {  // no expert is there
        if (blockIdx.x == 0) few_gates(a, tb, ch);
        for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.T * a.d; i += gridDim.x * kThreads) {
            if constexpr (W == MOE_F32) ((float*)a.y)[i] = 0.f;
            else ((uint16_t*)a.y)[i] = 0;
        }
        return;
    }
    auto is_gu = [&](int it) __attribute__((always_inline)) { return it >= 0 && it < gate_up; };
    auto down_of = [&](int it) __attribute__((always_inline)) { return down_item(it - gate_up, db, a.splits); };
    int it = __builtin_amdgcn_readfirstlane(tb.next);
    bool lost = false;
    Down<W, RB, CD, RD, RE> dn(a, tb);
    {
        GU gu(a, wv);
        const uint8_t* base = nullptr;
        const bool works = is_gu(it);  // fewer gate/up items than workgroups: some have none
        if (works) {
            base = gu.blocks_of(tb, it / nb, it % nb);
            gu.begin(base);
        }
        // the gates while the first weights are on their way; those of more tokens take longer than that: they are
        // formed while the first down item's are
        if (a.T <= kEarlyGates) few_gates(a, tb, ch);
        __syncthreads();  // the first item's number has been read
        if (works && asks) resolve(ask1);
        f32x4_t acc[GU::kM];
        auto put_sums = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < GU::kM; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[(wv * GU::kM + m) * 256 + acc_token<W>(lane, i) * 16 + acc_row<W>(lane, i)] = acc[m][i];
        };
        int next = it;
        while (works) {
            gu.put_scales(scales);
            __syncthreads();  // the next item is known, red is free, the scales are there
            next = __builtin_amdgcn_readfirstlane(tb.next);
            if (!is_gu(next)) break;
            if (asks) ask0 = few_request(gu_lists, home);
            const uint8_t* ahead = gu.blocks_of(tb, next / nb, next % nb);
            gu.template multiply<true>(acc, base, ahead, scales);
            base = ahead;
            put_sums();
            __syncthreads();
            if (asks) resolve(ask0);
            store_h<W, PB>(a, tb, it / nb, it % nb, red);
            it = next;
        }
        // the first down item's weights before the last gate/up item's products
        if (next >= 0) {
            dn.begin(down_of(next));
            dn.template load<0, RE>();
        }
        if (works) {
            gu.template multiply<false>(acc, base, nullptr, scales);
            put_sums();
            __syncthreads();
            store_h<W, PB>(a, tb, it / nb, it % nb, red);
        }
        it = next;
    }
    float* hscale = (float*)(dyn + a.h_area);
    if (it >= 0) dn.template load<RE, RD>();
    bool ask = true;
    if (a.T > kEarlyGates && (it >= 0 || blockIdx.x == 0)) few_gates(a, tb, ch);
    __syncthreads();
    while (it >= 0) {
        if (ask && asks) {
            const int next = few_resolve(dn_lists, db, a.splits, home, few_request(dn_lists, home));
            if (lane == 0) tb.next = next < 0 ? -1 : next + gate_up;
        }
        ask = false;
        if (dn.b0 < dn.b1) dn.stage(dyn, hscale, lost);
        __syncthreads();
        dn.run(ch, dyn, hscale);
        __syncthreads();  // the rows have been read
        if (dn.b1 < dn.c1) {
            dn.begin_batch(dn.b1);
        } else {
#pragma unroll
            for (int m = 0; m < RB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[wv * 256 * RB + acc_token<W>(lane, i) * 16 * RB + 16 * m + acc_row<W>(lane, i)] = dn.y[m][i];
            __syncthreads();
            store_y<RB>(a, W == MOE_F32, down_of(it), red, lost);
            it = __builtin_amdgcn_readfirstlane(tb.next);
            ask = true;
            __syncthreads();  // red and the number have been read
            if (it < 0) break;
            dn.begin(down_of(it));
        }
        dn.template load<0, RD>();
    }
}

struct FewLayout {  // workspace: status at byte 0, then
    size_t lists, logits, xq, xs, h, part, total;
    int splits;
};
FewLayout few_layout(int T, int d, int f, int E, int k, bool shared, moe_dtype w) {
    FewLayout l;
    const size_t rows = (size_t)T * k + (shared ? T : 0), esz = w == MOE_F32 || w == MOE_FP8_B128 ? 4 : 2;
    l.lists = 256;
    l.logits = l.lists + (size_t)2 * kLists * kListStride * 4;
    l.xq = align_up(l.logits + (size_t)T * E * 4, 256);
    l.xs = l.xq + (w == MOE_FP8_B128 ? align_up((size_t)T * d * 2, 256) : 0);
    l.h = l.xs + (w == MOE_FP8_B128 ? align_up((size_t)T * (d / 128) * 4, 256) : 0);
    l.part = l.h + rows * f * esz;
    l.splits = few_splits(T, d, f, E, k, shared, w);
    l.total = align_up(l.part + (size_t)(l.splits - 1) * T * d * 4, 256);
    return l;
}

template <bool kBf16>
void launch_prepare(const FewArgs& a, int quant_blocks, hipStream_t st) {
    const int fill = (int)std::min<size_t>(256, std::max<size_t>(4, (a.marks / 4 + 255) / 256));
    ProfScope p("few_prepare", st);
    if (a.T <= 2) {
        const int lb = (a.T * a.E + 3) / 4;
        few_prepare_kernel<kBf16, 1><<<lb + quant_blocks + fill, 256, 0, st>>>(a, lb, quant_blocks);
    } else {
        const int lb = ((a.T + 3) / 4 * a.E + 3) / 4;
        few_prepare_kernel<kBf16, 4><<<lb + quant_blocks + fill, 256, 0, st>>>(a, lb, quant_blocks);
    }
}

template <int W, int NS, int RG, int PB, int RB, int CD, int RD, int RE>
moe_status launch_shape(FewArgs a, hipStream_t st) {
    using FT = FewType<W>;
    // rows of h in LDS: as many as the call has, in whole rows if a full expert's fit
    a.items_most = std::min(a.T * a.k, a.E) + (a.shared_w ? 1 : 0);
    a.choice_area = (int)align_up(choice_bytes(a.items_most), 64);
    const int kArea = (132 << 10) - a.choice_area;
    const int nch = a.f / FT::kIn / CD, chunk = CD * act_step<W>(), rows = std::min(a.T * a.k + (a.shared_w ? a.T : 0), kFewRows + kFewTok);
    a.piece = std::min(nch, (kArea / a.T - 16) / chunk);
    const int row_bytes = a.piece * chunk + 16;
    a.rows_fit = std::min(rows, kArea / row_bytes);
    a.h_area = a.rows_fit * row_bytes;
    const int sums = kWaves * 2 * PB * 1024 + (W == MOE_INT4_G128 ? 2 * PB * 32 * (a.d / 128) : 0);
    const int lds = a.choice_area + std::max({a.h_area + (W == MOE_FP8_B128 ? a.rows_fit * a.piece * CD * 4 : 0), sums, kWaves * RB * 1024});
    auto kern = few_layer_kernel<W, NS, RG, PB, RB, CD, RD, RE>;
    MOE_HIP(hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds));
    // weights, steps of x held, steps a chunk, row blocks a down item: a profile tells the forms apart
    static const std::string name = std::string("few_layer_") + (W == MOE_F32 ? "f32" : W == MOE_BF16 ? "bf16" : W == MOE_INT4_G128 ? "int4" : "fp8") +
                                    "_" + std::to_string(NS) + "_" + std::to_string(CD) + "_" + std::to_string(RB);
    ProfScope ps(name.c_str(), st);
    // a workgroup a compute unit, fewer where there are fewer items
    const int64_t items = (int64_t)a.items_most * (a.f / 16 / PB) + a.d / 16 / RB * a.splits;
    kern<<<(unsigned)std::min<int64_t>(kFewUnits, items), kThreads, lds, st>>>(a);
    return MOE_OK;
}

template <int W>
moe_status launch_layer(const FewArgs& a, int rb, hipStream_t st) {
    if constexpr (W == MOE_BF16) {
        if (rb == 1) {
            if (a.d <= 1024) return launch_shape<W, 4, 4, 2, 1, 1, 12, 12>(a, st);
            if (a.d <= 2048) return launch_shape<W, 8, 8, 1, 1, 1, 12, 12>(a, st);
            if (a.d <= 4096) return launch_shape<W, 16, 8, 1, 1, 1, 12, 12>(a, st);
            return launch_shape<W, 0, 8, 1, 1, 1, 12, 12>(a, st);
        }
        if (a.d <= 1024) return launch_shape<W, 4, 4, 2, 4, 1, 6, 6>(a, st);
        if (a.d <= 2048) return launch_shape<W, 8, 8, 1, 4, 1, 6, 6>(a, st);
        if (a.d <= 4096) return launch_shape<W, 16, 8, 1, 4, 1, 6, 4>(a, st);
        return launch_shape<W, 0, 8, 1, 4, 1, 6, 4>(a, st);
    } else if constexpr (W == MOE_INT4_G128) {
        const bool even = a.f % 256 == 0;
        if (rb == 1) {
            if (even && a.d <= 2048) return launch_shape<W, 2, 2, 4, 1, 2, 7, 4>(a, st);
            if (even && a.d <= 4096) return launch_shape<W, 4, 4, 2, 1, 2, 7, 4>(a, st);
            return launch_shape<W, 0, 2, 2, 1, 1, 10, 6>(a, st);
        }
        if (even && a.d <= 2048) return launch_shape<W, 2, 2, 4, 4, 2, 2, 2>(a, st);
        if (even && a.d <= 4096) return launch_shape<W, 4, 4, 2, 4, 2, 2, 2>(a, st);
        return launch_shape<W, 0, 2, 2, 4, 1, 4, 4>(a, st);
    } else if constexpr (W == MOE_FP8_B128) {
        if (rb == 1) {
            if (a.d <= 2048) return launch_shape<W, 2, 2, 2, 1, 1, 8, 8>(a, st);
            if (a.d <= 4096) return launch_shape<W, 4, 4, 1, 1, 1, 8, 8>(a, st);
            return launch_shape<W, 0, 2, 1, 1, 1, 8, 8>(a, st);
        }
        if (a.d <= 2048) return launch_shape<W, 2, 2, 2, 4, 1, 3, 2>(a, st);
        if (a.d <= 4096) return launch_shape<W, 4, 4, 1, 4, 1, 3, 2>(a, st);
        return launch_shape<W, 0, 2, 1, 4, 1, 3, 2>(a, st);
    } else {
        if (rb == 1) return launch_shape<W, 0, 4, 1, 1, 1, 8, 8>(a, st);
        return launch_shape<W, 0, 4, 1, 4, 1, 3, 2>(a, st);
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_layer_few_workspace_bytes(int T, int d, int f, int E, int k, int has_shared, moe_dtype w) {
    if (T < 0 || T > kFewTok || E < 1 || E > kPermMaxE || k < 1 || k > E || k > kFewK || d % 64 != 0 || !slot_shape_ok(d, f, w)) return 0;
    return few_layout(T, d, f, E, k, has_shared != 0, w).total;
}

extern "C" moe_status moe_layer_few(const void* x, moe_dtype act, int T, int d, int f, int E, int k, const void* w_router,
                                    const float* bias, const int32_t* forced_idx, const int32_t* slot_of_expert,
                                    int n_slots, const void* slot_pool, size_t slot_stride, moe_dtype w,
                                    const void* shared_w, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                                    size_t ws_bytes, moe_stream s) {
    const char* fn = "moe_layer_few";
    MOE_CHECK(T >= 0 && T <= kFewTok, MOE_ESHAPE, "%s: T=%d must be in [0,%d]", fn, T, kFewTok);
    MOE_CHECK(act == MOE_F32 || act == MOE_BF16, MOE_EDTYPE, "%s: activations must be F32 or BF16", fn);
    MOE_CHECK(w == MOE_F32 || w == MOE_BF16 || w == MOE_INT4_G128 || w == MOE_FP8_B128, MOE_EDTYPE, "%s: unknown weight type %d", fn, (int)w);
    MOE_CHECK((act == MOE_F32) == (w == MOE_F32), MOE_EDTYPE, "%s: F32 weights go with F32 activations, the others with BF16", fn);
    MOE_CHECK(E >= 1 && E <= kPermMaxE && k >= 1 && k <= E && k <= kFewK, MOE_ESHAPE, "%s: need 1 <= k <= min(E, %d), E <= %d (k=%d E=%d)",
              fn, kFewK, kPermMaxE, k, E);
    MOE_CHECK(slot_shape_ok(d, f, w) && d % 64 == 0, MOE_ESHAPE, "%s: unsupported shape d=%d f=%d", fn, d, f);
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && w_router && slot_of_expert && slot_pool && topk_idx && topk_w && y && ws, MOE_EINVAL, "%s: NULL pointer", fn);
    MOE_CHECK(n_slots >= 1, MOE_EINVAL, "%s: n_slots=%d < 1", fn, n_slots);
    MOE_CHECK(slot_stride >= moe_slot_bytes(d, f, w) && slot_stride % 256 == 0, MOE_EINVAL,
              "%s: slot_stride %zu smaller than a slot (%zu) or not 256-aligned", fn, slot_stride, moe_slot_bytes(d, f, w));
    MOE_CHECK((((uintptr_t)slot_pool | (uintptr_t)shared_w) & 255) == 0, MOE_EINVAL,
              "%s: slot pool / shared expert must be 256-byte aligned", fn);
    MOE_CHECK((((uintptr_t)x | (uintptr_t)w_router | (uintptr_t)y | (uintptr_t)ws) & 15) == 0, MOE_EINVAL,
              "%s: x, w_router, y and ws must be 16-byte aligned", fn);
    MOE_CHECK((((uintptr_t)bias | (uintptr_t)forced_idx | (uintptr_t)slot_of_expert | (uintptr_t)topk_idx | (uintptr_t)topk_w) & 3) == 0,
              MOE_EINVAL, "%s: bias, forced_idx, slot_of_expert, topk_idx and topk_w must be 4-byte aligned", fn);
    const FewLayout l = few_layout(T, d, f, E, k, shared_w != nullptr, w);
    MOE_CHECK(ws_bytes >= l.total, MOE_ENOMEM, "%s: workspace of %zu bytes, need %zu", fn, ws_bytes, l.total);
    uint8_t* p = (uint8_t*)ws;
    FewArgs a{x, T, d, f, E, k, w_router, bias, forced_idx, slot_of_expert, n_slots, (const uint8_t*)slot_pool, slot_stride,
              (const uint8_t*)shared_w, topk_idx, topk_w, y, (int32_t*)p, (uint32_t*)(p + l.lists), (float*)(p + l.logits),
              (uint16_t*)(p + l.xq), (float*)(p + l.xs), (uint32_t*)(p + l.h), (uint32_t*)(p + l.part),
              l.part - l.h, (l.part + (size_t)(l.splits - 1) * T * d * 4 - l.h) / 4, l.splits};
    hipStream_t st = (hipStream_t)s;
    const int quant_blocks = w == MOE_FP8_B128 ? (T * (d / 128) + 3) / 4 : 0;
    if (act == MOE_BF16) launch_prepare<true>(a, quant_blocks, st);
    else launch_prepare<false>(a, quant_blocks, st);
    moe_status r = check_launch("few_prepare");
    if (r != MOE_OK) return r;
    const int rb = few_row_blocks(T, f, k, shared_w != nullptr, w);
    switch (w) {
        case MOE_F32: r = launch_layer<MOE_F32>(a, rb, st); break;
        case MOE_BF16: r = launch_layer<MOE_BF16>(a, rb, st); break;
        case MOE_INT4_G128: r = launch_layer<MOE_INT4_G128>(a, rb, st); break;
        default: r = launch_layer<MOE_FP8_B128>(a, rb, st); break;
    }
    if (r != MOE_OK) return r;
    return check_launch("few_layer");
}
