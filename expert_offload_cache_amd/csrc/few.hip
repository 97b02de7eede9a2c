// moe_layer_few: a whole MoE layer for at most kFewTok tokens in two launches.
//
//   logits = x Wr^T + bias;  S = the k largest;  g = softmax over S;
//   h_e = silu(x Wg_e^T) * (x Wu_e^T);  y = sum_{e in S} g_e (h_e Wd_e^T)  (+ the shared expert)
//
// Launch 1 (few_prepare_kernel): the logits in the fixed order of moe_route, for 8-bit weights the
// quantised rows of x, and the marks and counters that launch 2 starts from.
// Launch 2 (few_layer_kernel): every workgroup selects the experts for itself from the logits (T * E
// numbers), then the workgroups take work items in order: first all gate/up items (one expert, 16
// columns of h, all of its tokens), then the down items (16 columns of y, all experts, all tokens).
// With at most 16 tokens the tokens are one operand block of the matrix instructions, so an expert's
// weights are read once and its tokens need no gathering: columns of tokens that did not choose it are left out of
// the sums.  A down item holds all of a token's experts, so the gates are applied to binary32 sums in
// registers and no rows are written between.
//
// The hand-over of h.  A down item needs h of every expert, which other workgroups write in the same
// launch.  Launch 1 fills h with a mark (all bits set, which is a NaN that h never holds: a NaN
// result of those bits is stored as another NaN).  h is written and read with device-scope accesses of
// whole words, and a reader that finds the mark reads again: each word is its own flag.
// Why every wait ends: items are handed out by counters, gate/up items first, and gate/up items wait for
// nothing.  A workgroup gets a down item only after all gate/up items have been handed out to workgroups that
// run already, whatever else occupies the device.  (A second call that uses the same workspace
// at the same time breaks this; then the wait ends at its limit and the status word is set to 2.)
#include <hip/hip_runtime.h>

#include <algorithm>

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
constexpr int kWaves = 8;                  // of a workgroup of launch 2
constexpr int kThreads = 64 * kWaves;
constexpr int kLists = 8;                  // counters of each kind, a cache line each: one word takes 11 ns an increment
constexpr int kListStride = 64;            // words from a counter to the next
constexpr uint32_t kMark = 0xFFFFFFFFu;    // a word of h that is not written yet
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
    uint32_t* h;      // [rows, f] bf16 (binary32 for F32 and fp8)
    size_t h_words;
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
    for (size_t i = i0; i < a.h_words / 4; i += n) ((u32x4_t*)a.h)[i] = u32x4_t{kMark, kMark, kMark, kMark};
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
struct FewTable {
    int n_act, n_items;             // experts with weights to read; with the shared one
    int next;                       // the workgroup's next item
    int16_t expert[kFewRows + 1];   // item -> expert (-1: the shared one)
    uint16_t tokens[kFewRows + 1];  // item -> the tokens that chose it, a bit each
    int16_t row[kFewRows + 1];      // item -> its first row of h
    int slot[kFewRows + 1];
    int16_t item_of[1024];          // expert -> item, or -1
    uint32_t chosen[1024];          // expert -> tokens, a bit each
    int sel[kFewTok][kFewK];
    float gate[kFewTok][kFewK];
    float row_gate[kFewRows + kFewTok];
};

// binary32 -> an integer of the same order; NaN below everything
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = as_u32(v == 0.f ? 0.f : v);
    if (v != v) return 1u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) { return quarter_max(row16_max(v)); }

// One wave selects one token's experts: k rounds of the largest logit left (equal ones: the lowest id), and
// the gates as moe_route forms them.
__device__ __forceinline__ void few_select(const FewArgs& a, int t, FewTable& tb, bool write) {
    const int lane = threadIdx.x & 63;
    const float* row = a.logits + (size_t)t * a.E;
    int sel = 0;
    float val = 0.f;
    if (a.forced) {
        if (lane < a.k) {
            sel = a.forced[(size_t)t * a.k + lane];
            val = row[min(max(sel, 0), a.E - 1)];
        }
    } else {
        uint32_t key[16];
        const int per = (a.E + 63) / 64;
#pragma unroll
        for (int i = 0; i < 16; ++i) key[i] = i < per && lane + 64 * i < a.E ? order_key(row[lane + 64 * i]) : 0u;
        for (int r = 0; r < a.k; ++r) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < per) best = umax(best, key[i]);
            best = __builtin_amdgcn_readfirstlane(wave_max_u32(best));
            int id = -1;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < per && id < 0) {
                    const uint64_t at = __ballot(key[i] == best);
                    if (at) {
                        id = 64 * i + __builtin_ctzll(at);
                        if (lane == (id & 63)) key[i] = 0;
                    }
                }
            if (lane == r) sel = id;
        }
        val = lane < a.k ? row[sel] : 0.f;
    }
    double m = -INFINITY;
    for (int i = 0; i < a.k; ++i) m = fmax(m, (double)__shfl(val, i, 64));
    const double term = lane < a.k ? exp((double)val - m) : 0.0;
    double den = 0.0;
    for (int i = 0; i < a.k; ++i) den += __shfl(term, i, 64);
    if (lane < a.k) {
        const float g = (float)(term / den);
        if (write) {
            a.topk_idx[(size_t)t * a.k + lane] = sel;
            a.topk_w[(size_t)t * a.k + lane] = g;
        }
        tb.sel[t][lane] = min(max(sel, 0), a.E - 1);
        tb.gate[t][lane] = g;
    }
}

// The items of the call: the chosen experts in ascending order, the shared one last.
__device__ __forceinline__ void few_table(const FewArgs& a, FewTable& tb) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    for (int e = tid; e < a.E; e += kThreads) {
        tb.chosen[e] = 0;
        tb.item_of[e] = -1;
    }
    for (int t = wv; t < a.T; t += kWaves) few_select(a, t, tb, blockIdx.x == 0);
    __syncthreads();
    const int pairs = a.T * a.k;
    for (int p = tid; p < pairs; p += kThreads) {
        const int t = p / a.k;
        atomicOr(&tb.chosen[tb.sel[t][p - t * a.k]], 1u << t);
    }
    __syncthreads();
    if (wv == 0) {
        const uint64_t lt = (1ull << lane) - 1;
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const int e = e0 + lane;
            const uint32_t c = e < a.E ? tb.chosen[e] : 0;
            const int slot = c ? a.slot_of_expert[e] : 0;
            const bool there = slot >= 0 && slot < a.n_slots;
            // an absent expert adds nothing to y; one whose rows come from elsewhere is no error
            if (c && !there && slot != MOE_SLOT_ELSEWHERE && blockIdx.x == 0) *a.status = 1;
            const uint64_t on = __ballot(c && there);
            int mine = c && there ? __popc(c) : 0, incl = mine;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const int v = __shfl_up(incl, s, 64);
                if (lane >= s) incl += v;
            }
            if (c && there) {
                const int i = n + __popcll(on & lt);
                tb.expert[i] = (int16_t)e;
                tb.tokens[i] = (uint16_t)c;
                tb.row[i] = (int16_t)(rows + incl - mine);
                tb.slot[i] = slot;
                tb.item_of[e] = (int16_t)i;
            }
            n += __popcll(on);
            rows += __shfl(incl, 63, 64);
        }
        if (lane == 0) {
            tb.n_act = n;
            if (a.shared_w) {
                tb.expert[n] = -1;
                tb.tokens[n] = (uint16_t)((1u << a.T) - 1);
                tb.row[n] = (int16_t)rows;
                tb.slot[n] = -1;
            }
            tb.n_items = n + (a.shared_w ? 1 : 0);
        }
        if (a.shared_w && lane < a.T) tb.row_gate[rows + lane] = 1.0f;
    }
    __syncthreads();
    // the gate of each row; an id given twice for a token counts with the sum of its gates
    for (int p = tid; p < pairs; p += kThreads) {
        const int t = p / a.k, j = p - t * a.k, e = tb.sel[t][j], i = tb.item_of[e];
        float g = 0.f;
        bool first = true;
        for (int u = 0; u < a.k; ++u)
            if (tb.sel[t][u] == e) {
                g += tb.gate[t][u];
                first = first && u >= j;
            }
        if (i >= 0 && first) tb.row_gate[tb.row[i] + __popc(tb.tokens[i] & ((1u << t) - 1))] = g;
    }
    __syncthreads();
}

// The next work item of a kind (wave 0 only): item c + kLists v is the v-th of list c.  A workgroup
// starts with the list of its number and goes on to the others; -1: every list is handed out.
__device__ __forceinline__ int few_take(uint32_t* lists, int total, int home) {
    const int lane = threadIdx.x & 63;
    int c = home;
    for (;;) {
        uint32_t v = 0;
        if (lane == 0) v = __hip_atomic_fetch_add(lists + c * kListStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v = __builtin_amdgcn_readfirstlane(v);
        const int n = (total - c + kLists - 1) / kLists;
        if ((int)v < n) return c + kLists * (int)v;
        // another list that is not handed out yet
        const int o = (home + lane) % kLists;
        const uint32_t seen = lane < kLists ? __hip_atomic_load(lists + o * kListStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
        const uint64_t left = __ballot(lane < kLists && (int)seen < (total - o + kLists - 1) / kLists);
        if (!left) return -1;
        c = (home + __builtin_ctzll(left)) % kLists;
    }
}

// 16 bytes of h, read at device scope
__device__ __forceinline__ u32x4_t load_h(const uint32_t* p) {
    const uint64_t lo = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t hi = __hip_atomic_load((const uint64_t*)p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ __forceinline__ bool marked(u32x4_t v) { return v.x == kMark || v.y == kMark || v.z == kMark || v.w == kMark; }

// One gate/up item: 16 columns of h of one expert.  The waves split the inputs.
template <int W>
__device__ __forceinline__ void few_gate_up(const FewArgs& a, const FewTable& tb, int item, int b, float* red) {
    using FT = FewType<W>;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = __builtin_amdgcn_readfirstlane(tb.slot[item]);
    const uint8_t* base = slot < 0 ? a.shared_w : a.pool + (size_t)slot * a.stride;
    const uint8_t* wg = base + gu_block_offset(b, 0, a.d, (moe_dtype)W);
    const uint8_t* wu = base + gu_block_offset(b, 1, a.d, (moe_dtype)W);
    const int nst = a.d / FT::kIn, s0 = wv * nst / kWaves, s1 = (wv + 1) * nst / kWaves;
    const uint8_t* xrow = (W == MOE_FP8_B128 ? (const uint8_t*)a.xq : (const uint8_t*)a.x) +
                          (size_t)min(r16, a.T - 1) * a.d * (W == MOE_F32 ? 4 : 2);
    f32x4_t g = {0.f, 0.f, 0.f, 0.f}, u = g;
    constexpr int C = 4;  // steps whose loads are issued together
    for (int s = s0; s < s1; s += C) {
        u32x4_t vg[C][FT::kWV], vu[C][FT::kWV], vx[C][FT::kXV];
        float sg[C], su[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int st = min(s + c, s1 - 1);
#pragma unroll
            for (int v = 0; v < FT::kWV; ++v) {
                const size_t o = (size_t)st * FT::kWV * 1024 + (W == MOE_F32 ? lane * 32 + v * 16 : v * 1024 + lane * 16);
                vg[c][v] = __builtin_nontemporal_load((const u32x4_t*)(wg + o));
                vu[c][v] = __builtin_nontemporal_load((const u32x4_t*)(wu + o));
            }
#pragma unroll
            for (int v = 0; v < FT::kXV; ++v) vx[c][v] = *(const u32x4_t*)(xrow + (size_t)st * act_step<W>() + act_offset<W>(v, q));
            if constexpr (W == MOE_INT4_G128) {
                const size_t o = (size_t)nst * 1024 + ((size_t)r16 * nst + st) * 2;
                sg[c] = bf16_to_f32(*(const uint16_t*)(wg + o));
                su[c] = bf16_to_f32(*(const uint16_t*)(wu + o));
            } else if constexpr (W == MOE_FP8_B128) {
                const float sx = a.xs[(size_t)min(r16, a.T - 1) * nst + st];
                sg[c] = ((const float*)(wg + (size_t)16 * a.d))[st] * sx;
                su[c] = ((const float*)(wu + (size_t)16 * a.d))[st] * sx;
            } else {
                sg[c] = su[c] = 1.f;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (s + c < s1) {
                const f32x4_t xs = act_sum<W>(vx[c]);
                step_product<W>(g, vg[c], vx[c], sg[c], xs);
                step_product<W>(u, vu[c], vx[c], su[c], xs);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = acc_token<W>(lane, i) * 16 + acc_row<W>(lane, i);
        red[(2 * wv) * 256 + at] = g[i];
        red[(2 * wv + 1) * 256 + at] = u[i];
    }
    __syncthreads();
    if (tid < 256) {
        const int t = tid >> 4, r = tid & 15;
        float gs = red[tid], us = red[256 + tid];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            gs += red[(2 * w) * 256 + tid];
            us += red[(2 * w + 1) * 256 + tid];
        }
        const float v = silu_mul(gs, us);
        const uint32_t tokens = tb.tokens[item];
        const bool on = (tokens >> t) & 1;
        const size_t row = (size_t)(tb.row[item] + __popc(tokens & ((1u << t) - 1)));
        if constexpr (W == MOE_F32 || W == MOE_FP8_B128) {
            uint32_t o = as_u32(v);
            if (o == kMark) o = 0x7FFFFFFFu;
            if (on) __hip_atomic_store(a.h + row * a.f + b * 16 + r, o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else {
            uint32_t o = f32_to_bf16(v);
            o |= (uint32_t)__shfl_xor((int)o, 1, 64) << 16;
            if (o == kMark) o = 0x7FFF7FFFu;
            if (on && !(r & 1))
                __hip_atomic_store(a.h + (row * a.f + b * 16 + r) / 2, o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __syncthreads();
}

// One down item: 16 columns of y.  The waves split the (expert, step) pairs into runs.
template <int W>
__device__ __forceinline__ void few_down(const FewArgs& a, const FewTable& tb, int b, float* red, bool& lost) {
    using FT = FewType<W>;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, r16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nst = a.f / FT::kIn, total = tb.n_items * nst;
    const int u0 = (int)((int64_t)wv * total / kWaves), u1 = (int)((int64_t)(wv + 1) * total / kWaves);
    constexpr int HW = FT::kIn * (W == MOE_F32 || W == MOE_FP8_B128 ? 4 : 2) / 64;  // 16-byte vectors of h a lane reads a step
    constexpr int C = W == MOE_BF16 ? 8 : 2;
    f32x4_t y = {0.f, 0.f, 0.f, 0.f};
    int u = u0;
    while (u < u1) {
        const int item = u / nst, end = min(u1, (item + 1) * nst);
        const int slot = __builtin_amdgcn_readfirstlane(tb.slot[item]);
        const uint32_t tokens = __builtin_amdgcn_readfirstlane((int)tb.tokens[item]);
        const int row0 = __builtin_amdgcn_readfirstlane((int)tb.row[item]);
        const uint8_t* base = slot < 0 ? a.shared_w : a.pool + (size_t)slot * a.stride;
        const uint8_t* wd = base + down_block_offset(b, a.d, a.f, (moe_dtype)W);
        const bool on = (tokens >> r16) & 1;
        constexpr int kPer = W == MOE_F32 || W == MOE_FP8_B128 ? 1 : 2;  // elements a word
        const uint32_t* hrow = a.h + (size_t)(row0 + (on ? __popc(tokens & ((1u << r16) - 1)) : 0)) * (a.f / kPer);
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
        for (; u < end; u += C) {
            u32x4_t vw[C][FT::kWV];
            float sw[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int st = min(u + c, end - 1) - item * nst;
#pragma unroll
                for (int v = 0; v < FT::kWV; ++v)
                    vw[c][v] = __builtin_nontemporal_load((const u32x4_t*)(
                        wd + (size_t)st * FT::kWV * 1024 + (W == MOE_F32 ? lane * 32 + v * 16 : v * 1024 + lane * 16)));
                if constexpr (W == MOE_INT4_G128)
                    sw[c] = bf16_to_f32(*(const uint16_t*)(wd + (size_t)nst * 1024 + ((size_t)r16 * nst + st) * 2));
                else if constexpr (W == MOE_FP8_B128) sw[c] = ((const float*)(wd + (size_t)16 * a.f))[st];
                else sw[c] = 1.f;
            }
            u32x4_t vh[C][HW];
            for (int spin = 0;; ++spin) {
                bool wait = false;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int st = min(u + c, end - 1) - item * nst;
#pragma unroll
                    for (int v = 0; v < HW; ++v) {
                        int o;  // word of the row
                        if constexpr (W == MOE_FP8_B128) o = st * 128 + 64 * (v >> 2) + 16 * q + 4 * (v & 3);
                        else o = (st * act_step<W>() + act_offset<W>(v, q)) / 4;
                        vh[c][v] = on ? load_h(hrow + o) : u32x4_t{0u, 0u, 0u, 0u};
                        wait = wait || marked(vh[c][v]);
                    }
                }
                if (!__any(wait) || lost) break;
                if (spin == kSpinLimit) {
                    lost = true;
                    if (lane == 0) *a.status = 2;
                    break;
                }
                __builtin_amdgcn_s_sleep(2);
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (u + c < end) {
                    u32x4_t x[FT::kXV];
                    float scale = sw[c];
                    if constexpr (W == MOE_FP8_B128) {
                        uint32_t m = 0;
#pragma unroll
                        for (int v = 0; v < HW; ++v)
#pragma unroll
                            for (int i = 0; i < 4; ++i) m = umax(m, vh[c][v][i] & 0x7FFFFFFFu);
                        const float s = fp8_scale(quarter_max(m)), r = 1.0f / s;
                        u32x4_t p[2];
#pragma unroll
                        for (int v = 0; v < HW; ++v)
                            p[v >> 2][v & 3] = fp8_pack4(as_f32(vh[c][v].x), as_f32(vh[c][v].y), as_f32(vh[c][v].z), as_f32(vh[c][v].w), r);
                        const Wide8 hw = widen(join8(p[0], p[1]));
#pragma unroll
                        for (int v = 0; v < 4; ++v) x[v] = __builtin_bit_cast(u32x4_t, hw.v[v]);
                        scale *= s;
                    } else {
#pragma unroll
                        for (int v = 0; v < FT::kXV; ++v) x[v] = vh[c][v];
                    }
                    step_product<W>(acc, vw[c], x, scale, act_sum<W>(x));
                }
        }
        u = end;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = acc_token<W>(lane, i);
            if ((tokens >> t) & 1) y[i] = __builtin_fmaf(tb.row_gate[row0 + __popc(tokens & ((1u << t) - 1))], acc[i], y[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wv * 256 + acc_token<W>(lane, i) * 16 + acc_row<W>(lane, i)] = y[i];
    __syncthreads();
    if (tid < 256) {
        const int t = tid >> 4, r = tid & 15;
        float s = red[tid];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) s += red[w * 256 + tid];
        if (t < a.T) {
            const size_t at = (size_t)t * a.d + b * 16 + r;
            if constexpr (W == MOE_F32) ((float*)a.y)[at] = s;
            else ((uint16_t*)a.y)[at] = f32_to_bf16(s);
        }
    }
    __syncthreads();
}

template <int W>
__global__ __launch_bounds__(kThreads, 4) void few_layer_kernel(FewArgs a) {
    __shared__ FewTable tb;
    __shared__ float red[2 * kWaves * 256];
    few_table(a, tb);
    const int nb = a.f / 16, gate_up = tb.n_items * nb, down = a.d / 16;
    const int home = blockIdx.x % kLists;
    bool lost = false;
    for (int kind = 0; kind < 2; ++kind) {
        for (;;) {
            if (threadIdx.x < 64) {
                const int it = few_take(a.lists + kind * kLists * kListStride, kind ? down : gate_up, home);
                if (threadIdx.x == 0) tb.next = it;
            }
            __syncthreads();
            const int it = __builtin_amdgcn_readfirstlane(tb.next);
            __syncthreads();
            if (it < 0) break;
            if (kind == 0) few_gate_up<W>(a, tb, it / nb, it % nb, red);
            else few_down<W>(a, tb, it, red, lost);
        }
    }
}

struct FewLayout {  // workspace: status at byte 0, then
    size_t lists, logits, xq, xs, h, total, h_words;
};
FewLayout few_layout(int T, int d, int f, int E, int k, bool shared, moe_dtype w) {
    FewLayout l;
    const size_t rows = (size_t)T * k + (shared ? T : 0), esz = w == MOE_F32 || w == MOE_FP8_B128 ? 4 : 2;
    l.lists = 256;
    l.logits = l.lists + (size_t)2 * kLists * kListStride * 4;
    l.xq = align_up(l.logits + (size_t)T * E * 4, 256);
    l.xs = l.xq + (w == MOE_FP8_B128 ? align_up((size_t)T * d * 2, 256) : 0);
    l.h = l.xs + (w == MOE_FP8_B128 ? align_up((size_t)T * (d / 128) * 4, 256) : 0);
    l.h_words = rows * f * esz / 4;
    l.total = align_up(l.h + l.h_words * 4, 256);
    return l;
}

template <bool kBf16>
void launch_prepare(const FewArgs& a, int quant_blocks, hipStream_t st) {
    const int fill = (int)std::min<size_t>(256, std::max<size_t>(4, (a.h_words / 4 + 255) / 256));
    ProfScope p("few_prepare", st);
    if (a.T <= 2) {
        const int lb = (a.T * a.E + 3) / 4;
        few_prepare_kernel<kBf16, 1><<<lb + quant_blocks + fill, 256, 0, st>>>(a, lb, quant_blocks);
    } else {
        const int lb = ((a.T + 3) / 4 * a.E + 3) / 4;
        few_prepare_kernel<kBf16, 4><<<lb + quant_blocks + fill, 256, 0, st>>>(a, lb, quant_blocks);
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
    const FewLayout l = few_layout(T, d, f, E, k, shared_w != nullptr, w);
    MOE_CHECK(ws_bytes >= l.total, MOE_ENOMEM, "%s: workspace of %zu bytes, need %zu", fn, ws_bytes, l.total);
    uint8_t* p = (uint8_t*)ws;
    FewArgs a{x, T, d, f, E, k, w_router, bias, forced_idx, slot_of_expert, n_slots, (const uint8_t*)slot_pool, slot_stride,
              (const uint8_t*)shared_w, topk_idx, topk_w, y, (int32_t*)p, (uint32_t*)(p + l.lists), (float*)(p + l.logits),
              (uint16_t*)(p + l.xq), (float*)(p + l.xs), (uint32_t*)(p + l.h), l.h_words};
    hipStream_t st = (hipStream_t)s;
    const int quant_blocks = w == MOE_FP8_B128 ? (T * (d / 128) + 3) / 4 : 0;
    if (act == MOE_BF16) launch_prepare<true>(a, quant_blocks, st);
    else launch_prepare<false>(a, quant_blocks, st);
    moe_status r = check_launch("few_prepare");
    if (r != MOE_OK) return r;
    // two workgroups a compute unit, fewer where there are fewer items
    const int64_t items = (int64_t)(std::min(T * k, E) + (shared_w ? 1 : 0)) * (f / 16) + d / 16;
    const unsigned grid = (unsigned)std::min<int64_t>(512, items);
    ProfScope ps("few_layer", st);
    switch (w) {
        case MOE_F32: few_layer_kernel<MOE_F32><<<grid, kThreads, 0, st>>>(a); break;
        case MOE_BF16: few_layer_kernel<MOE_BF16><<<grid, kThreads, 0, st>>>(a); break;
        case MOE_INT4_G128: few_layer_kernel<MOE_INT4_G128><<<grid, kThreads, 0, st>>>(a); break;
        default: few_layer_kernel<MOE_FP8_B128><<<grid, kThreads, 0, st>>>(a); break;
    }
    return check_launch("few_layer");
}
