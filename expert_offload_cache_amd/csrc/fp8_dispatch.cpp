// moe_gemm_fp8 and moe_expert_ffn_fp8: argument checks and the choice of kernel.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fp8_ops.h"
#include "slot_layout.h"

using namespace moe;

namespace moe {

// n rows of w e4m3 values and their scales behind them
static size_t rows8_bytes(size_t n, int w) { return align_up(n * w, 256) + align_up(n * (w / 128) * 4, 256); }

// h of the streaming kernels, or x and h in 8 bits; never less than fewer tokens take, so that a workspace of the
// most tokens serves every call
size_t ffn_fp8_workspace(int T, int d, int f, int k, int has_shared) {
    const size_t per = (size_t)k + (has_shared ? 1 : 0);
    const size_t few = align_up(std::min(T, kFp8Stream) * per * f * 4, 256);
    const size_t many = T > kFp8Stream ? rows8_bytes(T, d) + rows8_bytes(T * per, f) : 0;
    return kWsHeader + kPlanBytes + std::max(few, many);
}

moe_status ffn_fp8_run(const FfnFp8& call, hipStream_t st) {
    FfnFp8 p = call;
    p.x8 = p.x_scale ? (const uint8_t*)p.a.x : nullptr;
    if (p.a.T <= kFp8Stream) {
        moe_status r = ffn_fp8_stream(p, kGateUp, st);
        return r != MOE_OK ? r : ffn_fp8_stream(p, kDown, st);
    }
    uint8_t* ws = (uint8_t*)p.a.h;
    if (!p.x8) {
        float* scale = (float*)(ws + align_up((size_t)p.a.T * p.a.d, 256));
        moe_status r = quant_rows_bf16(p.a.x, p.a.T, p.a.d, ws, scale, st);
        if (r != MOE_OK) return r;
        p.x8 = ws;
        p.x_scale = scale;
    }
    const size_t rows = (size_t)p.a.T * p.a.k + (p.a.shared_w ? (size_t)p.a.T : 0);
    p.h8 = ws + rows8_bytes(p.a.T, p.a.d);
    p.h_scale = (float*)(p.h8 + align_up(rows * p.a.f, 256));
    moe_status r = ffn_fp8_tile(p, kGateUp, st);
    return r != MOE_OK ? r : ffn_fp8_tile(p, kDown, st);
}

}  // namespace moe

extern "C" {

moe_status moe_gemm_fp8(const void* a, size_t lda, const float* a_scale, int M, int K, const void* w, size_t ldw,
                        const float* w_scale, int N, void* c, size_t ldc, moe_dtype out, moe_stream s) {
    MOE_CHECK(M >= 0 && N >= 1 && K >= 16 && K % 16 == 0, MOE_ESHAPE,
              "moe_gemm_fp8: need M >= 0, N >= 1 and K a positive multiple of 16 (M=%d N=%d K=%d)", M, N, K);
    MOE_CHECK(N <= (1 << 24) && K <= (1 << 20), MOE_ESHAPE, "moe_gemm_fp8: N=%d or K=%d too large", N, K);
    MOE_CHECK(out == MOE_F32 || out == MOE_BF16, MOE_EDTYPE, "moe_gemm_fp8: output must be F32 or BF16");
    if (M == 0) return MOE_OK;
    MOE_CHECK(a && a_scale && w && w_scale && c, MOE_EINVAL, "moe_gemm_fp8: NULL pointer");
    MOE_CHECK(lda >= (size_t)K && ldw >= (size_t)K && ldc >= (size_t)N, MOE_EINVAL,
              "moe_gemm_fp8: a row stride below the row");
    MOE_CHECK((uintptr_t)a % 16 == 0 && (uintptr_t)w % 16 == 0 && lda % 16 == 0 && ldw % 16 == 0, MOE_EINVAL,
              "moe_gemm_fp8: rows of a and w must start on 16 bytes");
    const size_t esz = out == MOE_BF16 ? 2 : 4;
    MOE_CHECK((uintptr_t)a_scale % 4 == 0 && (uintptr_t)w_scale % 4 == 0 && (uintptr_t)c % esz == 0, MOE_EINVAL,
              "moe_gemm_fp8: scales or c not aligned to their elements");
    GemmFp8 g;
    g.a = (const uint8_t*)a;
    g.lda = lda;
    g.a_scale = a_scale;
    g.w = (const uint8_t*)w;
    g.ldw = ldw;
    g.w_scale = w_scale;
    g.c = c;
    g.ldc = ldc;
    g.M = M;
    g.N = N;
    g.K = K;
    g.G = fp8_groups(K);
    g.c_bf16 = out == MOE_BF16;
    g.c_vec = (uintptr_t)c % 16 == 0 && ldc * esz % 16 == 0;
    float tile_us;
    const void* tile = gemm_fp8_best_tile(g, tile_us);
    if (tile && tile_us < gemm_fp8_stream_us(g)) return gemm_fp8_tile(g, tile, (hipStream_t)s);
    return gemm_fp8_stream(g, (hipStream_t)s);
}

moe_status moe_expert_ffn_fp8(const void* x, const float* x_scale, int T, int d, int f, int E, int k,
                              const int32_t* perm, const int32_t* offsets, const int32_t* counts,
                              const int32_t* slot_of_expert, int n_slots, const void* slot_pool, size_t slot_stride,
                              const void* shared_w, void* y_perm, moe_dtype y_dtype, void* ws, size_t ws_bytes,
                              moe_stream s) {
    FfnFp8 p{};
    moe_status r = ffn_prepare(p.a, "moe_expert_ffn_fp8", x, MOE_FP8_B128, T, d, f, E, k, perm, offsets, counts,
                               slot_of_expert, n_slots, slot_pool, slot_stride, MOE_FP8_B128, shared_w, y_perm, y_dtype,
                               true);
    if (r != MOE_OK || T == 0) return r;
    MOE_CHECK(x_scale && (uintptr_t)x_scale % 4 == 0, MOE_EINVAL, "moe_expert_ffn_fp8: NULL or misaligned x_scale");
    MOE_CHECK(ws && (uintptr_t)ws % 256 == 0, MOE_EINVAL,
              "moe_expert_ffn_fp8: workspace must not be NULL and must be 256-byte aligned");
    const size_t need = moe_workspace_bytes(T, d, f, E, k, shared_w != nullptr, MOE_BF16, MOE_FP8_B128);
    MOE_CHECK(ws_bytes >= need, MOE_ENOMEM, "moe_expert_ffn_fp8: workspace %zu < %zu bytes", ws_bytes, need);
    p.x_scale = x_scale;
    p.a.status = (int32_t*)ws;
    p.a.plan = (uint8_t*)ws + kWsHeader;
    p.a.h = (uint8_t*)ws + kWsHeader + kPlanBytes;
    return ffn_fp8_run(p, (hipStream_t)s);
}

}  // extern "C"
