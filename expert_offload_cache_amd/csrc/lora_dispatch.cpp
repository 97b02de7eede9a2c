// Entry points of moe_lora_linear: checks and the choice of kernels.
#include "lora.h"

using namespace moe;

extern "C" {

size_t moe_lora_workspace_bytes(int M, int r) {
    if (M < 0 || r < 8 || r > MOE_LORA_MAX_RANK || r % 8 != 0) return 0;
    return align_up((size_t)M * r * 4, 256) + kLoraPartBytes;
}

moe_status moe_lora_linear(const void* x, size_t ldx, int M, int K, const void* w, size_t ldw, int N, const void* base,
                           size_t ldb, moe_dtype base_dtype, const void* a, const void* b, int r, int n, const float* scale,
                           const int32_t* rank, const int32_t* adapter, void* y, size_t ldy, moe_dtype out, void* ws,
                           size_t ws_bytes, moe_stream s) {
    const char* fn = "moe_lora_linear";
    MOE_CHECK(M >= 0 && M <= (1 << 21), MOE_ESHAPE, "%s: M=%d must be in [0, 2^21]", fn, M);
    MOE_CHECK(K >= 8 && K % 8 == 0 && K <= (1 << 20), MOE_ESHAPE, "%s: K=%d must be a multiple of 8 in [8, 2^20]", fn, K);
    MOE_CHECK(N >= 1 && N <= (1 << 22), MOE_ESHAPE, "%s: N=%d must be in [1, 2^22]", fn, N);
    MOE_CHECK(r >= 8 && r % 8 == 0 && r <= MOE_LORA_MAX_RANK, MOE_ESHAPE, "%s: r=%d must be a multiple of 8 in [8, %d]", fn, r,
              MOE_LORA_MAX_RANK);
    MOE_CHECK(n >= 1 && n <= (1 << 20), MOE_ESHAPE, "%s: n=%d adapters must be in [1, 2^20]", fn, n);
    MOE_CHECK(out == MOE_F32 || out == MOE_BF16, MOE_EDTYPE, "%s: y must be F32 or BF16", fn);
    MOE_CHECK(!base || base_dtype == MOE_F32 || base_dtype == MOE_BF16, MOE_EDTYPE, "%s: base must be F32 or BF16", fn);
    if (M == 0) return MOE_OK;
    MOE_CHECK(x && a && b && scale && adapter && y && ws, MOE_EINVAL, "%s: NULL pointer", fn);
    MOE_CHECK(ldx >= (size_t)K && ldx % 8 == 0 && (!w || (ldw >= (size_t)K && ldw % 8 == 0)), MOE_EINVAL,
              "%s: rows of x and w must be at least K apart, a multiple of 8", fn);
    MOE_CHECK(ldy >= (size_t)N && (!base || ldb >= (size_t)N), MOE_EINVAL, "%s: rows of y and base must be at least N apart", fn);
    MOE_CHECK((((uintptr_t)x | (uintptr_t)w | (uintptr_t)a | (uintptr_t)b | (uintptr_t)ws) & 15) == 0, MOE_EINVAL,
              "%s: x, w, a, b and ws must be 16-byte aligned", fn);
    MOE_CHECK((((uintptr_t)scale | (uintptr_t)rank | (uintptr_t)adapter) & 3) == 0 && (uintptr_t)y % (out == MOE_F32 ? 4 : 2) == 0 &&
                  (uintptr_t)base % (base_dtype == MOE_F32 ? 4 : 2) == 0,
              MOE_EINVAL, "%s: scale, rank, adapter, y and base must be aligned to their elements", fn);
    MOE_CHECK(base != y || (base_dtype == out && ldb == ldy), MOE_EINVAL, "%s: y may be base only with its type and stride", fn);
    MOE_CHECK(ws_bytes >= moe_lora_workspace_bytes(M, r), MOE_ENOMEM, "%s: workspace of %zu bytes, need %zu", fn, ws_bytes,
              moe_lora_workspace_bytes(M, r));
    LoraArgs p{(const uint16_t*)x, ldx, M, K, (const uint16_t*)w, ldw, N, base, ldb, (const uint16_t*)a, (const uint16_t*)b, r, n,
               scale, rank, adapter, y, ldy, (float*)ws, (float*)((uint8_t*)ws + align_up((size_t)M * r * 4, 256)), 0, false};
    p.splits = lora_splits(p);
    auto starts_wide = [](const void* q, size_t ld, moe_dtype t) { return (((uintptr_t)q | ld * (t == MOE_F32 ? 4 : 2)) & 15) == 0; };
    p.wide = starts_wide(y, ldy, out) && (!base || starts_wide(base, ldb, base_dtype));
    hipStream_t st = (hipStream_t)s;
    moe_status e = lora_shrink(p, st);
    if (e != MOE_OK) return e;
    return lora_rows(p, base_dtype, out, st);
}

}  // extern "C"
