// moe_add_rmsnorm and moe_quant_fp8: rows of activations, read once.
//
//   h = x + residual (rounded to the rows' type, as it is kept for the next layer),
//   y = h / sqrt(mean(h^2) + eps) * weight,
// y rounded once to the rows' type and / or held in 8 bits (fp8.h) from its binary32 value.  The
// norm is of the rounded h, so the call gives what the addition and the norm give one by one.
//
// A row belongs to NW waves; lane l of wave w holds C chunks of 8 columns, chunk (w + i NW) 64 + l,
// in registers from the load to the last store, so a row is read once, and the 16 lanes of a
// 128-column group are neighbours: its largest magnitude is joined by four lane exchanges.  The sum
// of squares is joined in one fixed order (lanes, then waves through LDS); NW and C follow from
// the width alone, so a row's bits do not depend on how many rows the call has.
//
// Bound by memory: 8192 bf16 rows of 4096 with a residual and both outputs (303 MB) 58 us, 5.2 TB/s;
// 8192 bf16 rows of 2048 quantised (51 MB) 9.5 us, 5.3 TB/s (a 4 GiB copy reaches 4.8 TB/s; some of
// these rows are still in the last-level cache).  At most 16 columns a lane, so that a row stays in registers
// (28 of them at 4096 columns) and a compute unit holds 8 waves a SIMD.  One row of 4096 takes 4 us, a launch.
#include <hip/hip_runtime.h>

#include "fp8_ops.h"

namespace moe {
namespace {

struct RowArgs {
    const void* x;
    const void* residual;  // or nullptr
    const void* weight;    // norm only
    void* resid_out;       // or nullptr
    void* y;               // or nullptr
    uint8_t* q;            // or nullptr
    float* scale;
    int T, d;
    size_t ldx, ldr, ldro, ldy, ldq;
    float eps;
};

// 8 columns from c on, zeros past the row's end
template <typename E, bool VEC>
__device__ __forceinline__ void load8(const E* row, int c, int d, float (&v)[8]) {
    if constexpr (VEC) {
        if (c < d) {
            if constexpr (sizeof(E) == 2) {
                const uint4 r = *(const uint4*)(row + c);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = bf16_lo(w[i]);
                    v[2 * i + 1] = bf16_hi(w[i]);
                }
            } else {
                const float4 a = *(const float4*)(row + c), b = *(const float4*)(row + c + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.f;
            if (c + i < d) {
                if constexpr (sizeof(E) == 2) v[i] = bf16_to_f32((uint16_t)row[c + i]);
                else v[i] = row[c + i];
            }
        }
    }
}

template <typename E, bool VEC>
__device__ __forceinline__ void store8(E* row, int c, int d, const float (&v)[8]) {
    if constexpr (VEC) {
        if (c >= d) return;
        if constexpr (sizeof(E) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
            *(uint4*)(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *(float4*)(row + c) = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < d) {
                if constexpr (sizeof(E) == 2) row[c + i] = f32_to_bf16(v[i]);
                else row[c + i] = v[i];
            }
    }
}

// E, WE: element types of the rows and of the norm's weight.  VEC: every row starts on 16 bytes
// (q rows on 8) and d is a multiple of 8.  NW waves a row, 4 / NW rows a workgroup where NW < 4.
template <typename E, typename WE, bool NORM, bool VEC, int NW, int C>
__global__ __launch_bounds__((NW < 4 ? 4 : NW) * 64) void rows_kernel(RowArgs a) {
    constexpr int ROWS = NW < 4 ? 4 / NW : 1;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t0 = blockIdx.x * ROWS + wv / NW;
    const bool live = t0 < a.T;
    const size_t t = live ? t0 : a.T - 1;  // a row past the end repeats the last one and stores nothing
    const int w = wv % NW;
    float v[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i)
        load8<E, VEC>((const E*)a.x + t * a.ldx, ((w + i * NW) * 64 + lane) * 8, a.d, v[i]);
    if constexpr (NORM) {
        float wt[C][8];
#pragma unroll
        for (int i = 0; i < C; ++i)
            load8<WE, VEC>((const WE*)a.weight, ((w + i * NW) * 64 + lane) * 8, a.d, wt[i]);
        if (a.residual) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int c = ((w + i * NW) * 64 + lane) * 8;
                float r[8];
                load8<E, VEC>((const E*)a.residual + t * a.ldr, c, a.d, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] += r[j];
                    if constexpr (sizeof(E) == 2) v[i][j] = bf16_to_f32(f32_to_bf16(v[i][j]));
                }
                if (live) store8<E, VEC>((E*)a.resid_out + t * a.ldro, c, a.d, v[i]);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
        ss = as_f32(__builtin_amdgcn_readfirstlane(as_u32(wave_tree_sum(ss))));
        if constexpr (NW > 1) {
            __shared__ float part[NW < 4 ? 4 : NW];
            if (lane == 0) part[wv] = ss;
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) ss += part[wv - w + i];
        }
        const float rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * wt[i][j];
            if (a.y && live) store8<E, VEC>((E*)a.y + t * a.ldy, ((w + i * NW) * 64 + lane) * 8, a.d, v[i]);
        }
        if (!a.q) return;
    }
    const int G = (a.d + kFp8Group - 1) / kFp8Group;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = ((w + i * NW) * 64 + lane) * 8;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[i][j]));  // zeros past the row's end
        const float s = fp8_scale(row16_max(m));
        const float r = 1.0f / s;
        const uint32_t lo = fp8_pack4(v[i][0], v[i][1], v[i][2], v[i][3], r);
        const uint32_t hi = fp8_pack4(v[i][4], v[i][5], v[i][6], v[i][7], r);
        if (!live || c >= a.d) continue;
        uint8_t* qr = a.q + t * a.ldq + c;
        if constexpr (VEC) {
            *(uint2*)qr = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < a.d) qr[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
        }
        if ((lane & 15) == 0) a.scale[t * G + c / kFp8Group] = s;
    }
}

template <typename E, typename WE, bool NORM, bool VEC, int NW, int C>
moe_status launch_rows(const RowArgs& a, hipStream_t st, const char* name) {
    constexpr int ROWS = NW < 4 ? 4 / NW : 1, THREADS = (NW < 4 ? 4 : NW) * 64;
    constexpr int MOST = (1 << 30) / THREADS * ROWS;  // rows a launch: the grid's threads must stay below 2^32
    RowArgs r = a;
    for (int64_t t = 0; t < a.T; t += MOST) {
        r.T = (int)(a.T - t < MOST ? a.T - t : MOST);
        r.x = (const E*)a.x + t * a.ldx;
        if (a.residual) r.residual = (const E*)a.residual + t * a.ldr, r.resid_out = (E*)a.resid_out + t * a.ldro;
        if (a.y) r.y = (E*)a.y + t * a.ldy;
        if (a.q) r.q = a.q + t * a.ldq, r.scale = a.scale + t * fp8_groups(a.d);
        ProfScope p(name, st);
        rows_kernel<E, WE, NORM, VEC, NW, C><<<(unsigned)((r.T + ROWS - 1) / ROWS), THREADS, 0, st>>>(r);
        const moe_status s = check_launch(name);
        if (s != MOE_OK) return s;
    }
    return MOE_OK;
}

template <typename E, typename WE, bool NORM, bool VEC>
moe_status pick_rows(const RowArgs& a, hipStream_t st, const char* name) {
    const int chunks = (a.d + 7) / 8;
    if (chunks <= 64) return launch_rows<E, WE, NORM, VEC, 1, 1>(a, st, name);
    if (chunks <= 128) return launch_rows<E, WE, NORM, VEC, 2, 1>(a, st, name);
    if (chunks <= 256) return launch_rows<E, WE, NORM, VEC, 4, 1>(a, st, name);
    if (chunks <= 512) return launch_rows<E, WE, NORM, VEC, 4, 2>(a, st, name);
    if (chunks <= 1024) return launch_rows<E, WE, NORM, VEC, 8, 2>(a, st, name);
    return launch_rows<E, WE, NORM, VEC, 16, 2>(a, st, name);
}

template <typename E, typename WE, bool NORM>
moe_status run_rows(const RowArgs& a, hipStream_t st, const char* name) {
    auto aligned = [](const void* p, size_t ld, size_t esz, size_t to) {
        return !p || ((uintptr_t)p % to == 0 && ld * esz % to == 0);
    };
    const bool vec = a.d % 8 == 0 && aligned(a.x, a.ldx, sizeof(E), 16) && aligned(a.residual, a.ldr, sizeof(E), 16) &&
                     aligned(a.resid_out, a.ldro, sizeof(E), 16) && aligned(a.y, a.ldy, sizeof(E), 16) &&
                     aligned(a.q, a.ldq, 1, 8) && aligned(a.weight, 0, 1, 16);
    return vec ? pick_rows<E, WE, NORM, true>(a, st, name) : pick_rows<E, WE, NORM, false>(a, st, name);
}

constexpr int kMaxRow = 16384;

size_t elem(moe_dtype t) { return t == MOE_BF16 ? 2 : 4; }

}  // namespace

moe_status quant_rows_bf16(const void* x, int T, int d, uint8_t* q, float* scale, hipStream_t st) {
    RowArgs a{};
    a.x = x;
    a.q = q;
    a.scale = scale;
    a.T = T;
    a.d = d;
    a.ldx = a.ldq = (size_t)d;
    return run_rows<uint16_t, uint16_t, false>(a, st, "quant_fp8_bf16");
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_add_rmsnorm(const void* x, moe_dtype act, int T, int d, size_t ldx, const void* residual, size_t ldr,
                           const void* weight, moe_dtype w_dtype, float eps, void* resid_out, size_t ldro, void* y,
                           size_t ldy, void* q, size_t ldq, float* scale, moe_stream s) {
    MOE_CHECK(T >= 0 && d >= 1 && d <= kMaxRow, MOE_ESHAPE, "moe_add_rmsnorm: need T >= 0 and 1 <= d <= %d (T=%d d=%d)",
              kMaxRow, T, d);
    MOE_CHECK(act == MOE_F32 || act == MOE_BF16, MOE_EDTYPE, "moe_add_rmsnorm: rows must be F32 or BF16");
    MOE_CHECK(w_dtype == MOE_F32 || w_dtype == act, MOE_EDTYPE,
              "moe_add_rmsnorm: the weight must be F32 or have the rows' type");
    MOE_CHECK(eps >= 0.f, MOE_EINVAL, "moe_add_rmsnorm: eps must be at least 0");
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && weight && (y || q), MOE_EINVAL, "moe_add_rmsnorm: NULL rows or weight, or no output");
    MOE_CHECK(!q == !scale, MOE_EINVAL, "moe_add_rmsnorm: q and scale come together");
    MOE_CHECK(!residual == !resid_out, MOE_EINVAL, "moe_add_rmsnorm: residual and resid_out come together");
    MOE_CHECK(ldx >= (size_t)d && (!residual || (ldr >= (size_t)d && ldro >= (size_t)d)) &&
                  (!y || ldy >= (size_t)d) && (!q || ldq >= (size_t)d),
              MOE_EINVAL, "moe_add_rmsnorm: a row stride below d");
    const size_t esz = elem(act);
    MOE_CHECK((uintptr_t)x % esz == 0 && (uintptr_t)residual % esz == 0 && (uintptr_t)resid_out % esz == 0 &&
                  (uintptr_t)y % esz == 0 && (uintptr_t)weight % elem(w_dtype) == 0 && (uintptr_t)scale % 4 == 0,
              MOE_EINVAL, "moe_add_rmsnorm: a pointer is not aligned to its elements");
    RowArgs a{x, residual, weight, resid_out, y, (uint8_t*)q, scale, T, d, ldx, ldr, ldro, ldy, ldq, eps};
    hipStream_t st = (hipStream_t)s;
    if (act == MOE_F32) return run_rows<float, float, true>(a, st, "add_rmsnorm_f32");
    if (w_dtype == MOE_F32) return run_rows<uint16_t, float, true>(a, st, "add_rmsnorm_bf16");
    return run_rows<uint16_t, uint16_t, true>(a, st, "add_rmsnorm_bf16");
}

moe_status moe_quant_fp8(const void* x, moe_dtype act, int T, int d, size_t ldx, void* q, size_t ldq, float* scale,
                         moe_stream s) {
    MOE_CHECK(T >= 0 && d >= 1 && d <= kMaxRow, MOE_ESHAPE, "moe_quant_fp8: need T >= 0 and 1 <= d <= %d (T=%d d=%d)",
              kMaxRow, T, d);
    MOE_CHECK(act == MOE_F32 || act == MOE_BF16, MOE_EDTYPE, "moe_quant_fp8: rows must be F32 or BF16");
    if (T == 0) return MOE_OK;
    MOE_CHECK(x && q && scale, MOE_EINVAL, "moe_quant_fp8: NULL pointer");
    MOE_CHECK(ldx >= (size_t)d && ldq >= (size_t)d, MOE_EINVAL, "moe_quant_fp8: a row stride below d");
    MOE_CHECK((uintptr_t)x % elem(act) == 0 && (uintptr_t)scale % 4 == 0, MOE_EINVAL,
              "moe_quant_fp8: a pointer is not aligned to its elements");
    RowArgs a{};
    a.x = x;
    a.q = (uint8_t*)q;
    a.scale = scale;
    a.T = T;
    a.d = d;
    a.ldx = ldx;
    a.ldq = ldq;
    hipStream_t st = (hipStream_t)s;
    if (act == MOE_F32) return run_rows<float, float, false>(a, st, "quant_fp8_f32");
    return run_rows<uint16_t, uint16_t, false>(a, st, "quant_fp8_bf16");
}

}  // extern "C"
