// Block-128 FP8 operands: E4M3 codes with one scale per 128 values along the sum.
//
// An activation or gradient row carries one E8M0 byte per 128 values (2^(b-127)): the matrix
// instructions apply it themselves, and dividing by a power of two is exact, so a code depends on
// nothing but its value and its block's largest magnitude.  E4M3 is a floating-point format: a power
// of two loses nothing of a value's relative precision against amax / 448, at most one binade of
// the subnormal end.  A weight carries one scale per 128 x 128 block, float32 (a checkpoint's) or E8M0.
#pragma once
#include "common.h"

namespace moe {

constexpr int kFp8Block = 128;
__host__ __device__ inline int fp8_blocks(int n) { return (int)(((int64_t)n + kFp8Block - 1) / kFp8Block); }

constexpr uint32_t kFp8Inf = 0x7f800000u;
// Bits of |v| when v is finite, else 0: NaN and infinities take no part in a block's scale.
MOE_DEV uint32_t fp8_magnitude(float v) {
    const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
    return m < 0x7f800000u ? m : 0u;
}
// The smallest X with amax <= 448 2^X (448 = 1.75 2^8), kept in [-127, 127]; a zero block has -127.
MOE_DEV int fp8_exponent(uint32_t amax_bits) {
    const int X = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(X, -127);                                                // (at most 120)
}
MOE_DEV float fp8_inverse(int X) { return __uint_as_float((uint32_t)(127 - X) << 23); }   // 2^-X

// Four values times 2^-X as E4M3 codes, rounded to nearest even; NaN and infinities as NaN.  FINITE: there are none (a block's
// largest magnitude, taken over all of it, says so): a multiplication and half a conversion a value.
template <bool FINITE = false>
MOE_DEV uint32_t fp8_codes4(float a, float b, float c, float d, float inv) {
    auto q = [&](float v) __attribute__((always_inline)) {
        return FINITE || (__float_as_uint(v) & 0x7fffffffu) < 0x7f800000u ? v * inv : __uint_as_float(0x7fc00000u);
    };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), w, true);
}
MOE_DEV uint32_t fp8_abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest of 16 neighbouring lanes' values, in registers (DPP), the same in each of them.
MOE_DEV uint32_t fp8_max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));       // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));       // quad_perm [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));      // row_half_mirror
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));   // row_mirror
}

// Eight codes of an operand, bytes 8 i .., as bf16, exactly.
MOE_DEV bf16x8 fp8_widen8(const i32x8 &v, int i) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i], 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i], 1.0f, true);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i + 1], 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * i + 1], 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// silu(g) = g / (1 + e^-g) with the hardware exp2 and reciprocal (about 2 ulp).
MOE_DEV float fp8_silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.44269504088896341f));
}

// ------------------------------------------------------------------ the product kernels

// y[r][n] = sum over 128-blocks of ws 2^X sum_k w[n][k] x[r][k]; rows r of one expert each, or of one matrix.
struct Fp8Product {
    const uint8_t *x, *xs;        // codes [n_x][K], E8M0 scales [n_x][Kb]
    const void *x_values;         // fp8_rows16_launch: bf16 or float32 rows in place of codes (they fit kFp8RowsLds)
    int x_f32;
    int n_x;                      // rows of x
    const int32_t *sorted_pairs;  // gathered rows (x row = sorted_pairs[r] / k), or NULL
    int k;
    const uint8_t *w[2];          // codes [E][N][K]; the gated pair: gate, up
    const void *ws[2];            // scales (MOE_FP8_SCALE_*)
    int w_scale;
    int E, N, K, Kb;
    const int32_t *offsets;       // NULL: one matrix, rows 0 .. R-1
    int R;
    // one matrix
    void *y;                      // [R][N]
    const void *residual;         // of y's type, or NULL
    int y_f32;
    float *part;                  // [split][R][N] when the sum is split
    int bt, split;                // rows of a tile (64, 128, 192, 256) and parts of the sum
    // the gated pair
    float *h;                     // [R][N] float32 or NULL
    uint8_t *hq, *hs;             // h as codes [R][N] and scales [R][N/128]
};

// What moe_fp8_linear does with its sizes: rows of a tile and parts of the sum; no rows: the weights are streamed.
struct Fp8Plan {
    int bt, split;
};
Fp8Plan fp8_linear_plan(const moe_fp8_linear_desc *d);

moe_status fp8_product_launch(const Fp8Product &p, bool pair, hipStream_t s, const char *what);
// Few rows: the weights stream once (fp8_stream.hip).  fp8_stream_launch: rows of experts (float32 weight scales), the gated pair
// or float32 results of multiples of 4 columns; fp8_rows16_launch: up to 64 rows of one matrix, or rows of experts (float32
// weight scales and results), x as codes or, up to 16 rows, as x_values; its gated pair (16 rows of one matrix) writes h in
// float32 only.
moe_status fp8_stream_launch(const Fp8Product &p, bool pair, hipStream_t s, const char *what);
moe_status fp8_rows16_launch(const Fp8Product &p, bool pair, hipStream_t s, const char *what);
constexpr int kFp8RowsMax = 16;                           // quantised by the workgroups, or of a gated pair
constexpr int kFp8FewRows = 32;                           // of experts in all: fp8_rows16_launch
// LDS of rows that a workgroup quantises itself (codes, then scales); up to kFp8RowsLds of it
__host__ __device__ inline int fp8_row_lds(int Kb) { return Kb * kFp8Block + 16; }      // (16: rows fall on other banks)
inline size_t fp8_rows16_lds(int rows, int K) { return (size_t)rows * (fp8_row_lds(fp8_blocks(K)) + (size_t)fp8_blocks(K)); }
constexpr size_t kFp8RowsLds = 48 * 1024;
inline bool fp8_rows_fit(int rows, int K) { return rows <= kFp8RowsMax && fp8_rows16_lds(rows, K) <= kFp8RowsLds; }
// live: device, rows from *live on stay as they are; or NULL.
moe_status fp8_quantize_rows_launch(int rows, int cols, const void *x, bool f32, uint8_t *codes, uint8_t *scales, hipStream_t s,
                                    const int32_t *live = nullptr);

}  // namespace moe
