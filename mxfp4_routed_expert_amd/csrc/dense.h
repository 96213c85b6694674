// Dense bf16 feed-forward operators: shared declarations, activations and product epilogues.
//
// Three products cover the linear layer, the gated projections and their gradients, all over
// row-major bf16 matrices with float32 accumulation on v_mfma_f32_16x16x32_bf16:
//   forward       z  [T][n]    = x  [T][k] . W [n][k]^T     both operands contiguous along the sum
//   input grad    dx [T][k]    = dz [T][n] . W [n][k]       the weight strided along the sum
//   weight grad   dW [n][k]    = dz [T][n]^T . x [T][k]     both strided along the sum (over T)
// An epilogue works on four consecutive columns of one output row in float32, either straight
// from a tile's accumulators or, when the sum was split over workgroups, from the summed
// partial results; both callers run the same functor, so every form of an operator rounds at
// the same places.
#pragma once
#include "common.h"

namespace moe {

MOE_DEV uint32_t pack2_bf16(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};        // round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}
MOE_DEV void store4_bf16(uint16_t *p, const f32x4 v) {
    *(u32x2 *)p = u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
}
MOE_DEV f32x4 load4_bf16(const uint16_t *p) {
    const u32x2 w = *(const u32x2 *)p;
    const f32x2 a = bf16x2_to_f32x2(w[0]), b = bf16x2_to_f32x2(w[1]);
    return f32x4{a.x, a.y, b.x, b.y};
}
MOE_DEV uint16_t bf16_bits(float v) { return (uint16_t)(pack2_bf16(v, 0.0f) & 0xffffu); }

// ------------------------------------------------------------------ activations
// f(z) and f'(z) in float32.
//   silu       z s(z), s the logistic function          f' = s (1 + z (1 - s))
//   gelu       z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2  f' = Phi + z exp(-z^2/2) / sqrt(2 pi)
//   gelu_tanh  0.5 z (1 + tanh q) = z s(2q), q = sqrt(2/pi) (z + 0.044715 z^3): the logistic form
//              has no cancellation for negative z         f' = s + z s (1 - s) 2q'
//   relu       max(z, 0) (NaN stays NaN)                 f' = [z > 0]
// 1 - s is taken as s(-t), so it keeps its relative accuracy where s rounds to 1.
constexpr float kGeluA = 1.5957691216057308f;           // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

MOE_DEV float gelu_arg(float z) { return z * (kGeluA + (kGeluA * kGeluB) * z * z); }

MOE_DEV float act_f(int fn, float z) {
    if (fn == MOE_FN_NONE) return z;
    if (fn == MOE_FN_RELU) return z < 0.0f ? 0.0f : z;
    if (fn == MOE_FN_GELU) return 0.5f * z * erfcf(-0.70710678118654752f * z);
    const float t = fn == MOE_FN_SILU ? z : gelu_arg(z);
    return z / (1.0f + expf(-t));
}

// f(z) in a, f'(z) in d
MOE_DEV void act_fd(int fn, float z, float &a, float &d) {
    if (fn == MOE_FN_NONE) {
        a = z;
        d = 1.0f;
    } else if (fn == MOE_FN_RELU) {
        a = z < 0.0f ? 0.0f : z;
        d = z > 0.0f ? 1.0f : 0.0f;
    } else if (fn == MOE_FN_GELU) {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * z);
        a = z * phi;
        d = phi + z * (0.39894228040143268f * expf(-0.5f * z * z));
    } else {
        const bool si = fn == MOE_FN_SILU;
        const float t = si ? z : gelu_arg(z);
        const float s = 1.0f / (1.0f + expf(-t)), c = 1.0f / (1.0f + expf(t));
        const float dt = si ? 1.0f : kGeluA + (3.0f * kGeluA * kGeluB) * z * z;
        a = z * s;
        d = s + a * (c * dt);
    }
}

// ------------------------------------------------------------------ epilogues
// apply(r, c, a, b, ca, cb): columns c .. c+3 of row r (c a multiple of 4); a is the product, b
// the second matrix's when kPair.  With kColSum, ca / cb return what column sums add.  Columns
// at or past C hold nothing and are not stored.  Rows of C columns are accessed 4 at a time when
// C is a multiple of 4 (then every row start is aligned for it), else one at a time.

// y = f(z + bias) + residual
struct EpiLinear {
    static constexpr bool kPair = false, kColSum = false;
    const float *bias;
    const void *res;      // y's type, or NULL
    void *y;
    int C, fn, y_f32;
    float *cs = nullptr;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4, f32x4 &, f32x4 &) const {
        const size_t o = (size_t)r * C + c;
        if ((C & 3) == 0) {
            if (bias) a += *(const f32x4 *)(bias + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = act_f(fn, a[q]);
            if (y_f32) {
                if (res) a += *(const f32x4 *)((const float *)res + o);
                *(f32x4 *)((float *)y + o) = a;
            } else {
                if (res) a += load4_bf16((const uint16_t *)res + o);
                store4_bf16((uint16_t *)y + o, a);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (c + q >= C) break;
                float v = act_f(fn, a[q] + (bias ? bias[c + q] : 0.0f));
                if (y_f32) {
                    if (res) v += ((const float *)res)[o + q];
                    ((float *)y)[o + q] = v;
                } else {
                    if (res) v += bf16_to_f32(((const uint16_t *)res)[o + q]);
                    ((uint16_t *)y)[o + q] = bf16_bits(v);
                }
            }
        }
    }
};

// h = f(g + bg) * (u + bu); the pre-activations rounded to bf16 when the caller keeps them.
// C is a multiple of 8.
struct EpiGate {
    static constexpr bool kPair = true, kColSum = false;
    const float *bg, *bu;
    void *h;
    uint16_t *pre;        // [2][R][C] or NULL
    size_t plane;         // R * C
    int C, fn, h_f32;
    float *cs = nullptr;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4 b, f32x4 &, f32x4 &) const {
        const size_t o = (size_t)r * C + c;
        if (bg) a += *(const f32x4 *)(bg + c);
        if (bu) b += *(const f32x4 *)(bu + c);
        if (pre) {
            store4_bf16(pre + o, a);
            store4_bf16(pre + plane + o, b);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = act_f(fn, a[q]) * b[q];
        if (h_f32) *(f32x4 *)((float *)h + o) = a;
        else store4_bf16((uint16_t *)h + o, a);
    }
};

// Up to this many tokens a value that feeds a product is kept as several bf16 terms (its rounding, and
// the rounding of what is left) instead of one: the products are then bound by the weights' bytes,
// and the terms ride along as further rows of the same tile.  Beyond it dz (dg, du) is one bf16
// value, the operand type of the matrix cores: one rounding of 2^-8 at most per value, and the
// products cost half.
constexpr int kTermTokens = 64;

// What a bf16 rounding of v leaves (0 where the rounding is infinite or NaN).
MOE_DEV f32x4 low_terms(const f32x4 v) {
    f32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float h = (float)(__bf16)v[q];
        r[q] = fabsf(h) <= 3.4028234e38f ? v[q] - h : 0.0f;
    }
    return r;
}

// dz = dy * f'(z + bias), rounded to bf16 for the two gradient products (and its low terms, when
// lo is given); the bias gradient sums the unrounded values.  dz rows are ldz >= C wide (a multiple of 8); the columns past C are
// written as zeros, so the products may read whole 16-byte chunks.
struct EpiLinearBwd {
    static constexpr bool kPair = false, kColSum = true;
    const float *bias;
    const uint16_t *dy;
    uint16_t *dz, *lo;    // lo: NULL, or the low terms' rows
    int C, ldz, fn;
    float *cs;            // column-sum partials [..][csld] or NULL
    int csld;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4, f32x4 &ca, f32x4 &) const {
        const size_t o = (size_t)r * C + c;
        f32x4 g = {0.f, 0.f, 0.f, 0.f};
        if ((C & 3) == 0) {
            if (bias) a += *(const f32x4 *)(bias + c);
            g = load4_bf16(dy + o);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c + q < C) {
                    a[q] += bias ? bias[c + q] : 0.0f;
                    g[q] = bf16_to_f32(dy[o + q]);
                }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f, d;
            act_fd(fn, a[q], f, d);
            ca[q] = c + q < C ? g[q] * d : 0.0f;
        }
        const bool tail = c + 4 >= C && c + 4 < ldz;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        store4_bf16(dz + (size_t)r * ldz + c, ca);
        if (tail) store4_bf16(dz + (size_t)r * ldz + c + 4, zero);
        if (lo) {
            store4_bf16(lo + (size_t)r * ldz + c, low_terms(ca));
            if (tail) store4_bf16(lo + (size_t)r * ldz + c + 4, zero);
        }
    }
};

// dg = dh * u * f'(g), du = dh * f(g), rounded to bf16 into [R][2][C] (one row of 2C values, so
// the weight-gradient product sees one matrix; low terms as above); h = f(g) * u when asked for.
// C is a multiple of 8.
struct EpiGateBwd {
    static constexpr bool kPair = true, kColSum = true;
    const float *bg, *bu;
    const void *dh;       // bf16 or float32
    uint16_t *dgu, *lo;
    void *h;              // [R][C] or NULL
    int C, fn, dh_f32, h_f32;
    float *cs;            // column-sum partials [..][csld], csld = 2C, or NULL
    int csld;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4 b, f32x4 &ca, f32x4 &cb) const {
        if (bg) a += *(const f32x4 *)(bg + c);
        if (bu) b += *(const f32x4 *)(bu + c);
        grads(r, c, a, b, ca, cb);
    }
    MOE_DEV void grads(int r, int c, f32x4 g, f32x4 u, f32x4 &ca, f32x4 &cb) const {
        const size_t o = (size_t)r * C + c;
        const f32x4 d = dh_f32 ? *(const f32x4 *)((const float *)dh + o) : load4_bf16((const uint16_t *)dh + o);
        f32x4 hv;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f, df;
            act_fd(fn, g[q], f, df);
            ca[q] = d[q] * u[q] * df;
            cb[q] = d[q] * f;
            hv[q] = f * u[q];
        }
        store4_bf16(dgu + (size_t)r * 2 * C + c, ca);
        store4_bf16(dgu + (size_t)r * 2 * C + C + c, cb);
        if (lo) {
            store4_bf16(lo + (size_t)r * 2 * C + c, low_terms(ca));
            store4_bf16(lo + (size_t)r * 2 * C + C + c, low_terms(cb));
        }
        if (h) {
            if (h_f32) *(f32x4 *)((float *)h + o) = hv;
            else store4_bf16((uint16_t *)h + o, hv);
        }
    }
};

// The product itself: rows below rows0 to out0, the others to out1 (the gate's and up's gradients).
// C is a multiple of 8.
struct EpiStore {
    static constexpr bool kPair = false, kColSum = false;
    void *out0, *out1;
    int rows0, C, f32;
    float *cs = nullptr;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4, f32x4 &, f32x4 &) const {
        void *p = r < rows0 ? out0 : out1;
        const size_t o = (size_t)(r < rows0 ? r : r - rows0) * C + c;
        if (f32) *(f32x4 *)((float *)p + o) = a;
        else store4_bf16((uint16_t *)p + o, a);
    }
};

// float32 partial results of one part of a split sum: [split][mats][R][ld], ld = C rounded up to 4.
template <bool PAIR>
struct EpiPartial {
    static constexpr bool kPair = PAIR, kColSum = false;
    float *part;          // this part's first matrix
    size_t plane;         // R * ld
    int ld;
    float *cs = nullptr;
    MOE_DEV void apply(int r, int c, f32x4 a, f32x4 b, f32x4 &, f32x4 &) const {
        *(f32x4 *)(part + (size_t)r * ld + c) = a;
        if constexpr (PAIR) *(f32x4 *)(part + plane + (size_t)r * ld + c) = b;
    }
};

// ------------------------------------------------------------------ products

// The three operand layouts (rows operand, columns operand).
enum DenseForm { kFormNT = 0, kFormNN = 1, kFormTN = 2 };

// One product: out[r][c] = sum over segments s and k < K of rowop_s(r, k) * colop_s(c, k).
//   NT: rowop(r, k) = rp[s][r * ldr + k], colop(c, k) = cp[s][c * ldc + k]
//   NN: rowop as NT,                      colop(c, k) = cp[s][k * ldc + c]
//   TN: rowop(r, k) = rp[s][k * ldr + r], colop as NN
// Pair (NT, one segment): cp[0] and cp[1] are two matrices of C rows, both products wanted.
// Segments let one launch sum over the terms of a split operand, or over gate and up.  With
// terms > 1 the rows operand holds R / terms output rows of each term, one term's rows after the
// other's, and the results of a row's terms are added up (not for pairs).
// Every row start is 16-byte aligned; K (contiguous operands) and the widths of strided operands
// are multiples of 8.
struct DenseProduct {
    const uint16_t *rp[3];
    const uint16_t *cp[3];
    int nseg, terms, K;
    int R, C;             // R: rows of the rows operand, all terms
    int ldr, ldc;
    int rcols;            // TN: readable columns of a row-operand row (>= R, a multiple of 8)
};

// How a product runs: tile shape, parts of the sum.
struct DensePlan {
    int cfg;              // 0: 256 x 256, 1: 128 x 128, 2: 64 x 128 tiles
    int split;            // parts of the sum (1: the epilogue runs in the product kernel)
    int tr, tc;           // tiles along rows and columns
    int steps;            // 64-value steps of the sum, all segments
    int cs_rows;          // column-sum partial rows the launch writes
};
DensePlan dense_plan(int form, bool pair, int R, int C, int K, int nseg, int terms = 1);
size_t dense_plan_bytes(const DensePlan &pl, bool pair, int R, int C, int terms = 1);   // partial results

moe_status dense_linear_product(const DenseProduct &p, const DensePlan &pl, const EpiLinear &e, float *part, hipStream_t s);
moe_status dense_gate_product(const DenseProduct &p, const DensePlan &pl, const EpiGate &e, float *part, hipStream_t s);
moe_status dense_linear_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiLinearBwd &e, float *part,
                                    hipStream_t s);
moe_status dense_gate_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiGateBwd &e, float *part,
                                  hipStream_t s);
moe_status dense_nn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, hipStream_t s);
moe_status dense_tn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, hipStream_t s);

// Sum the parts of a split product and run the epilogue on the sums (dense_aux.hip).
template <class Epi>
moe_status dense_finish(int parts, const Epi &e, const float *part, int R, int C, hipStream_t s);
constexpr int kFinishRows = 2;    // rows per workgroup of the finish and saved-activation kernels

// out[c] = sum over rows of part[row][c] (column-sum partials), in row order.
moe_status dense_colsum_reduce(const float *part, int rows, int ld, int C0, float *out0, float *out1, hipStream_t s);
// Column-sum partials of a bf16 matrix [R][C]: part [ceil(R / kColRows)][csld].
constexpr int kColRows = 64;
moe_status dense_colsum(const uint16_t *a, int R, int C, float *part, int csld, hipStream_t s);
// Gradients of the gated product from saved pre-activations [2][R][C] (dense_aux.hip).
moe_status dense_gate_bwd_saved(const EpiGateBwd &e, const uint16_t *pre, int R, hipStream_t s);
// float32 rows [n] -> three bf16 planes [3][n] whose sum is the value exactly.
moe_status dense_split3(const float *x, uint16_t *planes, size_t n, hipStream_t s);
// Rows of C bf16 values -> rows of ld >= C, the tail zero.
moe_status dense_pad_rows(const uint16_t *x, uint16_t *out, int R, int C, int ld, hipStream_t s);

// Up to kGemvTokens tokens: one pass over the weights on the vector ALU (dense_gemv.hip).
constexpr int kGemvTokens = 8;
moe_status dense_linear_gemv(const void *x, bool x_f32, const uint16_t *w, int T, int n, int k, const EpiLinear &e,
                             hipStream_t s);
moe_status dense_gate_gemv(const void *x, const uint16_t *wg, const uint16_t *wu, int T, int f, int d, const EpiGate &e,
                           hipStream_t s);

// MXFP8 (mxfp8.hip)
moe_status mxfp8_dequant_launch(size_t rows, int cols, const uint8_t *codes, const uint8_t *scales, void *out, bool f32,
                                hipStream_t s);

}  // namespace moe
