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
// results that no kernel of the call reads: past the L2's lines (see EpiStore)
MOE_DEV void stream4_bf16(uint16_t *p, const f32x4 v) {
    __builtin_nontemporal_store(u32x2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])}, (u32x2 *)p);
}
MOE_DEV f32x4 load4_bf16(const uint16_t *p) {
    const u32x2 w = *(const u32x2 *)p;
    const f32x2 a = bf16x2_to_f32x2(w[0]), b = bf16x2_to_f32x2(w[1]);
    return f32x4{a.x, a.y, b.x, b.y};
}
MOE_DEV uint16_t bf16_bits(float v) { return (uint16_t)(pack2_bf16(v, 0.0f) & 0xffffu); }

// ------------------------------------------------------------------ activations
// f(z) and f'(z) in float32, on the hardware's exp2 and reciprocal (each within 1 ulp).
//   silu       z s(z), s the logistic function          f' = s (1 + z (1 - s))
//   gelu       z Phi(z), Phi the normal distribution     f' = Phi + z exp(-z^2/2) / sqrt(2 pi)
//   gelu_tanh  0.5 z (1 + tanh q) = z s(2q), q = sqrt(2/pi) (z + 0.044715 z^3): the logistic form
//              has no cancellation for negative z         f' = s + z s (1 - s) 2q'
//   relu       max(z, 0)                                 f' = [z > 0]; NaN stays NaN in both
// 1 - s is taken as e s with e = exp(-t), so it keeps its relative accuracy where s rounds to 1; there
// e is held below infinity (as is z^2 in q'), so that a product with a zero stays zero for every finite z.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = 1.5957691216057308f;           // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

MOE_DEV float gelu_arg(float z) { return z * (kGeluA + (kGeluA * kGeluB) * z * z); }
MOE_DEV float exp_neg(float t) { return __builtin_amdgcn_exp2f(-kLog2e * t); }
MOE_DEV float rcp(float v) { return __builtin_amdgcn_rcpf(v); }

// erfc(x) / 2 for x = |z| / sqrt 2, given E = exp(-z^2 / 2): E times a polynomial in t = 1 / (1 + 0.4 x)
// (least-squares fit of erfc(x) exp(x^2) / 2 with equalised relative error, 1.3e-7 over x >= 0).  Phi is that for
// negative z and 1 minus it otherwise: no cancellation on either side, and the value keeps its relative accuracy
// as far out as it is a normal number (z about -13).  A result rounded to bf16 takes it too: bf16 has float32's exponents, so
// the tail is stored, and a gated h is scaled by u first (4093 x 7168 x 2048 with bias: 107 us, 103 with a polynomial logit
// that holds to z = -5; a fit of six terms for bf16, 2^-18 of the value, measured the same 107).
MOE_DEV float phi_of(float z, float E) {
    const float t = rcp(fmaf(0.28284271f, fabsf(z), 1.0f));
    float q = 0.025137422606348991f;
    q = fmaf(q, t, -0.09147657454013824f);
    q = fmaf(q, t, 0.08458571135997772f);
    q = fmaf(q, t, -0.0028414966072887182f);
    q = fmaf(q, t, 0.07073443382978439f);
    q = fmaf(q, t, 0.08426576852798462f);
    q = fmaf(q, t, 0.10392211377620697f);
    q = fmaf(q, t, 0.11283475160598755f);
    q = fmaf(q, t, 0.11283793300390244f);
    q *= t * E;
    return z < 0.0f ? q : 1.0f - q;
}
MOE_DEV float gauss(float z) { return __builtin_amdgcn_exp2f((-0.5f * kLog2e) * z * z); }

template <int U>
MOE_DEV void act_rows(int fn, f32x4 (&a)[U]) {
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) a[u][q] = f(a[u][q]);
    };
    if (fn == MOE_FN_SILU) each([](float z) { return z * rcp(1.0f + exp_neg(z)); });
    else if (fn == MOE_FN_GELU) each([](float z) { return z * phi_of(z, gauss(z)); });
    else if (fn == MOE_FN_GELU_TANH) each([](float z) { return z * rcp(1.0f + exp_neg(gelu_arg(z))); });
    else if (fn == MOE_FN_RELU) each([](float z) { return z < 0.0f ? 0.0f : z; });
}

// f(z) in z's place, f'(z) in d
template <int U>
MOE_DEV void act_grad_rows(int fn, f32x4 (&z)[U], f32x4 (&d)[U]) {
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v = z[u][q], g;
                f(v, g);
                z[u][q] = v;
                d[u][q] = g;
            }
    };
    auto logistic = [](float &v, float t, float dt, float &g) {
        const float e = exp_neg(t), s = rcp(1.0f + e);
        v *= s;
        g = s + v * (fminf(e, 1e38f) * s * dt);
    };
    if (fn == MOE_FN_SILU) {
        each([&](float &v, float &g) { logistic(v, v, 1.0f, g); });
    } else if (fn == MOE_FN_GELU) {
        each([](float &v, float &g) {
            const float z = v, E = gauss(z), p = phi_of(z, E);
            v = z * p;
            g = p + z * (0.39894228040143268f * E);
        });
    } else if (fn == MOE_FN_GELU_TANH) {
        each([&](float &v, float &g) { logistic(v, gelu_arg(v), kGeluA + (3.0f * kGeluA * kGeluB) * fminf(v * v, 1e30f), g); });
    } else if (fn == MOE_FN_RELU) {
        each([](float &v, float &g) {
            g = v > 0.0f ? 1.0f : (v <= 0.0f ? 0.0f : v);
            v = v < 0.0f ? 0.0f : v;
        });
    } else {
        each([](float &, float &g) { g = 1.0f; });
    }
}

// ------------------------------------------------------------------ epilogues
// rows(cols(c), r, step, R, c, a, b, ca, cb): columns c .. c+3 (c a multiple of 4) of the rows r, r + step,
// ... below R, U of them: a is the product, b the second matrix's when kPair.  The U rows' loads go out
// together and every choice is made once for them.  With kColSum, what the rows add to the column sums
// is added to ca / cb.  Columns at or past C hold nothing and are not stored.  Rows of C columns are
// accessed 4 at a time when C is a multiple of 4 (then every row start is aligned for it), else one at
// a time.
constexpr f32x4 kZero4 = {0.f, 0.f, 0.f, 0.f};

template <int U>
MOE_DEV void load_rows(f32x4 (&v)[U], const void *p, bool f32, int C, int r, int step, int R, int c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t o = (size_t)min(r + u * step, R - 1) * C + c;
        if (f32) v[u] = *(const f32x4 *)((const float *)p + o);
        else v[u] = load4_bf16((const uint16_t *)p + o);
    }
}
template <int U>
MOE_DEV void store_rows(const f32x4 (&v)[U], void *p, bool f32, int ld, int r, int step, int R, int c) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (r + u * step < R) {
            const size_t o = (size_t)(r + u * step) * ld + c;
            if (f32) *(f32x4 *)((float *)p + o) = v[u];
            else store4_bf16((uint16_t *)p + o, v[u]);
        }
}
MOE_DEV f32x4 load_bias(const float *b, int c, int C) {
    f32x4 v = kZero4;
    if (b == nullptr) return v;
    if ((C & 3) == 0) return *(const f32x4 *)(b + c);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (c + q < C) v[q] = b[c + q];
    return v;
}

// y = f(z + bias) + residual
struct EpiLinear {
    static constexpr bool kPair = false, kColSum = false;
    const float *bias;
    const void *res;      // y's type, or NULL; may be y
    void *y;
    int C, fn, y_f32;
    float *cs = nullptr;
    int csld = 0;
    struct Cols {
        f32x4 bias;
    };
    MOE_DEV Cols cols(int c) const { return Cols{load_bias(bias, c, C)}; }
    template <int U>
    MOE_DEV void rows(const Cols &k, int r, int step, int R, int c, f32x4 (&a)[U], f32x4 (&)[U], f32x4 &, f32x4 &) const {
        f32x4 add[U];
        const bool vec = (C & 3) == 0;
        if (res && vec) load_rows(add, res, y_f32, C, r, step, R, c);
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] += k.bias;
        act_rows(fn, a);
        if (vec) {
            if (res) {
#pragma unroll
                for (int u = 0; u < U; ++u) a[u] += add[u];
            }
            store_rows(a, y, y_f32, C, r, step, R, c);
            return;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (r + u * step >= R || c + q >= C) continue;
                const size_t o = (size_t)(r + u * step) * C + c + q;
                float v = a[u][q];
                if (y_f32) {
                    if (res) v += ((const float *)res)[o];
                    ((float *)y)[o] = v;
                } else {
                    if (res) v += bf16_to_f32(((const uint16_t *)res)[o]);
                    ((uint16_t *)y)[o] = bf16_bits(v);
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
    int csld = 0;
    struct Cols {
        f32x4 bg, bu;
    };
    MOE_DEV Cols cols(int c) const { return Cols{load_bias(bg, c, C), load_bias(bu, c, C)}; }
    template <int U>
    MOE_DEV void rows(const Cols &k, int r, int step, int R, int c, f32x4 (&a)[U], f32x4 (&b)[U], f32x4 &, f32x4 &) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] += k.bg;
            b[u] += k.bu;
        }
        if (pre) {
            store_rows(a, pre, false, C, r, step, R, c);
            store_rows(b, pre + plane, false, C, r, step, R, c);
        }
        act_rows(fn, a);
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] *= b[u];
        store_rows(a, h, h_f32, C, r, step, R, c);
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
// lo is given); the bias gradient sums the unrounded values.  dz rows are ldz >= C wide (a multiple
// of 8); the columns past C are written as zeros, so the products may read whole 16-byte chunks.
struct EpiLinearBwd {
    static constexpr bool kPair = false, kColSum = true;
    const float *bias;
    const uint16_t *dy;
    uint16_t *dz, *lo;    // lo: NULL, or the low terms' rows
    int C, ldz, fn;
    float *cs;            // column-sum partials [..][csld] or NULL
    int csld;
    struct Cols {
        f32x4 bias;
    };
    MOE_DEV Cols cols(int c) const { return Cols{load_bias(bias, c, C)}; }
    template <int U>
    MOE_DEV void rows(const Cols &k, int r, int step, int R, int c, f32x4 (&a)[U], f32x4 (&)[U], f32x4 &ca, f32x4 &) const {
        f32x4 g[U], d[U];
        if ((C & 3) == 0) {
            load_rows(g, dy, false, C, r, step, R, c);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    g[u][q] = c + q < C ? bf16_to_f32(dy[(size_t)min(r + u * step, R - 1) * C + c + q]) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] += k.bias;
        act_grad_rows(fn, a, d);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int q = 0; q < 4; ++q) d[u][q] = c + q < C ? g[u][q] * d[u][q] : 0.0f;
            if (r + u * step < R) ca += d[u];
        }
        const bool tail = c + 4 >= C && c + 4 < ldz;
        store_rows(d, dz, false, ldz, r, step, R, c);
        if (lo) {
#pragma unroll
            for (int u = 0; u < U; ++u) d[u] = low_terms(d[u]);
            store_rows(d, lo, false, ldz, r, step, R, c);
        }
        if (tail) {
#pragma unroll
            for (int u = 0; u < U; ++u) d[u] = kZero4;
            store_rows(d, dz, false, ldz, r, step, R, c + 4);
            if (lo) store_rows(d, lo, false, ldz, r, step, R, c + 4);
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
    struct Cols {
        f32x4 bg, bu;
    };
    MOE_DEV Cols cols(int c) const { return Cols{load_bias(bg, c, C), load_bias(bu, c, C)}; }
    template <int U>
    MOE_DEV void rows(const Cols &k, int r, int step, int R, int c, f32x4 (&a)[U], f32x4 (&b)[U], f32x4 &ca, f32x4 &cb) const {
        f32x4 d[U], df[U];
        load_rows(d, dh, dh_f32, C, r, step, R, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] += k.bg;
            b[u] += k.bu;
        }
        act_grad_rows(fn, a, df);
        if (h) {
            f32x4 hv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) hv[u] = a[u] * b[u];
            store_rows(hv, h, h_f32, C, r, step, R, c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            b[u] = d[u] * b[u] * df[u];      // dg
            a[u] = d[u] * a[u];              // du
            if (r + u * step < R) {
                ca += b[u];
                cb += a[u];
            }
        }
        store_rows(b, dgu, false, 2 * C, r, step, R, c);
        store_rows(a, dgu, false, 2 * C, r, step, R, C + c);
        if (lo) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                b[u] = low_terms(b[u]);
                a[u] = low_terms(a[u]);
            }
            store_rows(b, lo, false, 2 * C, r, step, R, c);
            store_rows(a, lo, false, 2 * C, r, step, R, C + c);
        }
    }
};

// The product itself: rows below rows0 to out0, the others to out1 (the gate's and up's gradients).
// C is a multiple of 8.  Gradients leave as streaming stores, which keep the operands in the L2: weight gradients
// of 4096 x 6144 over 1024 tokens 62.7 -> 55.7 us, of 2368 x 7168 over 333 27.3 -> 25.3.  (The forward passes'
// results measured the same either way, partial results and checkpoints worse.)
struct EpiStore {
    static constexpr bool kPair = false, kColSum = false;
    void *out0, *out1;
    int rows0, C, f32;
    float *cs = nullptr;
    int csld = 0;
    struct Cols {};
    MOE_DEV Cols cols(int) const { return Cols{}; }
    template <int U>
    MOE_DEV void rows(const Cols &, int r, int step, int R, int c, f32x4 (&a)[U], f32x4 (&)[U], f32x4 &, f32x4 &) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r + u * step;
            if (row >= R) continue;
            void *p = row < rows0 ? out0 : out1;
            const size_t o = (size_t)(row < rows0 ? row : row - rows0) * C + c;
            if (f32) __builtin_nontemporal_store(a[u], (f32x4 *)((float *)p + o));
            else stream4_bf16((uint16_t *)p + o, a[u]);
        }
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

// How a product runs.  The first `full` tiles (whole rounds of workgroups over the CUs, or all) run with
// the epilogue in the product kernel; the sum of each of the rest is split into `split` parts over
// workgroups of the same launch, whose float32 results a second kernel adds up, in order, and finishes.
enum DenseTile { kTileL, kTileM, kTileS, kTileD, kTileW, kTileB, kTiles };   // the shapes in dense_gemm.h
struct DensePlan {
    int cfg;              // kTile*
    int tr, tc;           // tiles along rows and columns
    int full, split;
    int steps;            // 64-value steps of the sum, all segments; one a segment at least
    int cs_rows;          // column-sum partial rows the launch writes
    size_t part_bytes;    // partial results
};
DensePlan dense_plan(int form, bool pair, int R, int C, int K, int nseg, int terms = 1);

// Order of the tiles: kTileGroup row tiles share each column tile, so the tiles that run together on an XCD
// form a block and share both operands in its L2.
constexpr int kTileGroup = 4;
__host__ __device__ inline void tile_at(int slot, int tr, int tc, int &r, int &c) {
    const int per = kTileGroup * tc, g = slot / per, i = slot - g * per;
    const int n = tr - g * kTileGroup < kTileGroup ? tr - g * kTileGroup : kTileGroup;
    r = g * kTileGroup + i % n;
    c = i / n;
}
__host__ __device__ inline int tile_slot(int r, int c, int tr, int tc) {
    const int g = r / kTileGroup, n = tr - g * kTileGroup < kTileGroup ? tr - g * kTileGroup : kTileGroup;
    return g * kTileGroup * tc + c * n + (r - g * kTileGroup);
}

moe_status dense_linear_product(const DenseProduct &p, const DensePlan &pl, const EpiLinear &e, float *part, hipStream_t s);
moe_status dense_gate_product(const DenseProduct &p, const DensePlan &pl, const EpiGate &e, float *part, hipStream_t s);
moe_status dense_linear_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiLinearBwd &e, float *part,
                                    hipStream_t s);
moe_status dense_gate_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiGateBwd &e, float *part,
                                  hipStream_t s);

// The split tiles' parts.  Partial results: [split tile][part][br][bc], a pair tile's columns gate first.
struct DenseParts {
    const float *part;
    int full, split, terms, tr, tc, rows, C, br, lanes;   // lanes: threads a row, four columns (of each matrix) each
    int wgs;                                              // workgroups that sum them, kFinishRows rows of a tile each
};
constexpr int kFinishRows = 16;   // rows per workgroup there, and per column-sum row of the launch
constexpr int kSavedRows = 2;     // rows per workgroup of the saved pre-activations' gradients
// Workgroups of 256 threads in a launch: a grid holds fewer than 2^32 threads.  The two kernels that the size limits let pass
// it (few tokens of a very wide matrix, saved pre-activations of very many tokens) go out in pieces.
constexpr int kMaxGrid = 1 << 23;

// Sum the parts of the split tiles in order (the same order on every run), the terms of a row after each
// other, and run the epilogue.  Workgroup `wg` of 256 threads takes kFinishRows rows of a tile; LANES threads a
// row, four columns each, and a thread U rows, whose loads of all parts are independent.
constexpr int kFinishThreads = 256;
struct FinishPlace {
    int row, c;                                           // the workgroup's index along the rows; the thread's column
};
template <int LANES, class Epi>
MOE_DEV FinishPlace dense_finish_rows(const DenseParts &q, const Epi &epi, int wg, f32x4 &sa, f32x4 &sb) {
    constexpr int kStep = kFinishThreads / LANES, U = kFinishRows / kStep;
    constexpr int BC = LANES * 4 * (Epi::kPair ? 2 : 1);
    static_assert(U >= 1 && U * kStep == kFinishRows, "whole rows");
    const int blocks = q.br / kFinishRows;
    const int t = wg / blocks, rb = wg - t * blocks;
    int tr, tc;
    if (q.terms == 1) {
        tile_at(q.full + t, q.tr, q.tc, tr, tc);
    } else {                                      // (every tile is split) output rows are the first term's
        tr = t / q.tc;
        tc = t - tr * q.tc;
    }
    const int lane = threadIdx.x % LANES, er = threadIdx.x / LANES;
    const int c = tc * (LANES * 4) + 4 * lane, r = tr * q.br + rb * kFinishRows + er;
    if (c < q.C && r < q.rows) {
        f32x4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = b[u] = kZero4;
        for (int j = 0; j < q.terms; ++j) {
            const float *src[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int rr = min(r + u * kStep, q.rows - 1) + j * q.rows, rt = rr / q.br;
                src[u] = q.part + ((size_t)(tile_slot(rt, tc, q.tr, q.tc) - q.full) * q.split * q.br + (rr - rt * q.br)) * BC +
                         4 * lane;
            }
            for (int s = 0; s < q.split; ++s)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float *p = src[u] + (size_t)s * q.br * BC;
                    a[u] += *(const f32x4 *)p;
                    if constexpr (Epi::kPair) b[u] += *(const f32x4 *)(p + BC / 2);
                }
        }
        epi.rows(epi.cols(c), r, kStep, q.rows, c, a, b, sa, sb);
    }
    return FinishPlace{tr * blocks + rb, c};
}
// ... as a launch (dense_aux.hip), or, for a product's plain results, beside a later product (DenseLater)
template <class Epi>
moe_status dense_finish(const DenseParts &q, const Epi &e, hipStream_t s);
struct DenseLater {
    DenseParts q;                                         // q.wgs == 0: nothing
    EpiStore e;
};

// Column sums, in two steps of a fixed order: partial sums of kColRows rows of a bf16 matrix [rows][C]
// (kSideSum: out0 [ceil(rows / kColRows)][ld]), and the sum of partial rows [rows][ld] (kSideReduce: columns
// below C to out0, the next C to out1 unless it is NULL).  Either runs as its own launch or as further
// workgroups of a gradient product's.
constexpr int kColRows = 32;
enum DenseSideKind { kSideNone, kSideSum, kSideReduce };
struct DenseSide {
    int kind, rows, C, ld;
    const void *in;
    float *out0, *out1;
};
// workgroups of `threads` threads that a job takes
inline int dense_side_wgs(const DenseSide &j, int threads) {
    if (j.kind == kSideSum) return (j.rows + kColRows - 1) / kColRows * ((j.C + 4 * threads - 1) / (4 * threads));
    if (j.kind == kSideReduce) return ((j.out1 ? 2 : 1) * j.C + threads / 4 - 1) / (threads / 4);
    return 0;
}
// workgroup `wg` of a job; lds: 64 floats a wave
template <int THREADS>
MOE_DEV void dense_side_job(const DenseSide &j, int wg, float *lds) {
    if (j.kind == kSideSum) {
        const int n = (j.C + 4 * THREADS - 1) / (4 * THREADS);
        const int rb = wg / n, c = (wg - rb * n) * 4 * THREADS + 4 * threadIdx.x;
        if (c >= j.C) return;
        const uint16_t *a = (const uint16_t *)j.in;
        const int r0 = rb * kColRows, r1 = min(j.rows, r0 + kColRows);
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        if ((j.C & 3) == 0) {
#pragma unroll 8
            for (int r = r0; r < r1; ++r) s += load4_bf16(a + (size_t)r * j.C + c);
        } else {
            for (int r = r0; r < r1; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < j.C) s[q] += bf16_to_f32(a[(size_t)r * j.C + c + q]);
        }
        *(f32x4 *)(j.out0 + (size_t)rb * j.ld + c) = s;
        return;
    }
    // 64 columns for four waves; each sums its share of the rows, the four sums are joined in order (the same one in
    // workgroups of any size)
    constexpr int W = 4;
    static_assert(THREADS % (64 * W) == 0, "whole groups of waves");
    const int lane = lane_id(), w = wave_id() % W, group = wave_id() / W;
    const int C = (j.out1 ? 2 : 1) * j.C, c = (wg * (THREADS / (64 * W)) + group) * 64 + lane;
    const int lo = (int)((int64_t)j.rows * w / W), hi = (int)((int64_t)j.rows * (w + 1) / W);
    const float *part = (const float *)j.in;
    float s = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int r = lo; r < hi; ++r) s += part[(size_t)r * j.ld + c];
    }
    lds += group * (64 * W);
    lds[w * 64 + lane] = s;
    __syncthreads();
    if (w == 0 && c < C) {
        for (int i = 1; i < W; ++i) s += lds[i * 64 + lane];
        if (c < j.C) j.out0[c] = s;
        else j.out1[c - j.C] = s;
    }
}
moe_status dense_side_launch(const DenseSide &j, hipStream_t s);
// later: NULL, or where to leave the sum of the split tiles, for the next product
moe_status dense_nn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, const DenseSide &side,
                            DenseLater *later, hipStream_t s);
// later: what an input gradient left, summed beside this product's W tiles
moe_status dense_tn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, const DenseSide &side,
                            const DenseLater &later, hipStream_t s);
// Gradients of the gated product from saved pre-activations [2][R][C] (dense_aux.hip).
moe_status dense_gate_bwd_saved(const EpiGateBwd &e, const uint16_t *pre, int R, hipStream_t s);
// float32 rows [n] -> three bf16 planes [3][n] whose sum is the value exactly.
moe_status dense_split3(const float *x, uint16_t *planes, size_t n, hipStream_t s);
// Rows of C bf16 values -> rows of ld >= C, the tail zero.
moe_status dense_pad_rows(const uint16_t *x, uint16_t *out, int R, int C, int ld, hipStream_t s);

// Up to kGemvTokens tokens: one pass over the weights on the vector ALU (dense_gemv.hip).  Against the matrix cores,
// which split the sum of so few tiles and need a launch more (float32 rows two, for their terms), us in graphs with weights
// from HBM, forward products of 1 / 4 / 8 tokens:
//   7168 x 2368, bf16 rows      7.7 /  8.8 / 12.3    13.4 / 14.2 / 14.3
//   7168 x 2368, float32 rows   8.0 / 11.4 / 16.3    19.2 / 21.9 / 21.9
//   2048 x 7168, bf16 rows      7.0 /  8.3 /  9.9    17.0 / 17.6 / 17.6
//   2048 x 7168, float32 rows   7.0 / 10.2 / 18.7    24.3 / 30.1 / 30.1
//   gate and up 2048 x 7168    10.9 / 12.2 / 14.6    16.6 / 16.5 / 16.5
//   gate and up 2368 x 7168    13.5 / 15.2 / 18.9    17.2 / 17.1 / 17.2    (the one size where 8 tokens lose)
constexpr int kGemvTokens = 8;
moe_status dense_linear_gemv(const void *x, bool x_f32, const uint16_t *w, int T, int n, int k, const EpiLinear &e,
                             hipStream_t s);
moe_status dense_gate_gemv(const void *x, const uint16_t *wg, const uint16_t *wu, int T, int f, int d, const EpiGate &e,
                           hipStream_t s);

// MXFP8 (mxfp8.hip)
moe_status mxfp8_dequant_launch(size_t rows, int cols, const uint8_t *codes, const uint8_t *scales, void *out, bool f32,
                                hipStream_t s);

}  // namespace moe
