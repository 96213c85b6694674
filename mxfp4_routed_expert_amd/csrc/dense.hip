// Entry points of the dense bf16 layers: argument checks, plans, workspaces and launches.
#include "dense.h"

namespace moe {

namespace {

constexpr int kCUs = 256;            // the plan is a pure function of the sizes (workspace queries run anywhere)

// Tile shapes (dense_gemm.h) and their costs: us of a 64-value step of all the workgroups a CU holds, and
// of a tile's start and end.  Fitted to 2900 timings of the four products over 16 to 4096 rows, 1000 to
// 7168 columns and sums of 32 to 7168 values, operands not in the caches, every shape and split forced in
// turn; there the plan's choice takes 0.5% longer than the fastest on average (weight gradients 2.3%) and
// 15% at most (with the 256 x 128 tile, timed on 26 shapes, and streaming stores: 1% and 7%).  A weight gradient's sum is short and
// its result large, hence costs of its own.
struct Tile {
    int br, bc, wr, per_cu;
    double step, tile;
};
struct TileCosts {
    Tile t[kTiles];
    double one;                             // a step with one workgroup on a CU, relative to a full CU
    double finish;                          // us of the launch that sums partial results
    double part;                            // their bytes written or read in a us (partly in the caches)
};
constexpr TileCosts kCosts = {{{256, 256, 2, 1, 1.41, 4.7},
                               {128, 128, 2, 2, 1.05, 4.9},
                               {64, 128, 1, 2, 0.57, 6.2},
                               {128, 128, 2, 1, 0.53, 4.3},
                               {128, 128, 2, 4, 0.0, 0.0},
                               {256, 128, 4, 1, 0.77, 5.2}},
                              0.43, 4.9, 9.0e6};
constexpr TileCosts kWeightGradCosts = {{{256, 256, 2, 1, 1.26, 5.7},
                                         {128, 128, 2, 2, 0.91, 3.0},
                                         {64, 128, 1, 2, 0.0, 0.0},
                                         {128, 128, 2, 1, 0.0, 0.0},
                                         {128, 128, 2, 4, 1.65, 4.6},
                                         {256, 128, 4, 1, 0.70, 5.9}},
                                        0.30, 2.0, 6.7e6};
constexpr int kMaxSplit = 8;

}  // namespace

// The tile shape and split with the least estimated time.  Whole rounds of tiles over the CUs run
// unsplit; the tiles left over either make a round of their own or are split so that their parts fill
// one, at the cost of the partial results' traffic and a second launch.
DensePlan dense_plan(int form, bool pair, int R, int C, int K, int nseg, int terms) {
    DensePlan best = {};
    double best_t = 1e30;
    const int steps = (K > 0 ? (K + 63) / 64 : 1) * nseg;     // (a sum of no values is one step of zeros)
    const int mats = pair ? 2 : 1;
    const TileCosts &costs = form == kFormTN ? kWeightGradCosts : kCosts;
    for (int cfg = 0; cfg < kTiles; ++cfg) {
        // S cannot hold a strided rows operand; D's extra step in flight does not pay over the tokens' sums, which W takes
        if (form == kFormTN ? cfg == kTileS || cfg == kTileD : cfg == kTileW) continue;
        const Tile &t = costs.t[cfg];
        const int tr = (R + t.br - 1) / t.br, tc = (C + t.bc / mats - 1) / (t.bc / mats);
        const int64_t tiles = (int64_t)tr * tc, slots = (int64_t)kCUs * t.per_cu;
        // rounds of n workgroups of s steps each; a last round with fewer workgroups per CU runs faster
        auto rounds = [&](int64_t n, int s) {
            if (n <= 0) return 0.0;
            const int64_t k = (n + slots - 1) / slots, last = (n - (k - 1) * slots + kCUs - 1) / kCUs;
            const double share = t.per_cu == 1 ? 1.0 : costs.one + (1.0 - costs.one) * (double)last / t.per_cu;
            return ((double)(k - 1) + share) * (s * t.step + t.tile);
        };
        for (int split = 1; split <= kMaxSplit; ++split) {
            if (split > 1 && split * 4 > steps) break;
            const int64_t full = split * terms == 1 ? tiles : (terms > 1 ? 0 : tiles / slots * slots), tail = tiles - full;
            if (split > 1 && (tail == 0 || tail * split > slots)) break;
            double us = rounds(full, steps) + rounds(tail * split, (steps + split - 1) / split);
            const size_t bytes = (size_t)tail * split * t.br * t.bc * sizeof(float);
            if (tail > 0) {
                const double live = (double)(R < t.br ? R : t.br) / t.br;
                us += costs.finish + bytes * live * 2.0 / costs.part;
            }
            if (us < best_t) {
                best_t = us;
                best = DensePlan{cfg, tr, tc, (int)full, split, steps,
                                 tail > 0 ? (R / terms + t.br - 1) / t.br * (t.br / kFinishRows) : tr * t.wr, bytes};
            }
        }
    }
    return best;
}

namespace {

// Consecutive 256-byte-aligned pieces of a workspace; with a NULL base only the size counts.
struct Carve {
    char *base;
    size_t at = 0;
    template <class T = void>
    T *take(size_t bytes) {
        char *q = base ? base + at : nullptr;
        at = align_up(at + bytes, 256);
        return (T *)q;
    }
};

// Jobs that run in order beside the products of a call: those that no product is left for run at once, the others
// beside as late a product as they can (the weight gradient's small tiles leave more room beside them).
struct Sides {
    DenseSide job[2] = {};
    int n = 0, at = 0;
    void add(const DenseSide &j) { job[n++] = j; }
    moe_status keep(int products, hipStream_t s) {
        for (; n - at > products; ++at) MOE_TRY(dense_side_launch(job[at], s));
        return MOE_OK;
    }
    DenseSide next(int products) { return n - at >= products ? job[at++] : DenseSide{}; }   // `products` left with this one
};

bool fn_ok(int fn) { return fn >= MOE_FN_NONE && fn <= MOE_FN_RELU; }
template <class... P>
bool aligned16(P... p) {
    return (((uintptr_t)p | ...) & 15) == 0;
}
bool fits31(int64_t a, int64_t b) { return a * b < INT32_MAX; }

moe_status check_ws(const char *who, const void *ws, size_t have, size_t need) {
    if (need == 0) return MOE_OK;
    if (ws == nullptr || have < need) {
        set_error("%s: workspace of %zu bytes needed, got %zu", who, need, ws ? have : (size_t)0);
        return MOE_ERR_WORKSPACE;
    }
    MOE_REQUIRE(aligned16(ws), "%s: the workspace must be 16-byte aligned", who);
    return MOE_OK;
}

// ------------------------------------------------------------------ linear

moe_status check_linear(const char *who, const moe_linear_desc *d, bool backward) {
    MOE_REQUIRE(d != nullptr, "%s: NULL descriptor", who);
    MOE_REQUIRE(d->T >= 0 && d->n > 0 && d->kdim > 0 && d->kdim % 8 == 0,
                "%s: need T >= 0, n > 0, kdim > 0 and a multiple of 8 (T=%d n=%d kdim=%d)", who, d->T, d->n, d->kdim);
    MOE_REQUIRE(fn_ok(d->fn), "%s: unknown activation %d", who, d->fn);
    if (backward) {
        MOE_REQUIRE(d->x_dtype >= MOE_DT_BF16 && d->x_dtype <= MOE_DT_MXFP8, "%s: unknown x_dtype %d", who, d->x_dtype);
        MOE_REQUIRE(d->dx_dtype == MOE_DT_BF16 || d->dx_dtype == MOE_DT_F32, "%s: unknown dx_dtype %d", who, d->dx_dtype);
        MOE_REQUIRE(d->x_dtype != MOE_DT_MXFP8 || d->kdim % 32 == 0, "%s: MXFP8 kdim = %d is not a multiple of 32", who,
                    d->kdim);
    } else {
        MOE_REQUIRE(d->x_dtype == MOE_DT_BF16 || d->x_dtype == MOE_DT_F32, "%s: unknown x_dtype %d", who, d->x_dtype);
        MOE_REQUIRE(d->y_dtype == MOE_DT_BF16 || d->y_dtype == MOE_DT_F32, "%s: unknown y_dtype %d", who, d->y_dtype);
    }
    // (where few rows are kept as several terms these form one operand, whose tile offsets are 32-bit bytes: three of x for a
    // product on the matrix cores, two of dz behind an activation)
    const bool few = d->T <= kTermTokens, act = d->fn != MOE_FN_NONE;
    const int64_t x_rows = (int64_t)d->T * (few && d->x_dtype == MOE_DT_F32 && (backward ? act : d->T > kGemvTokens) ? 3 : 1);
    const int64_t z_rows = (int64_t)d->T * (few && backward && act ? 2 : 1);
    MOE_REQUIRE(fits31(z_rows, (int64_t)d->n + 8) && fits31(d->n, d->kdim) && fits31(x_rows, d->kdim), "%s: sizes overflow int32",
                who);
    return MOE_OK;
}

struct LinearWs {
    DensePlan plan;
    int terms, nseg;
    uint16_t *planes;
    float *part;
    size_t bytes;
};
LinearWs linear_ws(const moe_linear_desc *d, void *base) {
    LinearWs w = {};
    if (d->T <= kGemvTokens) return w;
    const bool f32 = d->x_dtype == MOE_DT_F32;
    Carve c{(char *)base};
    w.terms = f32 && d->T <= kTermTokens ? 3 : 1;
    w.nseg = f32 && w.terms == 1 ? 3 : 1;
    w.plan = dense_plan(kFormNT, false, d->T * w.terms, d->n, d->kdim, w.nseg, w.terms);
    w.planes = c.take<uint16_t>(f32 ? (size_t)3 * d->T * d->kdim * 2 : 0);
    w.part = c.take<float>(w.plan.part_bytes);
    w.bytes = c.at;
    return w;
}

// The sums of a linear layer's backward pass.  Up to kTermTokens tokens dz = dy f' is kept as two terms;
// a float32 x is three terms for z and its two leading ones (2^-16, and 2^-15 where dz's second term meets the
// first alone) for dw, whose result is bf16.
// The gradient products' partial results.  An input gradient's are summed beside the weight gradient's W tiles
// where it takes those (four workgroups a CU, the sum's fit between; larger tiles would have to end first): the
// weight gradient then has a place of its own for its parts.  61 tokens, 6144 x 2 x 2048: 46.9 -> 42.5 us, and
// 40.2 with the column sums there too.
template <class Ws>
void carve_parts(Carve &c, Ws &w, size_t first) {
    const size_t bx = w.px.part_bytes, bw = w.pw.part_bytes;
    w.sum_later = w.pw.cfg == kTileW;
    size_t n = first > bx ? first : bx;
    if (!w.sum_later && n < bw) n = bw;
    w.part = c.template take<float>(n);
    w.part_w = w.sum_later ? c.template take<float>(bw) : w.part;
}

struct LinearBwdWs {
    DensePlan pz, px, pw;
    int zterms, zseg;            // recomputed z: x's terms as rows or as segments
    int dterms;                  // terms of dz
    int wseg;                    // (dz term, x term) products in dw
    uint16_t *x, *dz;
    float *cs, *part, *part_w;
    bool sum_later;
    int ldz, csld, cs_rows;
    bool own_dz;
    size_t bytes;
};
LinearBwdWs linear_bwd_ws(const moe_linear_desc *d, void *base) {
    LinearBwdWs w = {};
    Carve c{(char *)base};
    const int T = d->T, n = d->n, k = d->kdim;
    const bool act = d->fn != MOE_FN_NONE, f32 = d->x_dtype == MOE_DT_F32, few = T <= kTermTokens;
    w.ldz = (n + 7) & ~7;
    w.csld = w.ldz;
    w.own_dz = act || w.ldz != n;          // dy itself serves as dz otherwise
    w.zterms = f32 && few ? 3 : 1;
    w.zseg = f32 && !few ? 3 : 1;
    w.dterms = act && few ? 2 : 1;
    w.wseg = (f32 ? 2 : 1) + (w.dterms - 1);
    w.pz = dense_plan(kFormNT, false, T * w.zterms, n, k, w.zseg, w.zterms);
    w.px = dense_plan(kFormNN, false, T * w.dterms, k, n, 1, w.dterms);
    w.pw = dense_plan(kFormTN, false, n, k, T, w.wseg);
    w.cs_rows = act ? w.pz.cs_rows : (T + kColRows - 1) / kColRows;
    w.x = c.take<uint16_t>(f32 ? (size_t)3 * T * k * 2 : (d->x_dtype == MOE_DT_MXFP8 ? (size_t)T * k * 2 : 0));
    w.dz = c.take<uint16_t>(w.own_dz ? (size_t)w.dterms * T * w.ldz * 2 : 0);
    w.cs = c.take<float>((size_t)w.cs_rows * w.csld * 4);
    size_t part = act ? w.pz.part_bytes : 0;
    carve_parts(c, w, part);
    w.bytes = c.at;
    return w;
}

// ------------------------------------------------------------------ gated

moe_status check_gateup(const char *who, const moe_gateup_desc *d, bool backward) {
    MOE_REQUIRE(d != nullptr, "%s: NULL descriptor", who);
    MOE_REQUIRE(d->T >= 0 && d->d_model > 0 && d->d_model % 8 == 0 && d->d_ff > 0 && d->d_ff % 8 == 0,
                "%s: need T >= 0 and d_model, d_ff positive multiples of 8 (T=%d d_model=%d d_ff=%d)", who, d->T, d->d_model,
                d->d_ff);
    MOE_REQUIRE(fn_ok(d->fn), "%s: unknown activation %d", who, d->fn);
    if (backward) {
        MOE_REQUIRE(d->x_dtype == MOE_DT_BF16 || d->x_dtype == MOE_DT_MXFP8, "%s: x_dtype %d is neither bf16 nor MXFP8", who,
                    d->x_dtype);
        MOE_REQUIRE(d->dh_dtype == MOE_DT_BF16 || d->dh_dtype == MOE_DT_F32, "%s: unknown dh_dtype %d", who, d->dh_dtype);
        MOE_REQUIRE(d->x_dtype != MOE_DT_MXFP8 || d->d_model % 32 == 0, "%s: MXFP8 d_model = %d is not a multiple of 32", who,
                    d->d_model);
    } else {
        MOE_REQUIRE(d->x_dtype == MOE_DT_BF16, "%s: x must be bf16 (x_dtype %d)", who, d->x_dtype);
    }
    MOE_REQUIRE(d->h_dtype == MOE_DT_BF16 || d->h_dtype == MOE_DT_F32, "%s: unknown h_dtype %d", who, d->h_dtype);
    const int64_t g_rows = (int64_t)d->T * (d->T <= kTermTokens && backward ? 2 : 1);     // (terms of dg and du)
    MOE_REQUIRE(fits31(g_rows, 2 * (int64_t)d->d_ff) && fits31(d->d_model, 2 * (int64_t)d->d_ff) &&
                    fits31(d->T, d->d_model),
                "%s: sizes overflow int32", who);
    return MOE_OK;
}

struct GateWs {
    DensePlan plan;
    float *part;
    size_t bytes;
};
GateWs gate_ws(const moe_gateup_desc *d, void *base) {
    GateWs w = {};
    if (d->T <= kGemvTokens) return w;
    Carve c{(char *)base};
    w.plan = dense_plan(kFormNT, true, d->T, d->d_ff, d->d_model, 1);
    w.part = c.take<float>(w.plan.part_bytes);
    w.bytes = c.at;
    return w;
}

struct GateBwdWs {
    DensePlan pg, px, pw;
    int terms;                   // of dg and du
    uint16_t *x, *dgu;
    float *cs, *part, *part_w;
    bool sum_later;
    int cs_rows;                 // with recomputed pre-activations
    int cs_rows_saved;
    size_t bytes;
};
GateBwdWs gate_bwd_ws(const moe_gateup_desc *d, void *base) {
    GateBwdWs w = {};
    Carve c{(char *)base};
    const int f = d->d_ff;
    w.pg = dense_plan(kFormNT, true, d->T, f, d->d_model, 1);
    w.terms = d->T <= kTermTokens ? 2 : 1;
    const int xr = d->T * w.terms;
    w.px = dense_plan(kFormNN, false, xr, d->d_model, f, 2, w.terms);
    w.pw = dense_plan(kFormTN, false, 2 * f, d->d_model, d->T, w.terms);
    w.cs_rows = w.pg.cs_rows;
    w.cs_rows_saved = (d->T + kSavedRows - 1) / kSavedRows;
    w.x = c.take<uint16_t>(d->x_dtype == MOE_DT_MXFP8 ? (size_t)d->T * d->d_model * 2 : 0);
    w.dgu = c.take<uint16_t>((size_t)xr * 2 * f * 2);
    w.cs = c.take<float>((size_t)(w.cs_rows > w.cs_rows_saved ? w.cs_rows : w.cs_rows_saved) * 2 * f * 4);
    size_t part = w.pg.part_bytes;
    carve_parts(c, w, part);
    w.bytes = c.at;
    return w;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_dense_linear_workspace(const moe_linear_desc *d) {
    return check_linear("moe_dense_linear_workspace", d, false) == MOE_OK ? linear_ws(d, nullptr).bytes : 0;
}

extern "C" moe_status moe_dense_linear(const moe_linear_desc *d, const void *x, const void *w, const float *bias,
                                       const void *residual, void *y, void *ws, size_t ws_bytes, moe_stream stream) {
    clear_error();
    MOE_TRY(check_linear("moe_dense_linear", d, false));
    if (d->T == 0) return MOE_OK;
    MOE_REQUIRE(x && w && y, "moe_dense_linear: NULL x, w or y");
    MOE_REQUIRE(aligned16(x, w, bias, residual, y), "moe_dense_linear: tensors must be 16-byte aligned");
    const LinearWs b = linear_ws(d, ws);
    MOE_TRY(check_ws("moe_dense_linear", ws, ws_bytes, b.bytes));
    hipStream_t s = (hipStream_t)stream;
    const bool f32 = d->x_dtype == MOE_DT_F32;
    EpiLinear e;
    e.bias = bias;
    e.res = residual;
    e.y = y;
    e.C = d->n;
    e.fn = d->fn;
    e.y_f32 = d->y_dtype == MOE_DT_F32;
    if (d->T <= kGemvTokens) return dense_linear_gemv(x, f32, (const uint16_t *)w, d->T, d->n, d->kdim, e, s);
    const size_t plane = (size_t)d->T * d->kdim;
    if (f32) MOE_TRY(dense_split3((const float *)x, b.planes, plane, s));
    DenseProduct p = {};
    p.nseg = b.nseg;
    p.terms = b.terms;
    for (int i = 0; i < p.nseg; ++i) {
        p.rp[i] = f32 ? b.planes + i * plane : (const uint16_t *)x;
        p.cp[i] = (const uint16_t *)w;
    }
    p.K = p.ldr = p.ldc = d->kdim;
    p.R = d->T * b.terms;
    p.C = d->n;
    return dense_linear_product(p, b.plan, e, b.part, s);
}

extern "C" size_t moe_dense_linear_backward_workspace(const moe_linear_desc *d) {
    return check_linear("moe_dense_linear_backward_workspace", d, true) == MOE_OK ? linear_bwd_ws(d, nullptr).bytes : 0;
}

extern "C" moe_status moe_dense_linear_backward(const moe_linear_desc *d, const void *dy, const void *x,
                                                const uint8_t *x_scales, const void *w, const float *bias, void *dx,
                                                void *dw, float *dbias, void *ws, size_t ws_bytes, moe_stream stream) {
    clear_error();
    MOE_TRY(check_linear("moe_dense_linear_backward", d, true));
    MOE_REQUIRE(dx || dw || dbias || d->T == 0, "moe_dense_linear_backward: no gradient asked for");
    const bool act = d->fn != MOE_FN_NONE, mx = d->x_dtype == MOE_DT_MXFP8;
    const bool need_x = act || dw, need_w = act || dx;
    if (d->T > 0) {
        MOE_REQUIRE(dy && (x || !need_x) && (w || !need_w), "moe_dense_linear_backward: NULL dy, x or w");
        MOE_REQUIRE(!(mx && need_x && !x_scales), "moe_dense_linear_backward: MXFP8 x without x_scales");
    }
    MOE_REQUIRE(aligned16(dy, x, w, bias, dx, dw, dbias), "moe_dense_linear_backward: tensors must be 16-byte aligned");
    const LinearBwdWs b = linear_bwd_ws(d, ws);
    MOE_TRY(check_ws("moe_dense_linear_backward", ws, ws_bytes, b.bytes));
    hipStream_t s = (hipStream_t)stream;
    const int T = d->T, n = d->n, k = d->kdim;
    const bool f32 = d->x_dtype == MOE_DT_F32;
    const size_t xplane = f32 ? (size_t)T * k : 0;
    const uint16_t *xb = (const uint16_t *)x;
    if (T > 0 && need_x && (mx || f32)) {
        if (mx) MOE_TRY(mxfp8_dequant_launch((size_t)T, k, (const uint8_t *)x, x_scales, b.x, false, s));
        else MOE_TRY(dense_split3((const float *)x, b.x, xplane, s));
        xb = b.x;
    }
    const uint16_t *dz = (const uint16_t *)dy;
    const size_t dzplane = (size_t)T * b.ldz;
    if (T > 0 && act) {
        DenseProduct p = {};
        p.nseg = b.zseg;
        p.terms = b.zterms;
        for (int i = 0; i < p.nseg; ++i) {
            p.rp[i] = xb + i * xplane;
            p.cp[i] = (const uint16_t *)w;
        }
        p.K = p.ldr = p.ldc = k;
        p.R = T * b.zterms;
        p.C = n;
        EpiLinearBwd e;
        e.bias = bias;
        e.dy = dz;
        e.dz = b.dz;
        e.lo = b.dterms > 1 ? b.dz + dzplane : nullptr;
        e.C = n;
        e.ldz = b.ldz;
        e.fn = d->fn;
        e.cs = dbias ? b.cs : nullptr;
        e.csld = b.csld;
        MOE_TRY(dense_linear_bwd_product(p, b.pz, e, b.part, s));
        dz = b.dz;
    } else if (T > 0) {
        if (b.own_dz && (dx || dw)) {
            MOE_TRY(dense_pad_rows(dz, b.dz, T, n, b.ldz, s));
            dz = b.dz;
        }
    }
    // the bias gradient's column sums ride along with the products: the sums of dy where dz is dy, then their total
    Sides sides;
    if (dbias && !act && T > 0) sides.add(DenseSide{kSideSum, T, n, b.csld, dy, b.cs, nullptr});
    if (dbias) sides.add(DenseSide{kSideReduce, T > 0 ? b.cs_rows : 0, n, b.csld, b.cs, dbias, nullptr});
    MOE_TRY(sides.keep((dx && T > 0) + (dw != nullptr), s));
    DenseLater later = {};
    if (dx && T > 0) {
        DenseProduct p = {};
        p.nseg = 1;
        p.terms = b.dterms;
        p.rp[0] = dz;
        p.cp[0] = (const uint16_t *)w;
        p.K = n;
        p.ldr = b.ldz;
        p.ldc = k;
        p.R = T * b.dterms;
        p.C = k;
        EpiStore e;
        e.out0 = dx;
        e.out1 = nullptr;
        e.rows0 = T;
        e.C = k;
        e.f32 = d->dx_dtype == MOE_DT_F32;
        MOE_TRY(dense_nn_product(p, b.px, e, b.part, sides.next(1 + (dw != nullptr)), b.sum_later && dw ? &later : nullptr, s));
    }
    if (dw) {
        // dz's leading term with x's one or two leading terms, then dz's low term with x's first
        DenseProduct p = {};
        p.terms = 1;
        p.nseg = b.wseg;
        for (int i = 0; i < p.nseg; ++i) {
            const bool lo = b.dterms > 1 && i == p.nseg - 1;
            p.rp[i] = lo ? dz + dzplane : dz;
            p.cp[i] = lo ? xb : xb + i * xplane;
        }
        p.K = T;
        p.ldr = b.ldz;
        p.ldc = k;
        p.R = n;
        p.C = k;
        p.rcols = b.ldz;
        EpiStore e;
        e.out0 = dw;
        e.out1 = nullptr;
        e.rows0 = n;
        e.C = k;
        e.f32 = 0;
        MOE_TRY(dense_tn_product(p, b.pw, e, b.part_w, sides.next(1), later, s));
    }
    return MOE_OK;
}

extern "C" size_t moe_dense_gateup_workspace(const moe_gateup_desc *d) {
    return check_gateup("moe_dense_gateup_workspace", d, false) == MOE_OK ? gate_ws(d, nullptr).bytes : 0;
}

extern "C" moe_status moe_dense_gateup(const moe_gateup_desc *d, const void *x, const void *w_gate, const void *w_up,
                                       const float *b_gate, const float *b_up, void *h, void *pre, void *ws,
                                       size_t ws_bytes, moe_stream stream) {
    clear_error();
    MOE_TRY(check_gateup("moe_dense_gateup", d, false));
    if (d->T == 0) return MOE_OK;
    MOE_REQUIRE(x && w_gate && w_up && h, "moe_dense_gateup: NULL x, w_gate, w_up or h");
    MOE_REQUIRE(aligned16(x, w_gate, w_up, b_gate, b_up, h, pre), "moe_dense_gateup: tensors must be 16-byte aligned");
    const GateWs b = gate_ws(d, ws);
    MOE_TRY(check_ws("moe_dense_gateup", ws, ws_bytes, b.bytes));
    EpiGate e;
    e.bg = b_gate;
    e.bu = b_up;
    e.h = h;
    e.pre = (uint16_t *)pre;
    e.plane = (size_t)d->T * d->d_ff;
    e.C = d->d_ff;
    e.fn = d->fn;
    e.h_f32 = d->h_dtype == MOE_DT_F32;
    hipStream_t s = (hipStream_t)stream;
    const uint16_t *xb = (const uint16_t *)x, *wg = (const uint16_t *)w_gate, *wu = (const uint16_t *)w_up;
    if (d->T <= kGemvTokens) return dense_gate_gemv(xb, wg, wu, d->T, d->d_ff, d->d_model, e, s);
    DenseProduct p = {};
    p.nseg = p.terms = 1;
    p.rp[0] = xb;
    p.cp[0] = wg;
    p.cp[1] = wu;
    p.K = p.ldr = p.ldc = d->d_model;
    p.R = d->T;
    p.C = d->d_ff;
    return dense_gate_product(p, b.plan, e, b.part, s);
}

extern "C" size_t moe_dense_gateup_backward_workspace(const moe_gateup_desc *d) {
    return check_gateup("moe_dense_gateup_backward_workspace", d, true) == MOE_OK ? gate_bwd_ws(d, nullptr).bytes : 0;
}

extern "C" moe_status moe_dense_gateup_backward(const moe_gateup_desc *d, const void *dh, const void *x,
                                                const uint8_t *x_scales, const void *w_gate, const void *w_up,
                                                const float *b_gate, const float *b_up, const void *pre, void *dx,
                                                void *dw_gate, void *dw_up, float *db_gate, float *db_up, void *h,
                                                void *ws, size_t ws_bytes, moe_stream stream) {
    clear_error();
    MOE_TRY(check_gateup("moe_dense_gateup_backward", d, true));
    MOE_REQUIRE(!dw_gate == !dw_up && !db_gate == !db_up,
                "moe_dense_gateup_backward: the gate's and up's gradients come together");
    MOE_REQUIRE(dx || dw_gate || db_gate || h || d->T == 0, "moe_dense_gateup_backward: no result asked for");
    const bool mx = d->x_dtype == MOE_DT_MXFP8, need_x = !pre || dw_gate;
    if (d->T > 0) {
        MOE_REQUIRE(dh && w_gate && w_up && (x || !need_x), "moe_dense_gateup_backward: NULL dh, x, w_gate or w_up");
        MOE_REQUIRE(!(mx && need_x && !x_scales), "moe_dense_gateup_backward: MXFP8 x without x_scales");
    }
    MOE_REQUIRE(aligned16(dh, x, w_gate, w_up, b_gate, b_up, pre, dx, dw_gate, dw_up, db_gate, db_up, h),
                "moe_dense_gateup_backward: tensors must be 16-byte aligned");
    const GateBwdWs b = gate_bwd_ws(d, ws);
    MOE_TRY(check_ws("moe_dense_gateup_backward", ws, ws_bytes, b.bytes));
    hipStream_t s = (hipStream_t)stream;
    const int T = d->T, f = d->d_ff, dm = d->d_model;
    const uint16_t *xb = (const uint16_t *)x, *wg = (const uint16_t *)w_gate, *wu = (const uint16_t *)w_up;
    if (T > 0 && mx && need_x) {
        MOE_TRY(mxfp8_dequant_launch((size_t)T, dm, (const uint8_t *)x, x_scales, b.x, false, s));
        xb = b.x;
    }
    if (T > 0) {
        EpiGateBwd e;
        e.bg = b_gate;
        e.bu = b_up;
        e.dh = dh;
        e.dgu = b.dgu;
        e.lo = b.terms > 1 ? b.dgu + (size_t)T * 2 * f : nullptr;
        e.h = h;
        e.dh_f32 = d->dh_dtype == MOE_DT_F32;
        e.h_f32 = d->h_dtype == MOE_DT_F32;
        e.C = f;
        e.fn = d->fn;
        e.cs = db_gate ? b.cs : nullptr;
        e.csld = 2 * f;
        if (pre) {
            MOE_TRY(dense_gate_bwd_saved(e, (const uint16_t *)pre, T, s));
        } else {
            DenseProduct p = {};
            p.nseg = p.terms = 1;
            p.rp[0] = xb;
            p.cp[0] = wg;
            p.cp[1] = wu;
            p.K = p.ldr = p.ldc = dm;
            p.R = T;
            p.C = f;
            MOE_TRY(dense_gate_bwd_product(p, b.pg, e, b.part, s));
        }
    }
    Sides sides;
    if (db_gate)
        sides.add(DenseSide{kSideReduce, T == 0 ? 0 : (pre ? b.cs_rows_saved : b.cs_rows), f, 2 * f, b.cs, db_gate, db_up});
    MOE_TRY(sides.keep((dx && T > 0) + (dw_gate != nullptr), s));
    DenseLater later = {};
    if (dx && T > 0) {
        DenseProduct p = {};
        p.nseg = 2;
        p.terms = b.terms;
        p.rp[0] = b.dgu;
        p.rp[1] = b.dgu + f;
        p.cp[0] = wg;
        p.cp[1] = wu;
        p.K = f;
        p.ldr = 2 * f;
        p.ldc = dm;
        p.R = T * b.terms;
        p.C = dm;
        EpiStore e;
        e.out0 = dx;
        e.out1 = nullptr;
        e.rows0 = T;
        e.C = dm;
        e.f32 = 0;
        MOE_TRY(dense_nn_product(p, b.px, e, b.part, sides.next(1 + (dw_gate != nullptr)), b.sum_later && dw_gate ? &later : nullptr, s));
    }
    if (dw_gate) {
        DenseProduct p = {};
        p.terms = 1;
        p.nseg = b.terms;
        for (int i = 0; i < p.nseg; ++i) {
            p.rp[i] = b.dgu + (size_t)i * T * 2 * f;
            p.cp[i] = xb;
        }
        p.K = T;
        p.ldr = 2 * f;
        p.ldc = dm;
        p.R = 2 * f;
        p.C = dm;
        p.rcols = 2 * f;
        EpiStore e;
        e.out0 = dw_gate;
        e.out1 = dw_up;
        e.rows0 = f;
        e.C = dm;
        e.f32 = 0;
        MOE_TRY(dense_tn_product(p, b.pw, e, b.part_w, sides.next(1), later, s));
    }
    return MOE_OK;
}
