// moe_fp8_linear: the product of block-128 FP8 operands, its argument checks and its plan.
// Few rows stream the weights (fp8_stream.hip; up to 16 short rows in one launch: 2048 x 7168 for one row 7.5 to 8.0 us); above, rows to
// codes, tiles, and the sum of parts where there are few tiles.
#include <algorithm>

#include "fp8.h"

namespace moe {
namespace {

// Rows of a tile and parts of the sum for R x N over Kb blocks: the least of this estimate, in microseconds, of a launch on 256
// compute units.  A step is one block of a tile: 1.55 us for 256 rows with every unit at work (measured from long sums, 1.3 with
// E8M0 scales), 0.6 of that with few.  A tile's start and end are 4 us and, when all write at once, 15 for 256 rows.  The tiles
// of a last, short round are halved or quartered.  Parts are written, and read by a second launch, at 6.5 TB/s.  Measured
// (us, x as codes; [rows, parts], what is taken first): 333 x 2368 x 7168 [64,4] 25.0, [128,4] 24.9, [128,8] 23.7, [256,6] 25.0,
// [64,3] 29.2; 1021 x 6144 x 2048 [128,1] 21.9, [256,1] 22.0, [192,1] 27.2, [64,1] 29.2, [128,2] 37.1; 1021 x 2048 x 6144 [128,3] 29.2,
// [256,2] 27.0, [128,2] 27.2, [256,1] 33.8; 2048 x 2368 x 7168 [128,1] 51.7, [192,2] 48.7, [256,1] 52.1, [64,1] 72.8; 2048 x 7168 x
// 2368 [256,1] 41.1, [128,1] 48.8, [192,1] 50.7; 7168 x 2368 x 2048 [192,1] 51.8, [256,1] 53.8, [128,1] 62.7; 4096 x 7168 x 7168 [256,1]
// 208, [192,1] 235, [128,1] 286; 200 x 2048 x 7168 [64,4] 24.7, [128,6] 21.3; 128 x 7168 x 2048 [64,1] 22.9, [128,3] 18.6.  So the choice is
// within 8 % of the best of these, but for few tiles, whose steps and starts take longer than the estimate says (tiles of 64 rows
// do not take turns): there more parts would take 14 to 19 % less.
using Plan = Fp8Plan;
Plan plan_of(int R, int N, int Kb) {
    constexpr int G = 256;
    const int NT = (N + 255) / 256;
    Plan best = {256, 1};
    double least = 1e30;
    for (int bt = 64; bt <= 256; bt += 64)
        for (int split = 1; split <= 16 && split <= Kb; ++split) {
            const int64_t items = (int64_t)((R + bt - 1) / bt) * NT * split, tail = items % G;
            const int f = tail > 0 && 4 * tail <= G ? std::min(4, bt / 64) : tail > 0 && 2 * tail <= G ? std::min(2, bt / 64) : 1;
            const double rounds = (double)(items / G) + (tail > 0 ? 1.0 / f : 0.0);
            const double busy = items >= G ? 1.0 : (double)items / G;
            const double step = (bt == 256 ? 1.55 : bt == 192 ? 1.3 : bt == 128 ? 1.0 : 0.8) * (0.6 + 0.4 * busy);
            const int steps = (Kb + split - 1) / split;
            double t = std::max(rounds, items < G ? 1.0 : rounds) * (steps * step + 4.0 + 15.0 * bt / 256 * busy);
            if (split > 1) t += 3.0 + (double)R * N * split * 8.0 / 6.5e6;
            if (t < least) {
                least = t;
                best = {bt, split};
            }
        }
    return best;
}

struct Layout {
    size_t xq = 0, xs = 0, part = 0, bytes = 0;
    Plan plan = {256, 1};
};
// Few rows stream the weights.  Every workgroup of 16 columns or more reads all of x, so it depends on the product's size from 17
// rows on.  Both sides, us (streamed; tiles as plan_of gives them; tiles of the best number of parts, where it gives another): 2048 x 7168,
// 17 rows 14.2, 18.7, 64 rows 25.8, 22.6; 7168 x 2048, 64 rows 20.9, 24.8, 19.4; 6144 x 4096, 32 rows 22.4, 22.0, 18.5, 48 rows
// 30.9, 23.2, 20.0; 7168 x 7168, 17 rows 23.2, 27.1, 22.4; 512 x 512, 64 rows 7.0, 11.9; 131072 x 1024, 17 rows 50.5, 43.3.  The border
// lies where the first two meet, 64 short wide rows apart.
bool few_rows(const moe_fp8_linear_desc *d) {
    return d->T <= kFp8RowsMax || (d->T <= 64 && (int64_t)d->T * d->n * d->kdim <= (int64_t)1 << 30);
}
// They take codes as they are, and quantise few enough values themselves.
bool direct_x(const moe_fp8_linear_desc *d) {
    return few_rows(d) && (d->x_dtype == MOE_DT_FP8 || fp8_rows_fit(d->T, d->kdim));
}
Layout layout_of(const moe_fp8_linear_desc *d) {
    Layout l;
    if (direct_x(d)) return l;                            // (quantised on the way, no parts)
    const int Kb = fp8_blocks(d->kdim);
    l.plan = fp8_linear_plan(d);
    size_t off = 0;
    auto take = [&](size_t b) {
        const size_t at = off;
        off += align_up(b, 256);
        return at;
    };
    if (d->x_dtype != MOE_DT_FP8) {
        l.xq = take((size_t)d->T * d->kdim);
        l.xs = take((size_t)d->T * Kb);
    }
    if (l.plan.split > 1) l.part = take((size_t)l.plan.split * d->T * d->n * sizeof(float));
    l.bytes = off;
    return l;
}

moe_status check_desc(const moe_fp8_linear_desc *d, const char *who) {
    MOE_REQUIRE(d != nullptr, "%s: desc is NULL", who);
    MOE_REQUIRE(d->T >= 0 && d->n >= 1 && d->kdim >= 16 && d->kdim % 16 == 0,
                "%s: need T >= 0, n >= 1 and kdim a positive multiple of 16 (T=%d n=%d kdim=%d)", who, d->T, d->n, d->kdim);
    MOE_REQUIRE(d->x_dtype == MOE_DT_BF16 || d->x_dtype == MOE_DT_F32 || d->x_dtype == MOE_DT_FP8, "%s: unknown x_dtype %d", who,
                d->x_dtype);
    MOE_REQUIRE(d->y_dtype == MOE_DT_BF16 || d->y_dtype == MOE_DT_F32, "%s: unknown y_dtype %d", who, d->y_dtype);
    MOE_REQUIRE(d->w_scale >= MOE_FP8_SCALE_F32 && d->w_scale <= MOE_FP8_SCALE_E8M0_ROW, "%s: unknown w_scale %d", who, d->w_scale);
    const int64_t T = d->T, n = d->n, k = d->kdim;
    MOE_REQUIRE(T * k < INT32_MAX && n * k < INT32_MAX && T * n < INT32_MAX, "%s: sizes overflow int32", who);
    return MOE_OK;
}

}  // namespace

Fp8Plan fp8_linear_plan(const moe_fp8_linear_desc *d) {
    return few_rows(d) ? Plan{0, 1} : plan_of(d->T, d->n, fp8_blocks(d->kdim));
}
}  // namespace moe

using namespace moe;

extern "C" size_t moe_fp8_linear_workspace(const moe_fp8_linear_desc *d) {
    if (check_desc(d, "moe_fp8_linear_workspace") != MOE_OK || d->T == 0) return 0;
    return layout_of(d).bytes;
}

extern "C" moe_status moe_fp8_linear(const moe_fp8_linear_desc *d, const void *x, const uint8_t *x_scales, const uint8_t *w,
                                     const void *w_scales, const void *residual, void *y, void *ws, size_t ws_bytes, moe_stream stream) {
    clear_error();
    const char *who = "moe_fp8_linear";
    MOE_TRY(check_desc(d, who));
    if (d->T == 0) return MOE_OK;
    MOE_REQUIRE(x && w && w_scales && y, "%s: NULL x, w, w_scales or y", who);
    MOE_REQUIRE((x_scales != nullptr) == (d->x_dtype == MOE_DT_FP8), "%s: x_scales belong to MOE_DT_FP8 codes, and to them only", who);
    MOE_REQUIRE((((uintptr_t)x | (uintptr_t)w | (uintptr_t)y | (uintptr_t)residual) & 15) == 0,
                "%s: x, w, y and residual must be 16-byte aligned", who);
    MOE_REQUIRE(d->w_scale != MOE_FP8_SCALE_F32 || ((uintptr_t)w_scales & 3) == 0, "%s: float32 scales must be 4-byte aligned", who);
    const Layout l = layout_of(d);
    if (l.bytes && (!ws || ws_bytes < l.bytes)) {
        set_error("%s: workspace of %zu bytes needed, %zu given", who, l.bytes, ws ? ws_bytes : (size_t)0);
        return MOE_ERR_WORKSPACE;
    }
    MOE_REQUIRE(((uintptr_t)ws & 15) == 0, "%s: the workspace must be 16-byte aligned", who);
    hipStream_t s = (hipStream_t)stream;
    unsigned char *base = (unsigned char *)ws;
    Fp8Product p = {};
    p.x = (const uint8_t *)x;
    p.xs = x_scales;
    if (d->x_dtype != MOE_DT_FP8 && direct_x(d)) {
        p.x_values = x;
        p.x_f32 = d->x_dtype == MOE_DT_F32;
    } else if (d->x_dtype != MOE_DT_FP8) {
        MOE_TRY(fp8_quantize_rows_launch(d->T, d->kdim, x, d->x_dtype == MOE_DT_F32, base + l.xq, base + l.xs, s));
        p.x = base + l.xq;
        p.xs = base + l.xs;
    }
    p.n_x = d->T;
    p.k = 1;
    p.w[0] = w;
    p.ws[0] = w_scales;
    p.w_scale = d->w_scale;
    p.E = 1;
    p.N = d->n;
    p.K = d->kdim;
    p.Kb = fp8_blocks(d->kdim);
    p.R = d->T;
    p.y = y;
    p.residual = residual;
    p.y_f32 = d->y_dtype == MOE_DT_F32;
    p.part = (float *)(base + l.part);
    p.bt = l.plan.bt;
    p.split = l.plan.split;
    if (few_rows(d)) return fp8_rows16_launch(p, false, s, who);
    return fp8_product_launch(p, false, s, who);
}
