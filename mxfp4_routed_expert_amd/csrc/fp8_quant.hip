// Block-128 FP8 codes: rows of activations and gradients (blocks along the row, along the columns, or both
// from one read) and weights (128 x 128 blocks), with transposed codes for the products that sum over the
// other axis; and the values back.
//
// All of it is bound by HBM: one read, and one byte a value for each form written.  4096 x 7168 bf16 to rows of codes 19 us
// (4.5 TB/s); 2048 x 7168 both ways 17 to 19 us (3.1 to 3.5 TB/s: one tile a workgroup, all of them resident, so that the reads come first
// and the writes after, and what is written is of a size that a plain fill takes at 4.8 TB/s); a weight of 7168 x 2368 with its
// transpose 16 to 18 us (4.0 TB/s).  2048 x 2368 both ways takes 9 to 10 us (2.2 TB/s: 304 tiles, little over one a CU).
// 4096 x 7168 codes back to bf16 18 us, to float32 31 (4.8 TB/s).
#include "fp8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool F32>
MOE_DEV void load8(const void *x, size_t at, float (&v)[8]) {          // 8 values from element `at`
    if constexpr (F32) {
        const f32x4 a = *(const f32x4 *)((const float *)x + at), b = *(const f32x4 *)((const float *)x + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 a = *(const u32x4 *)((const uint16_t *)x + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 f = bf16x2_to_f32x2(a[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// 16 lanes a block, 8 values a lane; the blocks of a row follow each other.  rows_live: rows from it on stay as they are (or NULL).
template <bool F32>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(const void *__restrict__ x, size_t blocks, int nb, int cols,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                            const int32_t *__restrict__ rows_live) {
    const size_t b = ((size_t)blockIdx.x * kThreads + threadIdx.x) >> 4;
    if (b >= blocks) return;
    const size_t row = b / (unsigned)nb;
    if (rows_live && (int64_t)row >= *rows_live) return;
    const int c = (int)(b - row * nb) * kFp8Block + 8 * (threadIdx.x & 15);
    const bool live = c < cols;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8<F32>(x, row * cols + c, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, fp8_magnitude(v[i]));
    m = fp8_max16(m);
    const int X = fp8_exponent(m);
    const float inv = fp8_inverse(X);
    if (live)
        *(u32x2 *)(codes + row * cols + c) = u32x2{fp8_codes4(v[0], v[1], v[2], v[3], inv), fp8_codes4(v[4], v[5], v[6], v[7], inv)};
    if ((threadIdx.x & 15) == 0) scales[b] = (uint8_t)(X + 127);
}

// A 128 x 128 tile a workgroup, an 8 x 4 part a thread: thread (tid / 32, tid % 32) holds rows 8 (tid / 32) ..,
// columns 4 (tid % 32) ...  Eight rows of one column are 8 neighbouring bytes of the transposed codes; they go
// through LDS so that a column's 128 bytes leave as one line.
//   WEIGHT: one scale for the tile; else one for each row (over its 128 columns) and one for each column.
// codes [rows][cols] or NULL; codes_t [cols][ld] or NULL, ld = rows rounded up to 16, zeros past the last row.
// The largest magnitudes are taken over all values first; only a tile with NaN or infinities looks at each value again.
constexpr int kTileThreads = 512;
template <bool F32>
MOE_DEV void load4(const void *x, size_t at, float (&v)[4]) {
    if constexpr (F32) {
        const f32x4 a = *(const f32x4 *)((const float *)x + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i];
    } else {
        const u32x2 a = *(const u32x2 *)((const uint16_t *)x + at);
        const f32x2 l = bf16x2_to_f32x2(a[0]), h = bf16x2_to_f32x2(a[1]);
        v[0] = l.x;
        v[1] = l.y;
        v[2] = h.x;
        v[3] = h.y;
    }
}

template <bool F32, bool WEIGHT>
__global__ __launch_bounds__(kTileThreads) void fp8_tile_kernel(const void *__restrict__ x, int rows, int cols, int ld, int nbr, int nbc,
                                                                uint8_t *__restrict__ codes, void *__restrict__ scales,
                                                                uint8_t *__restrict__ codes_t, void *__restrict__ scales_t, int f32_scales) {
    constexpr int kWaves = kTileThreads / kWave;
    __shared__ __align__(16) uint8_t tile[128][128];       // 16-byte piece p of column c at p ^ ((c >> 2) & 7)
    __shared__ uint32_t cmax[kWaves][128];
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int tr = blockIdx.y, tc = blockIdx.x;
    const int r0 = tr * 128 + 8 * (tid >> 5), cl = 4 * (tid & 31), c0 = tc * 128 + cl;
    // (every load at a valid place, unconditionally: behind a branch each waits for its own value before the next goes out)
    float v[8][4];
    const bool in = c0 < cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) load4<F32>(x, (size_t)min(r0 + i, rows - 1) * cols + (in ? c0 : 0), v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = in && r0 + i < rows ? v[i][j] : 0.0f;
    uint32_t rm[8], cm[4];
    bool finite;
    auto maxima = [&](auto all) __attribute__((always_inline)) {
        auto mag = [&](float f) __attribute__((always_inline)) { return decltype(all)::value ? fp8_abs_bits(f) : fp8_magnitude(f); };
#pragma unroll
        for (int i = 0; i < 8; ++i) rm[i] = max(max(mag(v[i][0]), mag(v[i][1])), max(mag(v[i][2]), mag(v[i][3])));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cm[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) cm[j] = max(cm[j], mag(v[i][j]));
        }
    };
    maxima(std::true_type{});
    {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, cm[j]);
        finite = __syncthreads_and(m < kFp8Inf);
    }
    if (!finite) maxima(std::false_type{});
    if constexpr (WEIGHT) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
        m = fp8_max16(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
        if (lane == 0) cmax[wave][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = max(m, cmax[w][0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) rm[i] = m;
#pragma unroll
        for (int j = 0; j < 4; ++j) cm[j] = m;
    } else {
        if (codes) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                rm[i] = fp8_max16(rm[i]);
                rm[i] = max(rm[i], (uint32_t)__shfl_xor((int)rm[i], 16, kWave));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cm[j] = max(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32, kWave));
            if (lane < 32) cmax[wave][4 * lane + j] = cm[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) cm[j] = max(cm[j], cmax[w][cl + j]);
    }
    auto put = [&](void *s, size_t at, uint32_t m) __attribute__((always_inline)) {
        const int X = fp8_exponent(m);
        // (2^X of a float32 scale: the smallest X is 2^-127, a subnormal)
        if (f32_scales) ((float *)s)[at] = e8m0_to_f32((uint32_t)(X + 127));
        else ((uint8_t *)s)[at] = (uint8_t)(X + 127);
    };
    if constexpr (WEIGHT) {
        if (tid == 0) {
            if (scales) put(scales, (size_t)tr * nbc + tc, rm[0]);
            if (scales_t) put(scales_t, (size_t)tc * nbr + tr, rm[0]);
        }
    } else {
        if (scales && (tid & 31) == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < rows) put(scales, (size_t)(r0 + i) * nbc + tc, rm[i]);
        }
        if (scales_t && tid < 32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < cols) put(scales_t, (size_t)(c0 + j) * nbr + tr, cm[j]);
        }
    }
    auto write = [&](auto all) __attribute__((always_inline)) {
        constexpr bool F = decltype(all)::value;
        if (codes && c0 < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < rows)
                    *(uint32_t *)(codes + (size_t)(r0 + i) * cols + c0) = fp8_codes4<F>(v[i][0], v[i][1], v[i][2], v[i][3], fp8_inverse(fp8_exponent(rm[i])));
        }
        if (codes_t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float inv = fp8_inverse(fp8_exponent(cm[j]));
                *(u32x2 *)&tile[cl + j][(8 * (tid >> 5)) ^ (16 * ((tid & 31) & 7))] = u32x2{fp8_codes4<F>(v[0][j], v[1][j], v[2][j], v[3][j], inv),
                                                               fp8_codes4<F>(v[4][j], v[5][j], v[6][j], v[7][j], inv)};
            }
        }
    };
    if (finite) write(std::true_type{});
    else write(std::false_type{});
    if (!codes_t) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 64 * i + (tid >> 3), r = 16 * (tid & 7);
        if (tc * 128 + c < cols && tr * 128 + r < ld)
            *(u32x4 *)(codes_t + (size_t)(tc * 128 + c) * ld + tr * 128 + r) = *(const u32x4 *)&tile[c][r ^ (16 * ((c >> 2) & 7))];
    }
}

// code * 2^(s - 127), 8 values a lane
template <bool F32>
__global__ __launch_bounds__(kThreads) void fp8_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                               size_t units, int cols, int nb, void *__restrict__ out) {
    const size_t u = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;
    const size_t row = 8 * u / (unsigned)cols;
    const int c = (int)(8 * u - row * cols);
    const u32x2 q = ((const u32x2 *)codes)[u];
    const float sc = e8m0_to_f32(scales[row * nb + (c >> 7)]);
    float v[8];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const f32x2 a = fp8x2_to_f32x2<false>(q[d]), b = fp8x2_to_f32x2<true>(q[d]);
        v[4 * d] = a.x * sc;
        v[4 * d + 1] = a.y * sc;
        v[4 * d + 2] = b.x * sc;
        v[4 * d + 3] = b.y * sc;
    }
    if constexpr (F32) {
        ((f32x4 *)out)[2 * u] = f32x4{v[0], v[1], v[2], v[3]};
        ((f32x4 *)out)[2 * u + 1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            o[i] = __builtin_bit_cast(uint32_t, b);
        }
        ((u32x4 *)out)[u] = o;
    }
}

// (a lane's access is 8 values; an operand's rows are multiples of 16)
moe_status check_sizes(const char *who, int32_t rows, int32_t cols, int32_t dtype, int32_t unit) {
    MOE_REQUIRE(rows >= 0 && cols > 0 && cols % unit == 0,
                "%s: need rows >= 0 and cols a positive multiple of %d (rows=%d cols=%d)", who, unit, rows, cols);
    MOE_REQUIRE(dtype == MOE_DT_BF16 || dtype == MOE_DT_F32, "%s: unknown dtype %d", who, dtype);
    MOE_REQUIRE(((int64_t)rows + 15) * cols < INT32_MAX, "%s: sizes overflow int32", who);
    return MOE_OK;
}

}  // namespace

moe_status fp8_quantize_rows_launch(int rows, int cols, const void *x, bool f32, uint8_t *codes, uint8_t *scales, hipStream_t s,
                                    const int32_t *live) {
    const int nb = fp8_blocks(cols);
    const size_t blocks = (size_t)rows * nb;
    const dim3 grid((unsigned)((blocks * 16 + kThreads - 1) / kThreads));
    if (f32) hipLaunchKernelGGL(fp8_rows_kernel<true>, grid, dim3(kThreads), 0, s, x, blocks, nb, cols, codes, scales, live);
    else hipLaunchKernelGGL(fp8_rows_kernel<false>, grid, dim3(kThreads), 0, s, x, blocks, nb, cols, codes, scales, live);
    return launch_check("fp8_rows_kernel");
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_fp8_quantize(int32_t rows, int32_t cols, const void *x, int32_t x_dtype, uint8_t *codes, uint8_t *scales,
                                       uint8_t *codes_t, uint8_t *scales_t, moe_stream stream) {
    clear_error();
    const char *who = "moe_fp8_quantize";
    MOE_TRY(check_sizes(who, rows, cols, x_dtype, 8));
    MOE_REQUIRE((codes == nullptr) == (scales == nullptr) && (codes_t == nullptr) == (scales_t == nullptr),
                "%s: codes and their scales come together or not at all", who);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes || codes_t, "%s: NULL codes and codes_t: nothing is asked for", who);
    MOE_REQUIRE(x != nullptr, "%s: NULL x", who);
    MOE_REQUIRE((((uintptr_t)x | (uintptr_t)codes | (uintptr_t)codes_t) & 15) == 0, "%s: values and codes must be 16-byte aligned", who);
    hipStream_t s = (hipStream_t)stream;
    if (!codes_t) return fp8_quantize_rows_launch(rows, cols, x, x_dtype == MOE_DT_F32, codes, scales, s);
    const int nbr = fp8_blocks(rows), nbc = fp8_blocks(cols), ld = (int)align_up(rows, 16);
    MOE_REQUIRE(nbr <= 65535, "%s: rows = %d above 65535 blocks", who, rows);
    const dim3 grid(nbc, nbr);
    if (x_dtype == MOE_DT_F32)
        hipLaunchKernelGGL((fp8_tile_kernel<true, false>), grid, dim3(kTileThreads), 0, s, x, rows, cols, ld, nbr, nbc, codes, scales,
                           codes_t, scales_t, 0);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<false, false>), grid, dim3(kTileThreads), 0, s, x, rows, cols, ld, nbr, nbc, codes, scales,
                           codes_t, scales_t, 0);
    return launch_check(who);
}

extern "C" moe_status moe_fp8_quantize_weight(int32_t n, int32_t kdim, const void *w, int32_t w_dtype, int32_t w_scale, uint8_t *codes,
                                              void *scales, uint8_t *codes_t, void *scales_t, moe_stream stream) {
    clear_error();
    const char *who = "moe_fp8_quantize_weight";
    MOE_TRY(check_sizes(who, n, kdim, w_dtype, 16));
    MOE_REQUIRE(w_scale == MOE_FP8_SCALE_F32 || w_scale == MOE_FP8_SCALE_E8M0, "%s: w_scale = %d is no block scale's type", who, w_scale);
    MOE_REQUIRE((codes == nullptr) == (scales == nullptr) && (codes_t == nullptr) == (scales_t == nullptr),
                "%s: codes and their scales come together or not at all", who);
    if (n == 0) return MOE_OK;
    MOE_REQUIRE(codes || codes_t, "%s: NULL codes and codes_t: nothing is asked for", who);
    MOE_REQUIRE(w != nullptr, "%s: NULL w", who);
    MOE_REQUIRE((((uintptr_t)w | (uintptr_t)codes | (uintptr_t)codes_t) & 15) == 0, "%s: values and codes must be 16-byte aligned", who);
    const int f32s = w_scale == MOE_FP8_SCALE_F32;
    MOE_REQUIRE(!f32s || (((uintptr_t)scales | (uintptr_t)scales_t) & 3) == 0, "%s: float32 scales must be 4-byte aligned", who);
    hipStream_t s = (hipStream_t)stream;
    const int nbr = fp8_blocks(n), nbc = fp8_blocks(kdim), ld = (int)align_up(n, 16);
    MOE_REQUIRE(nbr <= 65535, "%s: n = %d above 65535 blocks", who, n);
    const dim3 grid(nbc, nbr);
    if (w_dtype == MOE_DT_F32)
        hipLaunchKernelGGL((fp8_tile_kernel<true, true>), grid, dim3(kTileThreads), 0, s, w, n, kdim, ld, nbr, nbc, codes, scales, codes_t,
                           scales_t, f32s);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<false, true>), grid, dim3(kTileThreads), 0, s, w, n, kdim, ld, nbr, nbc, codes, scales, codes_t,
                           scales_t, f32s);
    return launch_check(who);
}

extern "C" moe_status moe_fp8_dequant(int32_t rows, int32_t cols, const uint8_t *codes, const uint8_t *scales, void *out,
                                      int32_t out_dtype, moe_stream stream) {
    clear_error();
    const char *who = "moe_fp8_dequant";
    MOE_TRY(check_sizes(who, rows, cols, out_dtype, 8));
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && out, "%s: NULL pointer argument", who);
    MOE_REQUIRE((((uintptr_t)out | (uintptr_t)codes) & 15) == 0, "%s: values and codes must be 16-byte aligned", who);
    const size_t units = (size_t)rows * cols / 8;
    const dim3 grid((unsigned)((units + kThreads - 1) / kThreads));
    hipStream_t s = (hipStream_t)stream;
    if (out_dtype == MOE_DT_F32)
        hipLaunchKernelGGL(fp8_dequant_kernel<true>, grid, dim3(kThreads), 0, s, codes, scales, units, cols, fp8_blocks(cols), out);
    else
        hipLaunchKernelGGL(fp8_dequant_kernel<false>, grid, dim3(kThreads), 0, s, codes, scales, units, cols, fp8_blocks(cols), out);
    return launch_check(who);
}
