// OCP MXFP8 (E4M3 elements, one E8M0 scale per 32 values): the 8-bit form of an activation kept
// for a backward pass.
//
// Conversion of a block (OCP Microscaling Formats v1.0): X = floor(log2 amax) - 8 (8 = the largest
// E4M3 exponent), kept in [-127, 127]; codes are the nearest E4M3 values of v / 2^X, ties to even,
// saturating at 448.  Both directions move 3 and 1/32 bytes a bf16 value and are bound by HBM: a
// lane takes 8 values, four neighbouring lanes a block.  8192 x 7168 (178 MB): 31.7 us to codes (5.6 TB/s),
// 26.5 back (6.7 TB/s, the codes partly in the last-level cache); 1024 x 6144: 5.5 and 8.5 us.
#include "dense.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool F32>
__global__ __launch_bounds__(kThreads) void mxfp8_quantize_kernel(const void *__restrict__ x, size_t units,
                                                                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const size_t u = (size_t)blockIdx.x * kThreads + threadIdx.x;        // 8 values; units is a multiple of 4
    if (u >= units) return;
    float v[8];
    if constexpr (F32) {
        const f32x4 a = ((const f32x4 *)x)[2 * u], b = ((const f32x4 *)x)[2 * u + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 a = ((const u32x4 *)x)[u];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 f = bf16x2_to_f32x2(a[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    // largest magnitude of the block as an integer: Inf and NaN sort above every finite value
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, kWave));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, kWave));
    const bool bad = m >= 0x7f800000u;
    const int eb = (int)(m >> 23);
    const int X = max(eb - 127 - 8, -127);                               // (zero and subnormal: eb = 0); at most 119
    const float inv = __uint_as_float((uint32_t)(127 - X) << 23);        // 2^-X
    uint32_t c[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(v[4 * d + i] * inv, -448.0f), 448.0f);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        c[d] = bad ? 0u : (uint32_t)w;
    }
    ((u32x2 *)codes)[u] = u32x2{c[0], c[1]};
    if ((u & 3) == 0) scales[u >> 2] = bad ? (uint8_t)255 : (uint8_t)(X + 127);
}

// code * 2^(s - 127), NaN under scale byte 255; rounded to bf16 (exact above bf16's subnormals)
template <bool F32>
__global__ __launch_bounds__(kThreads) void mxfp8_dequant_kernel(const uint8_t *__restrict__ codes,
                                                                 const uint8_t *__restrict__ scales, size_t units,
                                                                 void *__restrict__ out) {
    const size_t u = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (u >= units) return;
    const u32x2 c = ((const u32x2 *)codes)[u];
    const float sc = e8m0_to_f32(scales[u >> 2]);
    float v[8];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const f32x2 a = fp8x2_to_f32x2<false>(c[d]), b = fp8x2_to_f32x2<true>(c[d]);
        v[4 * d] = a.x * sc;
        v[4 * d + 1] = a.y * sc;
        v[4 * d + 2] = b.x * sc;
        v[4 * d + 3] = b.y * sc;
    }
    if constexpr (F32) {
        ((f32x4 *)out)[2 * u] = f32x4{v[0], v[1], v[2], v[3]};
        ((f32x4 *)out)[2 * u + 1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        ((u32x4 *)out)[u] = u32x4{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
    }
}

moe_status check_mxfp8(const char *who, int32_t rows, int32_t cols, const void *a, const uint8_t *codes, const uint8_t *scales,
                       int32_t dtype) {
    MOE_REQUIRE(rows >= 0 && cols > 0 && cols % 32 == 0,
                "%s: need rows >= 0 and cols a positive multiple of 32 (rows=%d cols=%d)", who, rows, cols);
    MOE_REQUIRE(dtype == MOE_DT_BF16 || dtype == MOE_DT_F32, "%s: unknown dtype %d", who, dtype);
    MOE_REQUIRE((int64_t)rows * cols < INT32_MAX, "%s: sizes overflow int32", who);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(a && codes && scales, "%s: NULL pointer argument", who);
    MOE_REQUIRE((((uintptr_t)a | (uintptr_t)codes) & 15) == 0, "%s: values and codes must be 16-byte aligned", who);
    return MOE_OK;
}

}  // namespace

moe_status mxfp8_dequant_launch(size_t rows, int cols, const uint8_t *codes, const uint8_t *scales, void *out, bool f32,
                                hipStream_t s) {
    const size_t units = rows * (size_t)cols / 8;
    const dim3 grid((unsigned)((units + kThreads - 1) / kThreads));
    if (f32) hipLaunchKernelGGL(mxfp8_dequant_kernel<true>, grid, dim3(kThreads), 0, s, codes, scales, units, out);
    else hipLaunchKernelGGL(mxfp8_dequant_kernel<false>, grid, dim3(kThreads), 0, s, codes, scales, units, out);
    return launch_check("moe_mxfp8_dequant");
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mxfp8_quantize(int32_t rows, int32_t cols, const void *x, int32_t x_dtype, uint8_t *codes,
                                         uint8_t *scales, moe_stream stream) {
    clear_error();
    MOE_TRY(check_mxfp8("moe_mxfp8_quantize", rows, cols, x, codes, scales, x_dtype));
    if (rows == 0) return MOE_OK;
    const size_t units = (size_t)rows * cols / 8;
    const dim3 grid((unsigned)((units + kThreads - 1) / kThreads));
    hipStream_t s = (hipStream_t)stream;
    if (x_dtype == MOE_DT_F32)
        hipLaunchKernelGGL(mxfp8_quantize_kernel<true>, grid, dim3(kThreads), 0, s, x, units, codes, scales);
    else
        hipLaunchKernelGGL(mxfp8_quantize_kernel<false>, grid, dim3(kThreads), 0, s, x, units, codes, scales);
    return launch_check("moe_mxfp8_quantize");
}

extern "C" moe_status moe_mxfp8_dequant(int32_t rows, int32_t cols, const uint8_t *codes, const uint8_t *scales, void *out,
                                        int32_t out_dtype, moe_stream stream) {
    clear_error();
    MOE_TRY(check_mxfp8("moe_mxfp8_dequant", rows, cols, out, codes, scales, out_dtype));
    if (rows == 0) return MOE_OK;
    return mxfp8_dequant_launch((size_t)rows, cols, codes, scales, out, out_dtype == MOE_DT_F32, (hipStream_t)stream);
}
