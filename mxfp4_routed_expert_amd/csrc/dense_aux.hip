// The passes around the dense products: sums of split products with their epilogues, gradients
// from saved pre-activations, column sums, and operand preparation.  All of them stream their
// data once and are bound by HBM (or, for decode-sized batches, by the launch).
#include "dense.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 4 * kThreads;      // columns per workgroup, four per thread

// Workgroup b of a (row block, column block) grid kept in one dimension (rows may exceed 65535).
struct Block {
    int rb, cb;
};
__host__ __device__ inline int col_blocks(int C) { return (C + kCols - 1) / kCols; }
MOE_DEV Block block_of(int C) {
    const int n = col_blocks(C);
    return Block{(int)blockIdx.x / n, (int)blockIdx.x % n};
}
dim3 block_grid(int R, int rows, int C) { return dim3((unsigned)((R + rows - 1) / rows) * (unsigned)col_blocks(C)); }

// Column-sum partials of this thread's four (pair: eight) columns: one row per workgroup row.
template <class Epi>
MOE_DEV void store_colsums(const Epi &epi, int rb, int C, int c, f32x4 sa, f32x4 sb) {
    if constexpr (Epi::kColSum) {
        if (epi.cs) {
            float *row = epi.cs + (size_t)rb * epi.csld;
            *(f32x4 *)(row + c) = sa;
            if constexpr (Epi::kPair) *(f32x4 *)(row + C + c) = sb;
        }
    }
}

// Sum the parts in order (the same order on every run) and run the epilogue.
template <class Epi>
__global__ __launch_bounds__(kThreads) void dense_finish_kernel(const float *__restrict__ part, int split, int R, int C,
                                                                int ld, Epi epi) {
    const Block bl = block_of(C);
    const int c = bl.cb * kCols + threadIdx.x * 4;
    if (c >= C) return;
    const size_t plane = (size_t)R * ld;
    constexpr int M = Epi::kPair ? 2 : 1;
    f32x4 sa = {0.f, 0.f, 0.f, 0.f}, sb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kFinishRows; ++i) {
        const int r = bl.rb * kFinishRows + i;
        if (r >= R) break;
        f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const float *src = part + (size_t)r * ld + c;
        for (int s = 0; s < split; ++s)
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += *(const f32x4 *)(src + (size_t)(s * M + m) * plane);
        f32x4 ca = {0.f, 0.f, 0.f, 0.f}, cb = {0.f, 0.f, 0.f, 0.f};
        epi.apply(r, c, v[0], v[1], ca, cb);
        sa += ca;
        sb += cb;
    }
    store_colsums(epi, bl.rb, C, c, sa, sb);
}

// Gradients of the gated product from the saved bf16 pre-activations [2][R][C].
__global__ __launch_bounds__(kThreads) void gate_bwd_saved_kernel(const uint16_t *__restrict__ pre, int R, EpiGateBwd epi) {
    const Block bl = block_of(epi.C);
    const int c = bl.cb * kCols + threadIdx.x * 4;
    if (c >= epi.C) return;
    f32x4 sa = {0.f, 0.f, 0.f, 0.f}, sb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kFinishRows; ++i) {
        const int r = bl.rb * kFinishRows + i;
        if (r >= R) break;
        const size_t o = (size_t)r * epi.C + c;
        f32x4 ca, cb;
        epi.grads(r, c, load4_bf16(pre + o), load4_bf16(pre + (size_t)R * epi.C + o), ca, cb);
        sa += ca;
        sb += cb;
    }
    store_colsums(epi, bl.rb, epi.C, c, sa, sb);
}

// Column sums of kColRows rows of a bf16 matrix.
__global__ __launch_bounds__(kThreads) void colsum_kernel(const uint16_t *__restrict__ a, int R, int C,
                                                          float *__restrict__ part, int ld) {
    const Block bl = block_of(C);
    const int c = bl.cb * kCols + threadIdx.x * 4;
    if (c >= C) return;
    const int r0 = bl.rb * kColRows, r1 = min(R, r0 + kColRows);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if ((C & 3) == 0) {
#pragma unroll 8
        for (int r = r0; r < r1; ++r) s += load4_bf16(a + (size_t)r * C + c);
    } else {
        for (int r = r0; r < r1; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c + q < C) s[q] += bf16_to_f32(a[(size_t)r * C + c + q]);
    }
    *(f32x4 *)(part + (size_t)bl.rb * ld + c) = s;
}

// Sum the partial rows: 64 columns a workgroup, four quarters of the rows, joined in order.
__global__ __launch_bounds__(kThreads) void colsum_reduce_kernel(const float *__restrict__ part, int rows, int ld, int C0,
                                                                 float *__restrict__ out0, float *__restrict__ out1) {
    __shared__ float s_q[4][64];
    const int lane = lane_id(), q = wave_id();
    const int C = out1 ? 2 * C0 : C0;
    const int c = blockIdx.x * 64 + lane;
    const int lo = (int)((int64_t)rows * q / 4), hi = (int)((int64_t)rows * (q + 1) / 4);
    float s = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int r = lo; r < hi; ++r) s += part[(size_t)r * ld + c];
    }
    s_q[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < C) {
        const float v = ((s_q[0][lane] + s_q[1][lane]) + s_q[2][lane]) + s_q[3][lane];
        if (c < C0) out0[c] = v;
        else out1[c - C0] = v;
    }
}

// v = hi + mid + lo exactly, each term the top eight significant bits of what is left
// (truncation, so no term can round up past the largest finite bf16).  A non-finite v is its own
// hi term and the others are zero.
MOE_DEV void split3(float v, uint32_t &h, uint32_t &m, uint32_t &l) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7f800000u) == 0x7f800000u) {
        h = (u >> 16) | ((u & 0xffffu) ? 0x40u : 0u);        // a NaN keeps a nonzero payload
        m = l = 0;
        return;
    }
    h = u >> 16;
    const float r1 = v - __uint_as_float(h << 16);
    m = __float_as_uint(r1) >> 16;
    const float r2 = r1 - __uint_as_float(m << 16);
    l = __float_as_uint(r2) >> 16;
}

__global__ __launch_bounds__(kThreads) void split3_kernel(const float *__restrict__ x, uint16_t *__restrict__ planes,
                                                          size_t n) {
    const size_t i = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 8;       // n is a multiple of 8
    if (i >= n) return;
    const f32x4 a = *(const f32x4 *)(x + i), b = *(const f32x4 *)(x + i + 4);
    u32x4 o[3];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t t0[3], t1[3];
        split3(d < 2 ? a[2 * d] : b[2 * d - 4], t0[0], t0[1], t0[2]);
        split3(d < 2 ? a[2 * d + 1] : b[2 * d - 3], t1[0], t1[1], t1[2]);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) o[pl][d] = t0[pl] | (t1[pl] << 16);
    }
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) *(u32x4 *)(planes + pl * n + i) = o[pl];
}

__global__ __launch_bounds__(kThreads) void pad_rows_kernel(const uint16_t *__restrict__ x, uint16_t *__restrict__ out,
                                                            size_t n, int C, int ld) {
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const size_t r = i / (unsigned)ld;
    const int c = (int)(i - r * (unsigned)ld);
    out[i] = c < C ? x[r * C + c] : (uint16_t)0;
}

}  // namespace

template <class Epi>
moe_status dense_finish(int parts, const Epi &e, const float *part, int R, int C, hipStream_t s) {
    hipLaunchKernelGGL(dense_finish_kernel<Epi>, block_grid(R, kFinishRows, C), dim3(kThreads), 0, s, part, parts, R, C, (C + 3) & ~3, e);
    return launch_check("dense product: sum of its parts");
}
template moe_status dense_finish<EpiLinear>(int, const EpiLinear &, const float *, int, int, hipStream_t);
template moe_status dense_finish<EpiGate>(int, const EpiGate &, const float *, int, int, hipStream_t);
template moe_status dense_finish<EpiLinearBwd>(int, const EpiLinearBwd &, const float *, int, int, hipStream_t);
template moe_status dense_finish<EpiGateBwd>(int, const EpiGateBwd &, const float *, int, int, hipStream_t);
template moe_status dense_finish<EpiStore>(int, const EpiStore &, const float *, int, int, hipStream_t);

moe_status dense_gate_bwd_saved(const EpiGateBwd &e, const uint16_t *pre, int R, hipStream_t s) {
    hipLaunchKernelGGL(gate_bwd_saved_kernel, block_grid(R, kFinishRows, e.C), dim3(kThreads), 0, s, pre, R, e);
    return launch_check("gated gradients");
}

moe_status dense_colsum(const uint16_t *a, int R, int C, float *part, int csld, hipStream_t s) {
    hipLaunchKernelGGL(colsum_kernel, block_grid(R, kColRows, C), dim3(kThreads), 0, s, a, R, C, part, csld);
    return launch_check("column sums");
}

moe_status dense_colsum_reduce(const float *part, int rows, int ld, int C0, float *out0, float *out1, hipStream_t s) {
    const int C = out1 ? 2 * C0 : C0;
    hipLaunchKernelGGL(colsum_reduce_kernel, dim3((unsigned)((C + 63) / 64)), dim3(kThreads), 0, s, part, rows, ld, C0, out0,
                       out1);
    return launch_check("column sums");
}

moe_status dense_split3(const float *x, uint16_t *planes, size_t n, hipStream_t s) {
    hipLaunchKernelGGL(split3_kernel, dim3((unsigned)((n / 8 + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, x, planes, n);
    return launch_check("float32 rows to bf16 terms");
}

moe_status dense_pad_rows(const uint16_t *x, uint16_t *out, int R, int C, int ld, hipStream_t s) {
    const size_t n = (size_t)R * ld;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, x, out, n, C, ld);
    return launch_check("padded rows");
}

}  // namespace moe
