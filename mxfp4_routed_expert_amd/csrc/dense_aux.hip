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

// Sum the parts of the split tiles.  Bound by the partial results, written just before and read from the last-level
// cache: gate and up of 512 x 2368, three parts (29 MB), 6.4 us, 4.5 TB/s with the launch; five parts of 61 x 6144, two
// terms (16 MB), 6.3 us as a launch of its own, half of it the launch.  (Loads of four parts at a time measured the same.)
template <int LANES, class Epi>
__global__ __launch_bounds__(kFinishThreads) void dense_finish_kernel(const DenseParts q, Epi epi) {
    constexpr int kStep = kFinishThreads / LANES;
    f32x4 sa = kZero4, sb = kZero4;
    const FinishPlace at = dense_finish_rows<LANES>(q, epi, blockIdx.x, sa, sb);
    if constexpr (Epi::kColSum) {
        if (epi.cs) {
            // column sums of the workgroup's rows, one partial row
            __shared__ f32x4 s_sum[Epi::kPair ? 2 : 1][kStep][LANES];
            const int lane = threadIdx.x % LANES, er = threadIdx.x / LANES;
            s_sum[0][er][lane] = sa;
            if constexpr (Epi::kPair) s_sum[1][er][lane] = sb;
            __syncthreads();
            if (er == 0 && at.c < q.C) {
                for (int i = 1; i < kStep; ++i) {
                    sa += s_sum[0][i][lane];
                    if constexpr (Epi::kPair) sb += s_sum[1][i][lane];
                }
                float *row = epi.cs + (size_t)at.row * epi.csld;
                *(f32x4 *)(row + at.c) = sa;
                if constexpr (Epi::kPair) *(f32x4 *)(row + q.C + at.c) = sb;
            }
        }
    }
}

// Gradients of the gated product from the saved bf16 pre-activations [2][R][C].  Two rows a workgroup, to fill
// the CUs with few tokens: 61 x 2048 takes 4.6 us, most of it the launch.
__global__ __launch_bounds__(kThreads) void gate_bwd_saved_kernel(const uint16_t *__restrict__ pre, int R, int rb0, EpiGateBwd epi) {
    Block bl = block_of(epi.C);
    bl.rb += rb0;
    const int c = bl.cb * kCols + threadIdx.x * 4;
    if (c >= epi.C) return;
    const int r = bl.rb * kSavedRows;
    f32x4 g[kSavedRows], u[kSavedRows], sa = kZero4, sb = kZero4;
    load_rows(g, pre, false, epi.C, r, 1, R, c);
    load_rows(u, pre + (size_t)R * epi.C, false, epi.C, r, 1, R, c);
    epi.rows(EpiGateBwd::Cols{kZero4, kZero4}, r, 1, R, c, g, u, sa, sb);
    if (epi.cs) {
        float *row = epi.cs + (size_t)bl.rb * epi.csld;
        *(f32x4 *)(row + c) = sa;
        *(f32x4 *)(row + epi.C + c) = sb;
    }
}

__global__ __launch_bounds__(kThreads) void side_kernel(const DenseSide j) {
    __shared__ float s_sum[kThreads];
    dense_side_job<kThreads>(j, blockIdx.x, s_sum);
}

// v = hi + mid + lo exactly (down to bf16's smallest value, 2^-133: what lies below is cut off).  hi is v's top eight significant
// bits (truncated, so it cannot round up past the largest finite bf16), mid what is left rounded to nearest, so that hi +
// mid alone is within 2^-16 of v on either side of it; lo is the rest, at most eight bits.  A non-finite v is its own
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
    const uint32_t b = __float_as_uint(r1);
    m = (b + 0x7fffu + ((b >> 16) & 1u)) >> 16;              // ties to even; |r1| is below hi's last place: no overflow
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
moe_status dense_finish(const DenseParts &q, const Epi &e, hipStream_t s) {
    const dim3 grid((unsigned)q.wgs);
#define MOE_FINISH(L) hipLaunchKernelGGL((dense_finish_kernel<L, Epi>), grid, dim3(kFinishThreads), 0, s, q, e)
    if (q.lanes == 64) MOE_FINISH(64);
    else if (q.lanes == 32) MOE_FINISH(32);
    else MOE_FINISH(16);
#undef MOE_FINISH
    return launch_check("dense product: sum of its parts");
}
template moe_status dense_finish<EpiLinear>(const DenseParts &, const EpiLinear &, hipStream_t);
template moe_status dense_finish<EpiGate>(const DenseParts &, const EpiGate &, hipStream_t);
template moe_status dense_finish<EpiLinearBwd>(const DenseParts &, const EpiLinearBwd &, hipStream_t);
template moe_status dense_finish<EpiGateBwd>(const DenseParts &, const EpiGateBwd &, hipStream_t);
template moe_status dense_finish<EpiStore>(const DenseParts &, const EpiStore &, hipStream_t);

moe_status dense_gate_bwd_saved(const EpiGateBwd &e, const uint16_t *pre, int R, hipStream_t s) {
    const int rbs = (R + kSavedRows - 1) / kSavedRows, cbs = col_blocks(e.C), most = max(1, kMaxGrid / cbs);
    for (int rb = 0; rb < rbs; rb += most)
        hipLaunchKernelGGL(gate_bwd_saved_kernel, dim3((unsigned)(min(rbs - rb, most) * cbs)), dim3(kThreads), 0, s, pre, R, rb, e);
    return launch_check("gated gradients");
}

moe_status dense_side_launch(const DenseSide &j, hipStream_t s) {
    const int wgs = dense_side_wgs(j, kThreads);
    if (wgs == 0) return MOE_OK;
    hipLaunchKernelGGL(side_kernel, dim3((unsigned)wgs), dim3(kThreads), 0, s, j);
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
