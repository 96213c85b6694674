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

// Sum the parts of the split tiles in order (the same order on every run), the terms of a row after each
// other, and run the epilogue.  A workgroup takes kFinishRows rows of a tile; LANES threads a row, four
// columns each, and a thread U rows, whose loads of all parts are independent.  Bound by the partial results,
// written just before and read from the last-level cache: gate and up of 512 x 2368, six parts (60 MB), 10.7
// us, 5.6 TB/s; five parts of 61 x 6144, two terms (16 MB), 6.3 us, half of it the launch.  (Loads of four
// parts at a time measured the same.)
template <int LANES, class Epi>
__global__ __launch_bounds__(kThreads) void dense_finish_kernel(const float *__restrict__ part, int full, int split, int terms,
                                                                int tr_n, int tc_n, int rows, int C, int br, Epi epi) {
    constexpr int kStep = kThreads / LANES, U = kFinishRows / kStep;
    constexpr int BC = LANES * 4 * (Epi::kPair ? 2 : 1);
    static_assert(U >= 1 && U * kStep == kFinishRows, "whole rows");
    const int blocks = br / kFinishRows;
    const int t = blockIdx.x / blocks, rb = blockIdx.x - t * blocks;
    int tr, tc;
    if (terms == 1) {
        tile_at(full + t, tr_n, tc_n, tr, tc);
    } else {                                      // (every tile is split) output rows are the first term's
        tr = t / tc_n;
        tc = t - tr * tc_n;
    }
    const int lane = threadIdx.x % LANES, er = threadIdx.x / LANES;
    const int c = tc * (LANES * 4) + 4 * lane, r = tr * br + rb * kFinishRows + er;
    const bool live = c < C && r < rows;
    f32x4 sa = kZero4, sb = kZero4;
    if (live) {
        f32x4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = b[u] = kZero4;
        for (int j = 0; j < terms; ++j) {
            const float *src[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int rr = min(r + u * kStep, rows - 1) + j * rows, rt = rr / br;
                src[u] = part + ((size_t)(tile_slot(rt, tc, tr_n, tc_n) - full) * split * br + (rr - rt * br)) * BC + 4 * lane;
            }
            for (int s = 0; s < split; ++s)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float *q = src[u] + (size_t)s * br * BC;
                    a[u] += *(const f32x4 *)q;
                    if constexpr (Epi::kPair) b[u] += *(const f32x4 *)(q + BC / 2);
                }
        }
        epi.rows(epi.cols(c), r, kStep, rows, c, a, b, sa, sb);
    }
    if constexpr (Epi::kColSum) {
        if (epi.cs) {
            // column sums of the workgroup's rows, one partial row
            __shared__ f32x4 s_sum[Epi::kPair ? 2 : 1][kStep][LANES];
            s_sum[0][er][lane] = sa;
            if constexpr (Epi::kPair) s_sum[1][er][lane] = sb;
            __syncthreads();
            if (er == 0 && c < C) {
                for (int i = 1; i < kStep; ++i) {
                    sa += s_sum[0][i][lane];
                    if constexpr (Epi::kPair) sb += s_sum[1][i][lane];
                }
                float *row = epi.cs + (size_t)(tr * blocks + rb) * epi.csld;
                *(f32x4 *)(row + c) = sa;
                if constexpr (Epi::kPair) *(f32x4 *)(row + C + c) = sb;
            }
        }
    }
}

// Gradients of the gated product from the saved bf16 pre-activations [2][R][C].  Two rows a workgroup, to fill
// the CUs with few tokens: 61 x 2048 takes 4.6 us, most of it the launch.
__global__ __launch_bounds__(kThreads) void gate_bwd_saved_kernel(const uint16_t *__restrict__ pre, int R, EpiGateBwd epi) {
    const Block bl = block_of(epi.C);
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
moe_status dense_finish(const DenseProduct &p, const DensePlan &pl, int br, int bc, const Epi &e, const float *part,
                        hipStream_t s) {
    const int rows = p.R / p.terms, blocks = br / kFinishRows;
    const int tiles = p.terms == 1 ? pl.tr * pl.tc - pl.full : (rows + br - 1) / br * pl.tc;
    const dim3 grid((unsigned)(tiles * blocks));
    const int lanes = bc / 4 / (Epi::kPair ? 2 : 1);
#define MOE_FINISH(L)                                                                                                    \
    hipLaunchKernelGGL((dense_finish_kernel<L, Epi>), grid, dim3(kThreads), 0, s, part, pl.full, pl.split, p.terms, pl.tr, \
                       pl.tc, rows, p.C, br, e)
    if (lanes == 64) MOE_FINISH(64);
    else if (lanes == 32) MOE_FINISH(32);
    else MOE_FINISH(16);
#undef MOE_FINISH
    return launch_check("dense product: sum of its parts");
}
template moe_status dense_finish<EpiLinear>(const DenseProduct &, const DensePlan &, int, int, const EpiLinear &, const float *,
                                            hipStream_t);
template moe_status dense_finish<EpiGate>(const DenseProduct &, const DensePlan &, int, int, const EpiGate &, const float *,
                                          hipStream_t);
template moe_status dense_finish<EpiLinearBwd>(const DenseProduct &, const DensePlan &, int, int, const EpiLinearBwd &,
                                               const float *, hipStream_t);
template moe_status dense_finish<EpiGateBwd>(const DenseProduct &, const DensePlan &, int, int, const EpiGateBwd &,
                                             const float *, hipStream_t);
template moe_status dense_finish<EpiStore>(const DenseProduct &, const DensePlan &, int, int, const EpiStore &, const float *,
                                           hipStream_t);

moe_status dense_gate_bwd_saved(const EpiGateBwd &e, const uint16_t *pre, int R, hipStream_t s) {
    hipLaunchKernelGGL(gate_bwd_saved_kernel, block_grid(R, kSavedRows, e.C), dim3(kThreads), 0, s, pre, R, e);
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
