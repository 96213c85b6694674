// Dense products of a few tokens (T <= 8): one pass over the weights on the vector ALU.
//
// Bound by the weight bytes (one token, in graphs, weights from HBM: 2048 x 7168 7.0 us, 4.2 TB/s; gate and up of 2368 x
// 7168 14.6 us, 4.7 TB/s; 6.0 and 13.7 us with weights partly in the last-level cache).  A workgroup of four waves owns four consecutive output columns (four gate and four up rows
// for the pair, eight columns with several float32 rows); its waves take every fourth 512-value piece of the
// sum, a lane 8 consecutive values of each row, so every load is a whole 1 KiB line run of one
// row and a wave keeps 8 or more of them in flight.  The tokens' values of a piece are read once
// per wave from the L2 and used for all the rows.  bf16 rows multiply with v_dot2_f32_bf16,
// float32 rows as float32.  The lanes' sums meet in a butterfly that halves the values per lane
// at every step, the waves' in LDS in a fixed order; then one thread a token runs the epilogue.
#include "dense.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kPiece = 512;             // values of a sum per wave and load

// Sums of v[0..V) over the wave: afterwards v[0] of lane l is the sum of value l >> (6 - log2 V).
template <int V>
MOE_DEV void butterfly(float (&v)[V]) {
    const int lane = lane_id();
    int o = 32;
    if constexpr (V > 1) {
        static_for<6>([&](auto st) {
            constexpr int n = V >> (st + 1);
            if constexpr (n >= 1) {
                const bool hi = lane & (32 >> st);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float keep = hi ? v[i + n] : v[i], send = hi ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor(send, 32 >> st, kWave);
                }
            }
        });
        o = 32 / V;
    }
    for (; o > 0; o >>= 1) v[0] += __shfl_xor(v[0], o, kWave);
}

template <int MT, bool F32X, int G, class Epi>
__global__ __launch_bounds__(64 * kWaves) void dense_gemv_kernel(const void *__restrict__ x, const uint16_t *__restrict__ w0,
                                                                 const uint16_t *__restrict__ w1, int T, int n, int K,
                                                                 int c0, Epi epi) {
    constexpr int NM = Epi::kPair ? 2 : 1, ROWS = 4 * NM * G, V = ROWS * MT;
    static_assert(NM == 1 || G == 1, "a pair is two groups of rows");
    static_assert(V <= 64, "one value per lane after the butterfly");
    __shared__ float s_sum[kWaves][V];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int c = c0 + blockIdx.x * (4 * G);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;

    const uint16_t *wrow[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) wrow[i] = (NM == 2 && i >= 4 ? w1 : w0) + (size_t)min(c + (NM == 2 ? i & 3 : i), n - 1) * K;

    // 8 values of every row and token from value k on; past the end of the sum both are zero
    auto piece = [&](int k, bool live) {
        u32x4 w[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) w[i] = __builtin_nontemporal_load((const MOE_GLOBAL u32x4 *)(wrow[i] + k));
        u32x4 xb[MT][F32X ? 2 : 1];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const size_t o = (size_t)min(t, T - 1) * K + k;
            if constexpr (F32X) {
                xb[t][0] = *(const MOE_GLOBAL u32x4 *)((const float *)x + o);
                xb[t][1] = *(const MOE_GLOBAL u32x4 *)((const float *)x + o + 4);
            } else {
                xb[t][0] = *(const MOE_GLOBAL u32x4 *)((const uint16_t *)x + o);
            }
        }
        if (!live) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) w[i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < (F32X ? 2 : 1); ++h) xb[t][h] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (F32X) {
                    const f32x2 wv = bf16x2_to_f32x2(w[i][d]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        float &a = acc[i * MT + t];
                        a = fmaf(wv.x, __uint_as_float(xb[t][d >> 1][2 * (d & 1)]), a);
                        a = fmaf(wv.y, __uint_as_float(xb[t][d >> 1][2 * (d & 1) + 1]), a);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[i * MT + t] = dot2_bf16(as_bf16x2(w[i][d]), as_bf16x2(xb[t][0][d]), acc[i * MT + t]);
                }
            }
    };
    const int full = K / kPiece;
#pragma unroll 2
    for (int i = wave; i < full; i += kWaves) piece(i * kPiece + lane * 8, true);
    if (full * kPiece < K && wave == full % kWaves) {
        const int k = full * kPiece + lane * 8;             // K is a multiple of 8: a lane's 8 values are all in or all out
        piece(min(k, K - 8), k < K);
    }

    butterfly(acc);
    constexpr int kLanesPer = 64 / V;
    if (lane % kLanesPer == 0) s_sum[wave][lane / kLanesPer] = acc[0];
    __syncthreads();
    const int t = threadIdx.x % MT, g = threadIdx.x / MT;    // token and group of four columns
    if (g < G && t < T && c + 4 * g < n) {
        f32x4 a[1] = {kZero4}, b[1] = {kZero4}, ca, cb;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                a[0][q] += s_sum[w][(4 * g + q) * MT + t];
                if constexpr (NM == 2) b[0][q] += s_sum[w][(4 + q) * MT + t];
            }
        epi.rows(epi.cols(c + 4 * g), t, 1, T, c + 4 * g, a, b, ca, cb);
    }
}

// G groups of four columns a workgroup: with four or more float32 rows their own bytes, read by every
// workgroup, outweigh four weight rows', so eight are taken (T = 4, 7168 x 2048: 10.5 -> 10.0 us; T = 8,
// 7168 x 2368: 19.3 -> 17.0 us); otherwise the smaller workgroups fill the CUs better (T = 1,
// 2048 x 7168: 6.9 us against 7.5).
template <bool F32X, class Epi>
moe_status launch(const void *x, const uint16_t *w0, const uint16_t *w1, int T, int n, int K, const Epi &e, hipStream_t s) {
    constexpr int G = F32X ? 2 : 1;
    auto run = [&](auto mt, auto g) {
        constexpr int MT = decltype(mt)::value, GG = decltype(g)::value;
        const int wgs = (n + 4 * GG - 1) / (4 * GG);
        for (int b = 0; b < wgs; b += kMaxGrid)
            hipLaunchKernelGGL((dense_gemv_kernel<MT, F32X, GG, Epi>), dim3((unsigned)min(wgs - b, kMaxGrid)), dim3(64 * kWaves), 0, s,
                               x, w0, w1, T, n, K, b * 4 * GG, e);
    };
    using One = std::integral_constant<int, 1>;
    using Many = std::integral_constant<int, G>;
    if (T == 1) run(One{}, One{});
    else if (T == 2) run(std::integral_constant<int, 2>{}, One{});
    else if (T <= 4) run(std::integral_constant<int, 4>{}, Many{});
    else run(std::integral_constant<int, 8>{}, Many{});
    return launch_check("dense product of a few tokens");
}

}  // namespace

moe_status dense_linear_gemv(const void *x, bool x_f32, const uint16_t *w, int T, int n, int k, const EpiLinear &e,
                             hipStream_t s) {
    return x_f32 ? launch<true>(x, w, w, T, n, k, e, s) : launch<false>(x, w, w, T, n, k, e, s);
}

moe_status dense_gate_gemv(const void *x, const uint16_t *wg, const uint16_t *wu, int T, int f, int d, const EpiGate &e,
                           hipStream_t s) {
    return launch<false>(x, wg, wu, T, f, d, e, s);
}

}  // namespace moe
