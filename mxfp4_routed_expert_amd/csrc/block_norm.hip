// What lies between two blocks: the norm after a block with dropout, gate and residual, and the norm before the
// next one with its 8-bit form, as one pass over the rows; and its gradients.
//
//   r(v) = 1 / sqrt(mean v^2 + eps),  n = z r(z) w_after (or z),  y = rs residual + gate m n,  u = y r(y) w_before,
// m the dropout factor (0 or 1 / (1 - p)).  Gradients, with t = dL/dy in all:
//   t = dy + r(y) (w_b du) - y r(y)^3 mean(w_b du y),          dresidual = rs t,   dw_before = sum_T du y r(y)
//   a = gate m t,  dz = r(z) (w_a a) - z r(z)^3 mean(w_a a z),  dw_after = sum_T a z r(z),  dgate = sum m t n.
// r^3 leaves float32 for rows that do not (2^50: 2^-150), so each r is multiplied with a factor of its own size: dz = r (w_a a -
// z r mean(w_a a z r)), y's the same.  A dropped element's m n is 0 in every sum, also where n is NaN or infinite.
// Both sums over a row that dz needs are known before t is (those of z, y and du) or follow from one more, so a row
// is in registers from its one read to its one write.
//
// A row belongs to a workgroup (or, when it is short, to a wave): chunks of 8 values, thread i takes chunks i, i +
// threads, ...  16 neighbouring lanes hold a 128-block of the 8-bit form.  The weights stay in LDS (a wave's own row: in
// registers) while a workgroup walks its rows; the column sums of the weights' gradients stay in registers, leave as one
// partial row a workgroup and are added in order by a second kernel: no atomics, the same bits every time.
//
// Bound by HBM.  8192 x 7168 bf16 with both norms, a channel gate, dropout and a residual: forward 94 us (5.0 TB/s; a copy
// 5.0 to 5.7 by card), backward with all gradients 136 us (5.2 TB/s).  Two rows in flight instead of one: the same.  512
// workgroups forward; 256 backward, since each adds a partial row of 8 d bytes: 509 x 6144 takes 15 us and 4 for the sums.
#include <algorithm>
#include <initializer_list>

#include "fp8.h"

namespace moe {
namespace {

constexpr int kMaxGroups = 512;        // workgroups of a forward launch that walks many rows
constexpr int kMaxParts = 256;         // of a backward one, and (a wave's own times 4) partial rows of its column sums
constexpr int kMaxThreads = 1024;
constexpr int kMaxD = 8 * 2 * kMaxThreads;

struct NormArgs {
    int T, d, chunks;                  // chunks = d / 8
    const void *z;
    const void *residual;
    const float *w_after, *w_before, *gate;
    int gate_kind;
    float eps, rs;
    uint32_t cut;                      // dropout: kept when 16 random bits >= cut
    float keep_scale;                  // 1 / (1 - cut / 65536)
    const uint64_t *rng;               // seed, offset
    void *y;
    uint16_t *u;
    uint8_t *codes, *scales;
    // gradients
    const uint16_t *du;
    const void *dy;
    void *dz, *dres;
    float *dgate_row;                  // [T], gate of a token
    float *part;                       // [2][groups][d]: sums for w_after / gate, then for w_before
    int groups;
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; SC 2011): 128 random bits for
// the chunk of 8 values whose number is the counter's low half.
struct Philox {
    uint32_t k0, k1, o0, o1;
    MOE_DEV void bits(uint64_t chunk, uint32_t (&c)[4]) const {
        c[0] = (uint32_t)chunk;
        c[1] = (uint32_t)(chunk >> 32);
        c[2] = o0;
        c[3] = o1;
        uint32_t a = k0, b = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p = (uint64_t)c[0] * 0xD2511F53u, q = (uint64_t)c[2] * 0xCD9E8D57u;
            const uint32_t n0 = (uint32_t)(q >> 32) ^ c[1] ^ a, n2 = (uint32_t)(p >> 32) ^ c[3] ^ b;
            c[1] = (uint32_t)q;
            c[3] = (uint32_t)p;
            c[0] = n0;
            c[2] = n2;
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
    }
};

typedef float f8[8];

// A row of a tensor as a buffer: reads past its end (or of a row or tensor that is not there) give zeros, writes there are
// dropped.  So a row's loads and stores stand in straight-line code and the compiler knows how many stores follow the next
// row's loads; with a branch around any of them it waits for all of them (every row for its own stores: 4.4 us a row).
typedef __amdgpu_buffer_rsrc_t Row;
MOE_DEV Row row_of(const void *p, int t, int T, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((char *)const_cast<void *>(p) + (size_t)t * bytes, 0, p && t < T ? bytes : 0, 0x00027000);
}
constexpr int kNowhere = 0x7ffffff0;                      // an offset past every row

// Eight values as they lie in memory, and in float32.
template <bool F32>
struct Raw8 {
    u32x4 w[F32 ? 2 : 1];
};
template <bool F32>
MOE_DEV void fetch8(Row r, int ch, Raw8<F32> &v) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i)
        v.w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (F32 ? 32 : 16) * ch + 16 * i, 0, 0));
}
template <bool F32>
MOE_DEV void widen8(const Raw8<F32> &r, f8 &v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
            v[i] = __uint_as_float(r.w[0][i]);
            v[4 + i] = __uint_as_float(r.w[1][i]);
        } else {
            const f32x2 f = bf16x2_to_f32x2(r.w[0][i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
MOE_DEV void load8f(const float *p, size_t at, f8 &v) {
    const f32x4 a = *(const f32x4 *)(p + at), b = *(const f32x4 *)(p + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}
template <bool F32>
MOE_DEV void store8(Row r, int ch, const f8 &v) {
    if constexpr (F32) {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, r, 32 * ch, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])}, r, 32 * ch + 16, 0, 0);
    } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};      // round to nearest even
            o[i] = __builtin_bit_cast(uint32_t, b);
        }
        __builtin_amdgcn_raw_buffer_store_b128(o, r, 16 * ch, 0, 0);
    }
}

// Sum over 16 neighbouring lanes, then over the wave, the same in every lane, in registers (DPP and lane swaps).
template <int CTRL>
MOE_DEV float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
MOE_DEV float sum16(float v) {
    v = dpp_add<0xB1>(v);        // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);        // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);       // row_half_mirror
    return dpp_add<0x140>(v);    // row_mirror
}
MOE_DEV float sum64(float v) {
    v = sum16(v);
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// The sums of N values over a row's threads, the same in all of them and in a fixed order.  lds: two buffers of N x 16,
// used in turn, so that one barrier does: a buffer is written again only after the next sum's barrier.
template <bool WAVE, int N>
MOE_DEV void row_sums(float (&s)[N], float *lds, int &turn) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sum64(s[i]);
    if constexpr (!WAVE) {
        float *at = lds + turn * (16 * 3);
        turn ^= 1;
        const int nw = blockDim.x >> 6, l = lane_id() & 15;
        if (lane_id() == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[16 * i + wave_id()] = s[i];
        }
        lds_barrier();                                    // (the next row's loads stay in flight)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = sum16(l < nw ? at[16 * i + l] : 0.0f);
    }
}

MOE_DEV Philox philox_of(const NormArgs &a) {
    Philox g = {0, 0, 0, 0};
    if (a.cut) {
        const uint64_t seed = a.rng[0], off = a.rng[1];
        g = Philox{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
    }
    return g;
}
// v times the dropout factors of a chunk; n: 0 where an element is dropped, whatever it held
MOE_DEV void drop8(const NormArgs &a, const Philox &g, uint64_t chunk, f8 &v, f8 *n = nullptr) {
    uint32_t c[4];
    g.bits(chunk, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t half = (i & 1) ? c[i >> 1] >> 16 : c[i >> 1] & 0xffffu;
        v[i] = half >= a.cut ? v[i] * a.keep_scale : 0.0f;
        if (n) (*n)[i] = half >= a.cut ? (*n)[i] : 0.0f;
    }
}

// The channels' factors of a thread's chunks.  A wave that walks rows keeps them in registers.  A workgroup keeps them in
// LDS, each thread its own (no barrier), and spends the registers on rows in flight: a row of 7168 bf16 values is 28 KB
// of two tensors, and a CU needs about 100 KB on its way to draw its share of the HBM rate.
template <bool WAVE, int NC>
struct Factors {
    f8 reg[WAVE ? NC : 1];
    f32x4 *lds;                                           // two planes of `chunks` x 4 values, a place for every thread's chunk
    int chunks;
    MOE_DEV void init(float *base, int n) {
        lds = (f32x4 *)base;
        chunks = n;
    }
    MOE_DEV void put(int c, int ch, const f8 &v) {
        if constexpr (WAVE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) reg[c][i] = v[i];
        } else {
            lds[ch] = f32x4{v[0], v[1], v[2], v[3]};
            lds[chunks + ch] = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
    MOE_DEV void get(int c, int ch, f8 &v) const {
        if constexpr (WAVE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = reg[c][i];
        } else {
            const f32x4 a = lds[ch], b = lds[chunks + ch];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
    }
};
// wc: w_after times the channels' gate; wb: w_before
template <bool WAVE, int NC>
MOE_DEV void factors_of(const NormArgs &a, int tid, int lanes, float *lds, Factors<WAVE, NC> &wc, Factors<WAVE, NC> &wb) {
    wc.init(lds, NC * lanes);
    wb.init(lds + 8 * NC * lanes, NC * lanes);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ch = tid + c * lanes;
        const bool live = ch < a.chunks;
        f8 v, w;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i] = 1.0f;
        if (a.w_after && live) load8f(a.w_after, 8 * (size_t)ch, v);
        if (a.w_before && live) load8f(a.w_before, 8 * (size_t)ch, w);
        if (a.gate_kind == MOE_GATE_CHANNEL && live) {
            f8 g;
            load8f(a.gate, 8 * (size_t)ch, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= g[i];
        }
        wc.put(c, ch, v);
        wb.put(c, ch, w);
    }
}
template <bool WAVE, int NC, bool ZF, bool YF, bool CODES>
__global__ __launch_bounds__(WAVE ? 256 : kMaxThreads) void block_norm_kernel(const NormArgs a) {
    __shared__ float lds[2 * 3 * 16];
    extern __shared__ __align__(16) float s_factors[];      // (a workgroup's rows: 16 NC floats a thread)
    const int lanes = WAVE ? kWave : blockDim.x;
    const int tid = WAVE ? lane_id() : threadIdx.x;
    const int group = WAVE ? __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + wave_id()) : blockIdx.x, groups = WAVE ? gridDim.x * 4 : gridDim.x;
    const float inv_d = 1.0f / (float)a.d;
    const int zb = (ZF ? 4 : 2) * a.d, yb = (YF ? 4 : 2) * a.d;      // bytes of a row
    int turn = 0;
    Raw8<ZF> zn[NC];
    Raw8<YF> rn[NC];
    auto fetch = [&](int t) __attribute__((always_inline)) {
        const Row z = row_of(a.z, t, a.T, zb), r = row_of(a.residual, t, a.T, yb);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            fetch8<ZF>(z, tid + c * lanes, zn[c]);
            fetch8<YF>(r, tid + c * lanes, rn[c]);
        }
    };
    fetch(group);
    Factors<WAVE, NC> wc, wb;
    factors_of<WAVE, NC>(a, tid, lanes, s_factors, wc, wb);
    const Philox rng = philox_of(a);
    for (int t = group; t < a.T; t += groups) {
        f8 v[NC], res[NC];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            widen8<ZF>(zn[c], v[c]);
            widen8<YF>(rn[c], res[c]);
        }
        fetch(t + groups);                                // the next row, while this one is worked on
        float rz = 1.0f;
        if (a.w_after) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] = fmaf(v[c][i], v[c][i], s[0]);
            row_sums<WAVE, 1>(s, lds, turn);
            rz = rsqrtf(fmaf(s[0], inv_d, a.eps));
        }
        rz *= a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
        const Row yr = row_of(a.y, t, a.T, yb);
        s[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ch = tid + c * lanes;
            f8 w;
            wc.get(c, ch, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= rz * w[i];
            if (a.cut) drop8(a, rng, (uint64_t)t * (unsigned)a.chunks + (unsigned)ch, v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float y = v[c][i];
                if (a.residual) y = fmaf(a.rs, res[c][i], y);
                if constexpr (!YF) y = (float)(__bf16)y;                   // (u is that of the y that is kept)
                v[c][i] = y;
                s[0] = fmaf(y, y, s[0]);
            }
            store8<YF>(yr, ch, v[c]);
        }
        const Row ur = row_of(a.u, t, a.T, 2 * a.d), cr = row_of(a.codes, t, a.T, a.d), sr = row_of(a.scales, t, a.T, (a.chunks + 15) >> 4);
        float ry = 0.0f;
        if (a.w_before) {
            row_sums<WAVE, 1>(s, lds, turn);
            ry = rsqrtf(fmaf(s[0], inv_d, a.eps));
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ch = tid + c * lanes;
            f8 w;
            wb.get(c, ch, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = (float)(__bf16)(v[c][i] * ry * w[i]);
            store8<false>(ur, ch, v[c]);
            if constexpr (CODES) {                                          // (of the rounded u, as moe_fp8_quantize(u))
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, fp8_magnitude(v[c][i]));
                m = fp8_max16(ch < a.chunks ? m : 0u);
                const int X = fp8_exponent(m);
                const float inv = fp8_inverse(X);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{fp8_codes4(v[c][0], v[c][1], v[c][2], v[c][3], inv), fp8_codes4(v[c][4], v[c][5], v[c][6], v[c][7], inv)},
                                                      cr, 8 * ch, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b8((unsigned char)(X + 127), sr, (ch & 15) == 0 ? ch >> 4 : kNowhere, 0, 0);
            }
        }
    }
}

template <bool WAVE, int NC, bool ZF, bool YF>
__global__ __launch_bounds__(WAVE ? 256 : kMaxThreads) void block_norm_backward_kernel(const NormArgs a) {
    __shared__ float lds[2 * 3 * 16];
    extern __shared__ __align__(16) float s_factors[];      // (a workgroup's rows: 16 NC floats a thread)
    const int lanes = WAVE ? kWave : blockDim.x;
    const int tid = WAVE ? lane_id() : threadIdx.x;
    const int group = WAVE ? __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + wave_id()) : blockIdx.x;
    const float inv_d = 1.0f / (float)a.d;
    const int zb = (ZF ? 4 : 2) * a.d, yb = (YF ? 4 : 2) * a.d;      // bytes of a row
    int turn = 0;
    Raw8<ZF> zn[NC];
    Raw8<YF> yn[NC], tn[NC];
    Raw8<false> gn[NC];
    auto fetch = [&](int t) __attribute__((always_inline)) {
        const Row z = row_of(a.z, t, a.T, zb), dy = row_of(a.dy, t, a.T, yb), y = row_of(a.y, t, a.T, yb), du = row_of(a.du, t, a.T, 2 * a.d);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ch = tid + c * lanes;
            fetch8<ZF>(z, ch, zn[c]);
            fetch8<YF>(dy, ch, tn[c]);
            fetch8<YF>(y, ch, yn[c]);
            fetch8<false>(du, ch, gn[c]);
        }
    };
    fetch(group);
    Factors<WAVE, NC> wc, wb;
    factors_of<WAVE, NC>(a, tid, lanes, s_factors, wc, wb);
    f8 sa[NC], sb[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sa[c][i] = sb[c][i] = 0.0f;
    const Philox rng = philox_of(a);
    for (int t = group; t < a.T; t += a.groups) {
        f8 z[NC], y[NC], g[NC], tt[NC];                     // g: du; tt: dL/dy
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            widen8<ZF>(zn[c], z[c]);
            widen8<YF>(tn[c], tt[c]);
            widen8<YF>(yn[c], y[c]);
            widen8<false>(gn[c], g[c]);
        }
        fetch(t + a.groups);                              // the next row, while this one is worked on
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            f8 w;
            wb.get(c, tid + c * lanes, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] = fmaf(z[c][i], z[c][i], s[0]);
                s[1] = fmaf(y[c][i], y[c][i], s[1]);
                s[2] = fmaf(g[c][i] * w[i], y[c][i], s[2]);
            }
        }
        if (a.w_after || a.w_before) row_sums<WAVE, 3>(s, lds, turn);
        const float rz = a.w_after ? rsqrtf(fmaf(s[0], inv_d, a.eps)) : 1.0f;
        if (a.w_before) {
            const float ry = rsqrtf(fmaf(s[1], inv_d, a.eps));
            const float k = ry * (ry * (s[2] * inv_d));
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                f8 w;
                wb.get(c, tid + c * lanes, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sb[c][i] = fmaf(g[c][i], y[c][i] * ry, sb[c][i]);
                    tt[c][i] += ry * fmaf(-y[c][i], k, g[c][i] * w[i]);
                }
            }
        }
        const float gt = a.gate_kind == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
        const Row rr = row_of(a.dres, t, a.T, yb);
        float q[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ch = tid + c * lanes;
            f8 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.rs * tt[c][i];
            store8<YF>(rr, ch, o);
            f8 n;
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = z[c][i] * rz;
            if (a.cut) drop8(a, rng, (uint64_t)t * (unsigned)a.chunks + (unsigned)ch, tt[c], &n);
            f8 w;
            wc.get(c, ch, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sa[c][i] = fmaf(gt * tt[c][i], n[i], sa[c][i]);
                tt[c][i] *= w[i];
                q[0] = fmaf(tt[c][i], n[i], q[0]);
            }
        }
        if (a.w_after || a.dgate_row) row_sums<WAVE, 1>(q, lds, turn);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(q[0]), row_of(a.dgate_row, t, a.T, 4), tid == 0 ? 0 : kNowhere, 0, 0);
        const float mean = gt * q[0] * inv_d;
        const Row zr = row_of(a.dz, t, a.T, zb);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            // (no norm after: dz does not depend on z, which may be infinite)
#pragma unroll
            for (int i = 0; i < 8; ++i) tt[c][i] = a.w_after ? rz * fmaf(-(z[c][i] * rz), mean, gt * tt[c][i]) : gt * tt[c][i];
            store8<ZF>(zr, tid + c * lanes, tt[c]);
        }
    }
    if (!a.part || group >= a.groups) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ch = tid + c * lanes;
        if (ch >= a.chunks) continue;
        store8<true>(row_of(a.part, group, a.groups, 4 * a.d), ch, sa[c]);
        if (a.w_before) store8<true>(row_of(a.part, a.groups + group, 2 * a.groups, 4 * a.d), ch, sb[c]);
    }
}

// Column sums of the partial rows: 64 columns a workgroup, a sixteenth of the rows a wave, added in order.
// blockIdx.y == 0: S = sum of gate_token m t z r(z), dw_after = gate_channel S, dgate = w_after S; 1: dw_before.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void block_norm_sums_kernel(const float *__restrict__ part, int groups, int d, const float *w_after,
                                                                        const float *gate_channel, float *dw_after, float *dgate,
                                                                        float *dw_before) {
    __shared__ float q[kSumWaves][64];
    const int c = blockIdx.x * 64 + lane_id();
    const int w = wave_id();
    float s = 0.0f;
    if (c < d) {
        const float *p = part + (size_t)blockIdx.y * groups * d + c;
        const int r1 = groups * (w + 1) / kSumWaves;
#pragma unroll 8
        for (int r = groups * w / kSumWaves; r < r1; ++r) s += p[(size_t)r * d];
    }
    q[w][lane_id()] = s;
    __syncthreads();
    if (w || c >= d) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) s += q[i][lane_id()];
    if (blockIdx.y == 1) {
        dw_before[c] = s;
    } else {
        if (dw_after) dw_after[c] = gate_channel ? s * gate_channel[c] : s;
        if (dgate) dgate[c] = w_after ? s * w_after[c] : s;
    }
}

// One wave a row up to 1024 values, else a workgroup of the fewest whole waves with 1 chunk a thread, or 2 above 8192 values.
struct NormShape {
    bool wave;
    int nc, threads, grid, groups;
};
NormShape shape_of(int T, int d, bool backward) {
    const int most = backward ? kMaxParts : kMaxGroups;
    const int chunks = d / 8;
    NormShape s;
    s.wave = chunks <= 128;
    if (s.wave) {
        s.nc = chunks <= 64 ? 1 : 2;
        s.threads = 256;
        s.grid = (int)std::min<int64_t>(((int64_t)T + 3) / 4, most);
        s.groups = 4 * s.grid;
    } else {
        s.nc = chunks <= kMaxThreads ? 1 : 2;
        s.threads = (int)align_up((chunks + s.nc - 1) / s.nc, kWave);
        s.grid = std::min(T, most);
        s.groups = s.grid;
    }
    return s;
}

template <bool WAVE, int NC>
void launch(const NormArgs &a, const NormShape &sh, bool zf, bool yf, bool backward, hipStream_t s) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)sh.grid), dim3((unsigned)sh.threads), sh.wave ? 0 : 16 * sizeof(float) * sh.nc * sh.threads, s, a); };
    if (backward) {
        if (zf) yf ? go(block_norm_backward_kernel<WAVE, NC, true, true>) : go(block_norm_backward_kernel<WAVE, NC, true, false>);
        else yf ? go(block_norm_backward_kernel<WAVE, NC, false, true>) : go(block_norm_backward_kernel<WAVE, NC, false, false>);
    } else {
        auto with = [&](auto codes) {
            constexpr bool C = decltype(codes)::value;
            if (zf) yf ? go(block_norm_kernel<WAVE, NC, true, true, C>) : go(block_norm_kernel<WAVE, NC, true, false, C>);
            else yf ? go(block_norm_kernel<WAVE, NC, false, true, C>) : go(block_norm_kernel<WAVE, NC, false, false, C>);
        };
        if (a.codes) with(std::true_type{});
        else with(std::false_type{});
    }
}
void launch_any(const NormArgs &a, const NormShape &sh, bool zf, bool yf, bool backward, hipStream_t s) {
    if (sh.wave) {
        if (sh.nc == 1) launch<true, 1>(a, sh, zf, yf, backward, s);
        else launch<true, 2>(a, sh, zf, yf, backward, s);
    } else {
        if (sh.nc == 1) launch<false, 1>(a, sh, zf, yf, backward, s);
        else launch<false, 2>(a, sh, zf, yf, backward, s);
    }
}

moe_status check_desc(const moe_block_norm_desc *n, const char *who) {
    MOE_REQUIRE(n != nullptr, "%s: desc is NULL", who);
    MOE_REQUIRE(n->T >= 0 && n->d > 0 && n->d % 8 == 0, "%s: need T >= 0 and d a positive multiple of 8 (T=%d d=%d)", who, n->T, n->d);
    if (n->d > kMaxD) {
        set_error("%s: d = %d above %d", who, n->d, kMaxD);
        return MOE_ERR_UNSUPPORTED;
    }
    MOE_REQUIRE((int64_t)n->T * n->d < INT32_MAX, "%s: sizes overflow int32", who);
    MOE_REQUIRE(n->z_dtype == MOE_DT_BF16 || n->z_dtype == MOE_DT_F32, "%s: unknown z_dtype %d", who, n->z_dtype);
    MOE_REQUIRE(n->y_dtype == MOE_DT_BF16 || n->y_dtype == MOE_DT_F32, "%s: unknown y_dtype %d", who, n->y_dtype);
    MOE_REQUIRE(n->gate >= MOE_GATE_NONE && n->gate <= MOE_GATE_CHANNEL, "%s: unknown gate %d", who, n->gate);
    MOE_REQUIRE(n->eps > 0.0f && n->eps < 3.0e38f, "%s: eps = %g must be positive and finite", who, (double)n->eps);
    MOE_REQUIRE(n->residual_scale > -3.0e38f && n->residual_scale < 3.0e38f, "%s: residual_scale must be finite", who);
    MOE_REQUIRE(n->dropout >= 0.0f && n->dropout < 1.0f, "%s: dropout = %g outside [0, 1)", who, (double)n->dropout);
    return MOE_OK;
}
uint32_t cut_of(const moe_block_norm_desc *n) {
    const uint32_t cut = (uint32_t)((double)n->dropout * 65536.0 + 0.5);
    return cut < 65535u ? cut : 65535u;
}
NormArgs args_of(const moe_block_norm_desc *n, const void *z, const float *w_after, const float *gate, const uint64_t *rng,
                 const float *w_before) {
    NormArgs a = {};
    a.T = n->T;
    a.d = n->d;
    a.chunks = n->d / 8;
    a.z = z;
    a.w_after = w_after;
    a.w_before = w_before;
    a.gate = gate;
    a.gate_kind = n->gate;
    a.eps = n->eps;
    a.rs = n->residual_scale;
    a.cut = cut_of(n);
    a.keep_scale = (float)(65536.0 / (65536.0 - (double)a.cut));
    a.rng = rng;
    return a;
}
inline bool aligned16(std::initializer_list<const void *> l) {
    uintptr_t m = 0;
    for (const void *p : l) m |= (uintptr_t)p;
    return (m & 15) == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_norm(const moe_block_norm_desc *n, const void *z, const float *w_after, const float *gate,
                                     const uint64_t *rng, const void *residual, const float *w_before, void *y, void *u,
                                     uint8_t *u_codes, uint8_t *u_scales, moe_stream stream) {
    clear_error();
    const char *who = "moe_block_norm";
    MOE_TRY(check_desc(n, who));
    if (n->T == 0) return MOE_OK;
    MOE_REQUIRE((gate != nullptr) == (n->gate != MOE_GATE_NONE), "%s: gate and its kind do not agree", who);
    MOE_REQUIRE((u_codes != nullptr) == (u_scales != nullptr), "%s: u_codes and u_scales come together or not at all", who);
    MOE_REQUIRE(!(u || u_codes) == !w_before, "%s: w_before and the normed outputs u, u_codes come together or not at all", who);
    MOE_REQUIRE(cut_of(n) == 0 || rng, "%s: dropout needs rng", who);
    MOE_REQUIRE(z != nullptr, "%s: NULL z", who);
    MOE_REQUIRE(y || u || u_codes, "%s: no output asked for", who);
    MOE_REQUIRE(aligned16({z, w_after, residual, w_before, y, u, u_codes}) && (n->gate != MOE_GATE_CHANNEL || aligned16({gate})),
                "%s: tensors must be 16-byte aligned", who);
    MOE_REQUIRE(((uintptr_t)gate & 3) == 0 && ((uintptr_t)rng & 7) == 0, "%s: gate or rng is misaligned", who);
    NormArgs a = args_of(n, z, w_after, gate, rng, w_before);
    a.residual = residual;
    a.y = y;
    a.u = (uint16_t *)u;
    a.codes = u_codes;
    a.scales = u_scales;
    const NormShape sh = shape_of(n->T, n->d, false);
    launch_any(a, sh, n->z_dtype == MOE_DT_F32, n->y_dtype == MOE_DT_F32, false, (hipStream_t)stream);
    return launch_check(who);
}

extern "C" size_t moe_block_norm_backward_workspace(const moe_block_norm_desc *n) {
    if (check_desc(n, "moe_block_norm_backward_workspace") != MOE_OK || n->T == 0) return 0;
    return (size_t)2 * shape_of(n->T, n->d, true).groups * n->d * sizeof(float);
}

extern "C" moe_status moe_block_norm_backward(const moe_block_norm_desc *n, const void *z, const float *w_after, const float *gate,
                                              const uint64_t *rng, const void *y, const float *w_before, const void *du, const void *dy,
                                              void *dz, void *dresidual, float *dw_after, float *dgate, float *dw_before, void *ws,
                                              size_t ws_bytes, moe_stream stream) {
    clear_error();
    const char *who = "moe_block_norm_backward";
    MOE_TRY(check_desc(n, who));
    // (a token's gate of no tokens may be NULL)
    MOE_REQUIRE((gate != nullptr) == (n->gate != MOE_GATE_NONE) || (n->T == 0 && n->gate == MOE_GATE_TOKEN),
                "%s: gate and its kind do not agree", who);
    MOE_REQUIRE(!dw_after || w_after, "%s: dw_after without w_after", who);
    MOE_REQUIRE(!dgate || n->gate != MOE_GATE_NONE, "%s: dgate without gate", who);
    MOE_REQUIRE(!dw_before || w_before, "%s: dw_before without w_before", who);
    MOE_REQUIRE(cut_of(n) == 0 || rng, "%s: dropout needs rng", who);
    MOE_REQUIRE(aligned16({w_after, w_before}) && (n->gate != MOE_GATE_CHANNEL || aligned16({gate})), "%s: tensors must be 16-byte aligned", who);
    MOE_REQUIRE((((uintptr_t)gate | (uintptr_t)dw_after | (uintptr_t)dgate | (uintptr_t)dw_before) & 3) == 0 && ((uintptr_t)rng & 7) == 0,
                "%s: gate, rng or a float32 gradient is misaligned", who);
    hipStream_t s = (hipStream_t)stream;
    const bool channel = n->gate == MOE_GATE_CHANNEL;
    const bool sums_a = dw_after || (dgate && channel), sums = sums_a || dw_before;
    NormArgs a = args_of(n, z, w_after, gate, rng, w_before);
    if (n->T > 0) {
        MOE_REQUIRE(dz || dresidual || sums || dgate, "%s: no gradient asked for", who);
        MOE_REQUIRE(dy || w_before, "%s: NULL dy without w_before: no gradient reaches y", who);
        MOE_REQUIRE((du != nullptr) == (w_before != nullptr) && (!w_before || y), "%s: w_before, du and y come together", who);
        MOE_REQUIRE(z || !((dz && w_after) || dgate || dw_after), "%s: NULL z", who);
        MOE_REQUIRE(aligned16({z, y, du, dy, dz, dresidual, ws}), "%s: tensors must be 16-byte aligned", who);
        const size_t need = sums ? moe_block_norm_backward_workspace(n) : 0;
        if (need && (!ws || ws_bytes < need)) {
            set_error("%s: workspace of %zu bytes needed, %zu given", who, need, ws ? ws_bytes : (size_t)0);
            return MOE_ERR_WORKSPACE;
        }
        const NormShape sh = shape_of(n->T, n->d, true);
        a.y = (void *)y;
        a.du = (const uint16_t *)du;
        a.dy = dy;
        a.dz = dz;
        a.dres = dresidual;
        a.dgate_row = channel ? nullptr : dgate;
        a.part = sums ? (float *)ws : nullptr;
        a.groups = sh.groups;
        launch_any(a, sh, n->z_dtype == MOE_DT_F32, n->y_dtype == MOE_DT_F32, true, s);
        MOE_TRY(launch_check(who));
    }
    if (sums) {                                           // (no tokens: zeros)
        const dim3 grid((unsigned)((n->d + 63) / 64), dw_before ? 2 : 1);
        hipLaunchKernelGGL(block_norm_sums_kernel, grid, dim3(64 * kSumWaves), 0, s, a.part, a.groups, n->d, w_after, channel ? gate : nullptr,
                           dw_after, channel ? dgate : nullptr, dw_before);
        MOE_TRY(launch_check(who));
    }
    return MOE_OK;
}
