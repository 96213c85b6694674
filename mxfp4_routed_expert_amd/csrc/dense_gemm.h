// The dense bf16 product kernel on the matrix cores (see dense.h for the products).
//
// A workgroup computes one BR x BC tile of the output; each wave owns a (16 TR) x (16 TC) part as
// MFMA tiles.  The columns operand is the MFMA's first operand and the rows operand its second,
// so a lane's four accumulators are four consecutive columns of one row.  The sum advances in
// steps of 64 values; the operands of one to three steps (kStages) are in LDS, copied there from
// global memory without passing through registers, while earlier ones are multiplied.
//
// LDS of a step.  An operand contiguous along the sum is kept as rows of 64 values (128 bytes),
// 16-byte chunk c of row r at position c ^ ((r >> 1) & 7): an operand read takes one chunk of 16
// rows and touches each 16-byte bank group once.  An operand strided along the sum is kept as it
// lies in memory, 64 rows (one per value of the sum) of BR or BC values, and read with the
// transposing LDS read (ds_read_b64_tr_b16): a group of 16 lanes supplies 4 rows of 16 values and
// lane i receives column i of the four.  Its 16-byte chunk c of row k sits at c ^ 2g(k), g(k) =
// (k & 3) | ((k >> 3) & 1) << 2: the eight 32-byte row pieces that half a wave reads then fall on
// eight different bank groups.  (The conflict counter reads 0 for all three forms.)
//
// Values past the end of the sum are copied from a zero page (for both operands), rows past the
// end of a matrix repeat its last row and their results are not stored.
//
// What bounds it.  A step of the 256 x 256 tile is 2048 cycles of matrix instructions, 1.0 - 1.1 us at the 1.9 -
// 2.1 GHz that the card holds under them; it measures 1.05 - 1.15 us with its operands in the last-level cache (4096
// x 4096 x 8192: 182 us, 1.51 PFLOP/s) and 1.3 - 1.4 from HBM.  A step of a 128 x 128 tile (512 cycles) measures
// 0.41 us from the last-level cache and 0.58 from HBM: a CU's misses in flight are limited, to 47 bytes a ns from
// HBM and 77 from the last-level cache against 115 of L2 hits, however many copies are issued ahead (four and
// five stages measured the same as three).
#pragma once
#include "dense.h"

namespace moe {

// The shapes, with sizes at which each is the fastest (us, operands from HBM):
//   4093 x 7168 x 2048                              L 115  B 128  M 148  D 157  S 163
//   1024 x 7168 x 2048                              B 34.5  M 40  D 46  S 52  L 56
//   512 x 7168 x 2368                               D 28  S 34  B 36  M 39  L 63
//   input gradient, 2060 x 7176 x 272               M 26  S 31  B 33  D 33  L 34
//   16 x 7168 x 2048, the sum split by 4            S 14.4  D 16  M 18  L 24
//   weight gradient, 2048 x 2048 over 512 tokens    M 12.9  B 13.2  W 15.6  L 19.7
//   weight gradient, 2368 x 7168 over 333 tokens    W 25  M 28  B 31  L 33
struct CfgL {                // 8 waves of 128 x 64, alternating
    static constexpr int BR = 256, BC = 256, WR = 2, WC = 4, kStages = 2;
    static constexpr bool kAlternate = true;
};
struct CfgM {                // 4 waves of 64 x 64, two workgroups a CU: one's start and end beside the other's products
    static constexpr int BR = 128, BC = 128, WR = 2, WC = 2, kStages = 2;
    static constexpr bool kAlternate = false;
};
struct CfgS {                // 4 waves of 64 x 32, two workgroups a CU
    static constexpr int BR = 64, BC = 128, WR = 1, WC = 4, kStages = 3;
    static constexpr bool kAlternate = false;
};
struct CfgW {                // as M with one buffer and one set of operands: four workgroups a CU, for the short sums of weight gradients
    static constexpr int BR = 128, BC = 128, WR = 2, WC = 2, kStages = 1;
    static constexpr bool kAlternate = false;
};
struct CfgD {                // as M with a step more in flight, one workgroup a CU
    static constexpr int BR = 128, BC = 128, WR = 2, WC = 2, kStages = 3;
    static constexpr bool kAlternate = false;
};
struct CfgB {                // 8 waves of 64 x 64: half the misses of D for the columns operand of a product
    static constexpr int BR = 256, BC = 128, WR = 4, WC = 2, kStages = 3;
    static constexpr bool kAlternate = false;
};

constexpr int kBK = 64;
#define MOE_INLINE __attribute__((always_inline))

struct GemmArgs {
    DenseProduct p;
    int tr, tc, full, split, steps, seg_steps;
    int cs_sub;           // column-sum rows per wave row of a tile
    float *part;
    int main_wgs, side_wgs;   // workgroups of the product; the next ones run `side`, those past them `later`
    DenseSide side;
    DenseLater later;
};

__device__ __attribute__((aligned(16))) const uint32_t g_dense_zero[4] = {0, 0, 0, 0};

// global -> LDS copies, 16 bytes a lane, to dst + 16 lane (asm: the compiler would otherwise wait for
// all copies in flight before every LDS read; the loop waits for exactly what it needs; the s_nop is the
// wait state between a write of M0 and its use by a copy).
MOE_DEV void copy16(const void *base, uint32_t voff, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
MOE_DEV void copy16_addr(const void *src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(lds) : "memory");
}
MOE_DEV const uint16_t *uniform16(const uint16_t *q) {
    const uint64_t v = (uint64_t)(uintptr_t)q;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint16_t *)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// (by value: a choice between captured variables would put them all in scratch memory)
MOE_DEV const uint16_t *pick(int i, const uint16_t *a, const uint16_t *b, const uint16_t *c) { return i == 0 ? a : (i == 1 ? b : c); }

MOE_DEV int ks_swz(int k) { return ((k & 3) | (((k >> 3) & 1) << 2)) << 1; }

// One operand's tile of N free indices: copies of a step and MFMA operand reads.
template <bool STRIDED, int N, int NW>
struct Operand {
    static constexpr int kBytes = N * kBK * 2;                // of one step
    static constexpr int kCopies = kBytes / 1024 / NW;        // copy instructions per wave and step
    static_assert(kBytes % (1024 * NW) == 0, "whole copies per wave");
    static_assert(!STRIDED || N >= 128, "the chunk permutation of strided rows spans 16 chunks");
    uint32_t voff[kCopies];

    // this wave's copy t covers LDS bytes [(wave * kCopies + t) * 1024, +1024) of the step
    static MOE_DEV int slot(int wave, int t) { return wave * kCopies + t; }
    // contiguous: LDS row and chunk position of this lane's 16 bytes
    static MOE_DEV int kc_row(int wave, int t, int lane) { return slot(wave, t) * 8 + (lane >> 3); }
    static MOE_DEV int kc_chunk(int row, int lane) { return (lane & 7) ^ ((row >> 1) & 7); }
    // strided: k within the step and chunk of this lane's 16 bytes
    static constexpr int kRowLanes = N / 8;                   // lanes per k row
    static MOE_DEV int ks_k(int wave, int t, int lane) { return slot(wave, t) * (64 / kRowLanes) + lane / kRowLanes; }
    static MOE_DEV int ks_chunk(int k, int lane) { return (lane & (kRowLanes - 1)) ^ ks_swz(k); }
};

template <class Cfg, int FORM, class Epi>
__global__ __launch_bounds__(64 * Cfg::WR *Cfg::WC, Cfg::kStages == 1 ? 4 : 2) void dense_gemm_kernel(const GemmArgs ga, Epi epi) {
    constexpr int BR = Cfg::BR, BC = Cfg::BC, NW = Cfg::WR * Cfg::WC;
    constexpr int TR = BR / Cfg::WR / 16, TC = BC / Cfg::WC / 16;
    constexpr bool RS = FORM == kFormTN, CS = FORM != kFormNT, PAIR = Epi::kPair;
    static_assert(!PAIR || FORM == kFormNT, "pairs are forward products");
    using OpR = Operand<RS, BR, NW>;
    using OpC = Operand<CS, BC, NW>;
    constexpr int kStage = OpR::kBytes + OpC::kBytes;
    extern __shared__ __align__(16) unsigned char smem[];

    if constexpr (std::is_same_v<Epi, EpiStore>)
        if ((int)blockIdx.x >= ga.main_wgs) {
            const int wg = blockIdx.x - ga.main_wgs;
            if (wg < ga.side_wgs) {
                dense_side_job<64 * NW>(ga.side, wg, (float *)smem);
            } else if constexpr (Cfg::kStages == 1) {
                static_assert(64 * NW == kFinishThreads, "as in the launch of its own");
                f32x4 sa, sb;
                if (ga.later.q.lanes == 64) dense_finish_rows<64>(ga.later.q, ga.later.e, wg - ga.side_wgs, sa, sb);
                else dense_finish_rows<32>(ga.later.q, ga.later.e, wg - ga.side_wgs, sa, sb);
            }
            return;
        }
    const DenseProduct &p = ga.p;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int wr = wave / Cfg::WC, wc = wave % Cfg::WC;
    const int lr = lane & 15, lg = lane >> 4;

    // ---- which tile and part of the sum: of each launch part (full tiles, then split ones), XCD x
    // (workgroups x, x + 8, ...) takes a contiguous run
    const int tail = ga.tr * ga.tc - ga.full;
    const bool split_tile = (int)blockIdx.x >= ga.full;
    int slot, sp = 0;
    {
        const int b = split_tile ? blockIdx.x - ga.full : blockIdx.x, G = split_tile ? tail * ga.split : ga.full;
        const int x = b & 7, q = G >> 3, rem = G & 7;
        slot = x * q + min(x, rem) + (b >> 3);
        if (split_tile) {
            sp = slot / tail;
            slot = ga.full + slot - sp * tail;
        }
    }
    int tr, tc;
    tile_at(slot, ga.tr, ga.tc, tr, tc);
    constexpr int kPairCols = BC / 2;                       // columns of each matrix in a pair tile
    const int r0 = tr * BR, c0 = tc * (PAIR ? kPairCols : BC);
    const int parts = split_tile ? ga.split : 1;
    const int s0 = (int)((int64_t)ga.steps * sp / parts), s1 = (int)((int64_t)ga.steps * (sp + 1) / parts);

    // ---- copy sources
    OpR opr;
    OpC opc;
#pragma unroll
    for (int t = 0; t < OpR::kCopies; ++t) {
        if constexpr (!RS) {
            const int row = OpR::kc_row(wave, t, lane);
            opr.voff[t] = 2u * ((uint32_t)min(row, p.R - 1 - r0) * (uint32_t)p.ldr + 8u * OpR::kc_chunk(row, lane));
        } else {
            const int k = OpR::ks_k(wave, t, lane);
            opr.voff[t] = 2u * ((uint32_t)k * (uint32_t)p.ldr + (uint32_t)min(8 * OpR::ks_chunk(k, lane), p.rcols - 8 - r0));
        }
    }
    // pair tile: LDS row j of the columns operand is, within wave wc's 16 TC rows, gate column
    // j % (8 TC) in the first half and up column in the second
    constexpr int kWCols = 16 * TC, kHalf = 8 * TC;
    auto pair_mat = [&](int row) MOE_INLINE { return (row % kWCols) / kHalf; };
    auto pair_col = [&](int row) MOE_INLINE { return row / kWCols * kHalf + row % kHalf; };
#pragma unroll
    for (int t = 0; t < OpC::kCopies; ++t) {
        if constexpr (!CS) {
            const int row = OpC::kc_row(wave, t, lane);
            const int col = PAIR ? pair_col(row) : row;
            opc.voff[t] = 2u * ((uint32_t)min(col, p.C - 1 - c0) * (uint32_t)p.ldc + 8u * OpC::kc_chunk(row, lane));
        } else {
            const int k = OpC::ks_k(wave, t, lane);
            opc.voff[t] = 2u * ((uint32_t)k * (uint32_t)p.ldc + (uint32_t)min(8 * OpC::ks_chunk(k, lane), p.C - 8 - c0));
        }
    }

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
    // Copies of the next step (s0, s0 + 1, ... in order) into stage st.  The sources advance by a constant per
    // step and start over at a segment's end; all of it stays in scalar registers (a division per step in
    // their place cost more than the step's matrix instructions).
    int seg = s0 / ga.seg_steps;
    int live = p.K - (s0 - seg * ga.seg_steps) * kBK;        // values of the sum left in the segment
    const uint16_t *rb, *cb, *ub = nullptr;
    // (held in registers: a reload of the arguments inside the loop would make every LDS wait a full one)
    const uint16_t *rp0 = uniform16(p.rp[0]), *rp1 = uniform16(p.rp[1]), *rp2 = uniform16(p.rp[2]);
    const uint16_t *cp0 = uniform16(p.cp[0]), *cp1 = uniform16(p.cp[1]), *cp2 = uniform16(p.cp[2]);
    auto sources = [&](int k0) MOE_INLINE {
        rb = pick(seg, rp0, rp1, rp2);
        cb = pick(PAIR ? 0 : seg, cp0, cp1, cp2);
        rb += RS ? (size_t)k0 * p.ldr + r0 : (size_t)r0 * p.ldr + k0;
        cb += CS ? (size_t)k0 * p.ldc + c0 : (size_t)c0 * p.ldc + k0;
        if constexpr (PAIR) ub = cp1 + (size_t)c0 * p.ldc + k0;
    };
    sources(p.K - live);
    const size_t radv = RS ? (size_t)kBK * p.ldr : kBK, cadv = CS ? (size_t)kBK * p.ldc : kBK;
    // copy t (the rows operand's, then the columns operand's) into stage st; tail: the segment's last, partial step
    constexpr int kPer = OpR::kCopies + OpC::kCopies;
    auto piece = [&](auto tt, int st, auto tail) MOE_INLINE {
        constexpr int t = decltype(tt)::value;
        constexpr bool R = t < OpR::kCopies;
        constexpr int u = R ? t : t - OpR::kCopies;
        const uint32_t at = lds0 + st * kStage + (R ? OpR::slot(wave, u) * 1024 : OpR::kBytes + OpC::slot(wave, u) * 1024);
        uint32_t off;
        const uint16_t *b;
        int k;
        if constexpr (R) {
            off = opr.voff[u];
            b = rb;
            k = RS ? OpR::ks_k(wave, u, lane) : 8 * OpR::kc_chunk(OpR::kc_row(wave, u, lane), lane);
        } else {
            off = opc.voff[u];
            b = PAIR ? pick(pair_mat(OpC::slot(wave, u) * 8), cb, ub, ub) : cb;
            k = CS ? OpC::ks_k(wave, u, lane) : 8 * OpC::kc_chunk(OpC::kc_row(wave, u, lane), lane);
        }
        if constexpr (decltype(tail)::value) {
            const void *a = (const char *)b + off;
            copy16_addr(k < live ? a : (const void *)g_dense_zero, at);
        } else {
            copy16(uniform16(b), off, at);
        }
    };
    auto advance = [&]() MOE_INLINE {
        live -= kBK;
        if (live > 0) {
            rb += radv;
            cb += cadv;
            if constexpr (PAIR) ub += cadv;
        } else if (seg + 1 < p.nseg) {
            ++seg;
            live = p.K;
            sources(0);
        }
    };
    auto issue = [&](int st) MOE_INLINE {
        if (live >= kBK) static_for<kPer>([&](auto t) MOE_INLINE { piece(t, st, std::false_type{}); });
        else static_for<kPer>([&](auto t) MOE_INLINE { piece(t, st, std::true_type{}); });
        advance();
    };

    f32x4 acc[TC][TR];
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
        for (int j = 0; j < TR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    // MFMA operand of free indices f0 .. f0+15 (f0 a multiple of 16), values 32 ks + 8 lg .. +7
    auto frag_c = [&](int base, int f0, int ks) MOE_INLINE {            // contiguous
        const int at = base + f0 * 128 + lr * 128 + (((4 * ks + lg) ^ (lr >> 1)) << 4);
        return *(const bf16x8 *)(smem + at);
    };
    auto frag_s = [&](int base, int f0, int ks, auto width) MOE_INLINE { // strided
        constexpr int W = decltype(width)::value;            // free indices of the tile
        const int k = 32 * ks + 8 * lg + (lr >> 2);
        const int chunk = ((f0 >> 3) + ((lr & 3) >> 1)) ^ ks_swz(k);
        const int at = base + k * (2 * W) + chunk * 16 + (lr & 1) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(uintptr_t)(lds0 + at));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(uintptr_t)(lds0 + at + 4 * 2 * W));
        const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        return __builtin_bit_cast(bf16x8, v);
    };
    struct Frags {
        bf16x8 r[TR], c[TC];
    };
    // operand q of a half step, in the order the products want them: a column operand, the row operands, the other
    // column operands
    auto read_one = [&](Frags &f, auto qq, int st, int ks) MOE_INLINE {
        constexpr int q = decltype(qq)::value;
        if constexpr (q >= 1 && q <= TR) {
            constexpr int j = q - 1;
            const int f0 = wr * 16 * TR + 16 * j;
            if constexpr (RS) f.r[j] = frag_s(st * kStage, f0, ks, std::integral_constant<int, BR>{});
            else f.r[j] = frag_c(st * kStage, f0, ks);
        } else {
            constexpr int i = q == 0 ? 0 : q - TR;
            const int f0 = wc * 16 * TC + 16 * i, base = st * kStage + OpR::kBytes;
            if constexpr (CS) f.c[i] = frag_s(base, f0, ks, std::integral_constant<int, BC>{});
            else f.c[i] = frag_c(base, f0, ks);
        }
    };
    auto read = [&](Frags &f, int st, int ks) MOE_INLINE {
        static_for<TR + TC>([&](auto q) MOE_INLINE { read_one(f, q, st, ks); });
    };
    // The products of one half step, with the whole copies P0 .. P1-1 into stage st spread between them: a copy
    // occupies the CU's address unit for 16 cycles, and a wave that issues one after another waits for it
    // instead of multiplying.
    using Zero = std::integral_constant<int, 0>;
    using Half = std::integral_constant<int, kPer / 2>;
    using All = std::integral_constant<int, kPer>;
    auto multiply_copy = [&](const Frags &f, auto p0, auto p1, int st) MOE_INLINE {
        constexpr int n = decltype(p1)::value - decltype(p0)::value, every = TC * TR / (n > 0 ? n : 1);
        static_assert(n == 0 || every >= 1, "a copy between products");
        static_for<TC * TR>([&](auto m) MOE_INLINE {
            constexpr int i = m / TR, j = m % TR;
            if constexpr (n > 0 && m % every == 0 && m / every < n) {
                __builtin_amdgcn_sched_barrier(0);
                piece(std::integral_constant<int, decltype(p0)::value + m / every>{}, st, std::false_type{});
                __builtin_amdgcn_sched_barrier(0);
            }
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.c[i], f.r[j], acc[i][j], 0, 0, 0);
        });
    };
    // The products of one half step with the reads of the next one's operands between them (a wave that issues its
    // reads one after another waits for the LDS instead of multiplying), and the whole copies P0 .. P1-1 into stage cst.
    auto multiply_read = [&](const Frags &f, Frags &g, int st, int ks, auto p0, auto p1, int cst) MOE_INLINE {
        constexpr int NM = TC * TR, NR = TR + TC, read_every = NM * 3 / 4 / NR > 1 ? NM * 3 / 4 / NR : 1;
        constexpr int n = decltype(p1)::value - decltype(p0)::value, every = NM / (n > 0 ? n : 1);
        static_assert((n == 0 || every >= 1) && NR * read_every <= NM + read_every - 1, "reads and copies between products");
        static_for<NM>([&](auto m) MOE_INLINE {
            constexpr int i = m / TR, j = m % TR;
            if constexpr (m % read_every == 0 && m / read_every < NR) {
                read_one(g, std::integral_constant<int, m / read_every>{}, st, ks);
                __builtin_amdgcn_sched_barrier(0);
            }
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.c[i], f.r[j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (n > 0 && m % every == every - 1 && m / every < n) {
                piece(std::integral_constant<int, decltype(p0)::value + m / every>{}, cst, std::false_type{});
                __builtin_amdgcn_sched_barrier(0);
            }
        });
    };
    auto multiply = [&](const Frags &f) MOE_INLINE { multiply_copy(f, Zero{}, Zero{}, 0); };
    // Most steps' copies are whole ones of the current segment.  They run in loops without a branch, whose
    // instructions all fit beside the matrix instructions; a step at a segment's end, or with nothing more to copy,
    // runs by itself.
    auto next_source = [&]() MOE_INLINE {
        rb += radv;
        cb += cadv;
        if constexpr (PAIR) ub += cadv;
    };
    auto whole_steps = [&](int most) MOE_INLINE { return max(0, min(most, live / kBK)); };
    auto whole_done = [&](int n) MOE_INLINE {
        live -= n * kBK;
        if (n > 0 && live <= 0 && seg + 1 < p.nseg) {
            ++seg;
            live = p.K;
            sources(0);
        }
    };

    if constexpr (Cfg::kAlternate) {
        // Two waves share a SIMD: wave w of the first half of the workgroup and w + NW/2 of the second.  While
        // one multiplies (32 matrix instructions), the other reads its next operands from LDS, then they
        // change places at a barrier: the matrix cores never wait for an LDS read.  The second half runs one
        // phase behind.  A step is four phases of a wave: read, multiply, read, multiply; numbered from the
        // first half's, step s reads its buffer in phases 4s .. 4s + 3 (the last one is the second half's).
        // Step s + 1's copies into the other buffer go out between matrix instructions, the second half's in
        // phase 4s (its last of step s - 1), the first half's in 4s + 1, and have landed at the end of 4s + 3.
        auto phase_end = [&]() MOE_INLINE {
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        auto read_end = [&]() MOE_INLINE {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
        };
        auto copies_end = [&]() MOE_INLINE {                 // (also a read's or a multiplication's end)
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        Frags f;
        auto run = [&](auto second) MOE_INLINE {
            constexpr bool S2 = decltype(second)::value;
            // one step: with COPY, the whole copies of step s + 1 (first half) or s + 2 (second half)
            auto step = [&](int s, auto copy) MOE_INLINE {
                constexpr bool COPY = decltype(copy)::value;
                const int st = (s - s0) & 1;
                read(f, st, 0);
                read_end();
                if constexpr (COPY && !S2) multiply_copy(f, Zero{}, All{}, st ^ 1);
                else multiply(f);
                phase_end();
                read(f, st, 1);
                if constexpr (S2) {
                    copies_end();
                    __builtin_amdgcn_s_setprio(1);
                } else {
                    read_end();
                }
                if constexpr (COPY && S2) multiply_copy(f, Zero{}, All{}, st);
                else multiply(f);
                if constexpr (S2) phase_end();
                else copies_end();
                if constexpr (COPY) next_source();
            };
            constexpr int kAhead = S2 ? 2 : 1;
            if (S2) {
                if (s0 + 1 < s1) issue(1);
                phase_end();
            }
            int s = s0;
            while (s < s1) {
                const int n = whole_steps(s1 - kAhead - s);
                for (int i = 0; i < n; ++i, ++s) step(s, std::true_type{});
                whole_done(n);
                if (s >= s1) break;
                // a step whose copies are the segment's partial step, or none (they go out at its start, or, the second
                // half's, once it has read its last operands)
                const int st = (s - s0) & 1;
                if (!S2 && s + 1 < s1) issue(st ^ 1);
                read(f, st, 0);
                read_end();
                multiply(f);
                phase_end();
                read(f, st, 1);
                if constexpr (S2) copies_end();
                else read_end();
                if (S2 && s + 2 < s1) issue(st);
                multiply(f);
                if constexpr (S2) phase_end();
                else copies_end();
                ++s;
            }
            if (!S2) phase_end();
        };
        if (s0 < s1) {
            issue(0);
            copies_end();
            if (wave >= NW / 2) run(std::true_type{});
            else run(std::false_type{});
        }
    } else if constexpr (Cfg::kStages == 1) {
        // the CU's other workgroups multiply while this one copies
        Frags f;
        for (int s = s0; s < s1; ++s) {
            issue(0);
            asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int ks = 0; ks < kBK / 32; ++ks) {
                read(f, 0, ks);
                multiply(f);
            }
            if (s + 1 < s1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    } else {
        // Operands are read one 32-value half step ahead of the products that use them, so reads and matrix
        // instructions overlap.  After the barrier in the middle of step s every operand of it has been read:
        // its buffer is free, and the copies of step s + kStages go into it, between the matrix instructions of
        // the two half steps that follow.
        constexpr int kStages = Cfg::kStages;
        static_assert(kPer * (kStages - 2) < 64, "the wait counter's range");
        auto landed = [&](bool newer) MOE_INLINE {           // the oldest step's copies, then all waves meet
            if (newer) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kPer * (kStages - 2)) : "memory");
            else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        };
        // (tells the compiler that the older operands are there, so that it waits for no newer one)
        auto reads_done = [&]() MOE_INLINE { __builtin_amdgcn_s_waitcnt(0xc07f); };
        if (s0 < s1) {
            Frags f0, f1;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i)
                if (s0 + i < s1) issue(i);
            landed(s0 + kStages - 1 <= s1);
            if (s0 + kStages - 1 < s1) issue(kStages - 1);
            read(f0, 0, 0);
            read(f1, 0, 1);
            multiply(f0);
            // from the middle of step s to the middle of step s + 1
            int st = 0;
            auto step = [&](int s, auto copy) MOE_INLINE {
                constexpr bool COPY = decltype(copy)::value;
                landed(COPY || s + kStages <= s1);
                const int free = st;
                st = st + 1 == kStages ? 0 : st + 1;
                if (!COPY && s + kStages < s1) issue(free);
                reads_done();
                multiply_read(f1, f0, st, 0, Zero{}, std::conditional_t<COPY, Half, Zero>{}, free);
                reads_done();
                multiply_read(f0, f1, st, 1, Half{}, std::conditional_t<COPY, All, Half>{}, free);
                if constexpr (COPY) next_source();
            };
            int s = s0;
            while (s + 1 < s1) {
                const int n = whole_steps(s1 - kStages - s);
                for (int i = 0; i < n; ++i, ++s) step(s, std::true_type{});
                whole_done(n);
                if (s + 1 < s1) step(s++, std::false_type{});
            }
            multiply(f1);
        }
    }

    // ---- epilogue.  Lane (lr, lg) of MFMA tile (i, j) holds columns 4 lg .. 4 lg + 3 of row lr.  The
    // wave's tile goes through LDS (32 or 64 rows at a time, 16-byte chunk c of row r at c ^ (r & 15 or 7)) so
    // that 8 or 16 neighbouring lanes take one row: whole lines are read and written, and the
    // epilogue's code appears once.
    constexpr int kCh = 4 * TC;                              // 16-byte chunks of a float32 row of the wave's tile
    // MFMA tile rows per pass: as many as the operands' LDS holds, at most 4
    constexpr int kJP = NW * 4 * 16 * kCh * 16 <= Cfg::kStages * kStage ? 4 : 2;
    constexpr int kLanes = PAIR ? kCh / 2 : kCh, kRows = 64 / kLanes;
    constexpr int U = 4;                                     // row groups handled together
    static_assert(NW * kJP * 16 * kCh * 16 <= Cfg::kStages * kStage, "the passes fit in the operands' LDS");
    static_assert(kCh == 8 || kCh == 16, "chunk permutation");
    static_assert(kJP * 16 % (kRows * U) == 0, "whole groups");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");    // every wave has read its last operands
    unsigned char *mine = smem + wave * (kJP * 16 * kCh * 16);
    const int ec = lane % kLanes, er = lane / kLanes;
    const int c = c0 + wc * (PAIR ? kHalf : kWCols) + 4 * ec;
    const bool live_c = c < p.C;
    typename Epi::Cols cols = epi.cols(live_c ? c : 0);
    float *ptile = ga.part + (size_t)((slot - ga.full) * ga.split + sp) * (BR * BC) + (c - c0);
    f32x4 sa = kZero4, sb = kZero4;
    static_for<TR / kJP>([&](auto pass) {
#pragma unroll
        for (int j = 0; j < kJP; ++j)
#pragma unroll
            for (int i = 0; i < TC; ++i)
                *(f32x4 *)(mine + (16 * j + lr) * (kCh * 16) + (((4 * i + lg) ^ (lr & (kCh - 1))) << 4)) =
                    acc[i][pass * kJP + j];
#pragma unroll 1
        for (int it = 0; it < kJP * 16 / kRows; it += U) {
            const int row0 = it * kRows + er;                // rows row0 + u * kRows of the pass
            const int lrow = wr * 16 * TR + pass * kJP * 16 + row0, r = r0 + lrow;
            f32x4 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = row0 + u * kRows;
                const unsigned char *src = mine + row * (kCh * 16);
                a[u] = *(const f32x4 *)(src + ((ec ^ (row & (kCh - 1))) << 4));
                if constexpr (PAIR) b[u] = *(const f32x4 *)(src + (((ec + kLanes) ^ (row & (kCh - 1))) << 4));
            }
            if (!live_c || r >= p.R) continue;
            if (split_tile) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (r + u * kRows >= p.R) continue;
                    float *dst = ptile + (lrow + u * kRows) * BC;
                    *(f32x4 *)dst = a[u];
                    if constexpr (PAIR) *(f32x4 *)(dst + kPairCols) = b[u];
                }
            } else {
                epi.rows(cols, r, kRows, p.R, c, a, b, sa, sb);
            }
        }
    });
    if constexpr (Epi::kColSum) {
        if (epi.cs && !split_tile) {
            // the wave's 16 TR rows: cs_sub partial rows, the first with the sum
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int o = kLanes; o < 64; o <<= 1) {
                    sa[q] += __shfl_xor(sa[q], o, kWave);
                    if constexpr (PAIR) sb[q] += __shfl_xor(sb[q], o, kWave);
                }
            if (live_c) {
                float *row = epi.cs + (size_t)((tr * Cfg::WR + wr) * ga.cs_sub) * epi.csld;
                for (int i = er; i < ga.cs_sub; i += kRows) {
                    *(f32x4 *)(row + (size_t)i * epi.csld + c) = i ? kZero4 : sa;
                    if constexpr (PAIR) *(f32x4 *)(row + (size_t)i * epi.csld + p.C + c) = i ? kZero4 : sb;
                }
            }
        }
    }
}

// The product with its epilogue, and the sum of its split tiles: at once, or left in `leave`.  `later`: the one a
// product before this left.
template <class Cfg, int FORM, class Epi>
moe_status dense_run_cfg(const DenseProduct &p, const DensePlan &pl, const Epi &e, float *part, const DenseSide &side,
                         DenseLater *leave, const DenseLater &later, hipStream_t s) {
    constexpr int lds = Cfg::kStages * (Cfg::BR + Cfg::BC) * kBK * 2, kThreads = 64 * Cfg::WR * Cfg::WC;
    const int tiles = pl.tr * pl.tc;
    const bool tail = pl.full < tiles;
    GemmArgs ga{p, pl.tr, pl.tc, pl.full, pl.split, pl.steps, pl.steps / p.nseg, tail ? Cfg::BR / Cfg::WR / kFinishRows : 1,
                part, pl.full + (tiles - pl.full) * pl.split, dense_side_wgs(side, kThreads), side, later};
    hipLaunchKernelGGL((dense_gemm_kernel<Cfg, FORM, Epi>), dim3((unsigned)(ga.main_wgs + ga.side_wgs + later.q.wgs)), dim3(kThreads),
                       lds, s, ga, e);
    MOE_TRY(launch_check("dense product"));
    if (!tail) return MOE_OK;
    const int rows = p.R / p.terms, blocks = Cfg::BR / kFinishRows;
    const int sums = p.terms == 1 ? tiles - pl.full : (rows + Cfg::BR - 1) / Cfg::BR * pl.tc;
    const DenseParts q{part, pl.full, pl.split, p.terms, pl.tr, pl.tc, rows, p.C, Cfg::BR, Cfg::BC / 4 / (Epi::kPair ? 2 : 1), sums * blocks};
    if constexpr (std::is_same_v<Epi, EpiStore>)
        if (leave) {
            *leave = DenseLater{q, e};
            return MOE_OK;
        }
    return dense_finish(q, e, s);
}

template <int FORM, class Epi>
moe_status dense_run(const DenseProduct &p, const DensePlan &pl, const Epi &e, float *part, hipStream_t s, const DenseSide &side = {},
                     DenseLater *leave = nullptr, const DenseLater &later = {}) {
    if (pl.cfg == kTileL) return dense_run_cfg<CfgL, FORM>(p, pl, e, part, side, leave, later, s);
    if (pl.cfg == kTileB) return dense_run_cfg<CfgB, FORM>(p, pl, e, part, side, leave, later, s);
    if constexpr (FORM == kFormTN) {
        if (pl.cfg == kTileW) return dense_run_cfg<CfgW, FORM>(p, pl, e, part, side, leave, later, s);
    } else {
        if (pl.cfg == kTileS) return dense_run_cfg<CfgS, FORM>(p, pl, e, part, side, leave, later, s);
        if (pl.cfg == kTileD) return dense_run_cfg<CfgD, FORM>(p, pl, e, part, side, leave, later, s);
    }
    return dense_run_cfg<CfgM, FORM>(p, pl, e, part, side, leave, later, s);
}

}  // namespace moe
