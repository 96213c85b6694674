// Products of block-128 FP8 operands on the matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4).
//
// One instruction sums a whole 128-block of a 16 x 16 tile.  The weight rows are its first operand and
// the activation rows its second, so a lane's four accumulators are four consecutive columns of one
// activation row, and that row's E8M0 scale goes in as the second operand's scale.  A weight's E8M0
// scale (128 x 128 block, or one per row) goes in as the first operand's scale: the accumulators run on in the
// instruction.  A float32 weight scale cannot: the block's product is formed from zero and added with a fused
// multiply, acc += s p; s is the same in every lane, since a wave's weight rows lie in one 128-block.
//
// Item: up to 256 activation rows of one expert (or of the one matrix) by 256 weight rows (the gated pair: 128
// columns of gate and of up).  8 waves, two along the weight rows and four along the activation rows; a wave
// owns 128 weight rows x 16 TT activation rows (TT = 4, 3, 2, 1 by how many rows there are).  The sum advances by
// one block, 128 bytes a row; the operands of two (TT = 4, 3) or three steps are in LDS, copied there without
// passing through registers.  16-byte chunk c of LDS row r is at c ^ ((r >> 1) & 7): an operand read takes one
// chunk of 16 rows and touches each bank group once.
//
// The instruction aligns each group of 8 neighbouring products to the largest and keeps 13 bits below it (measured by adding
// powers of two): a sum of 8 loses under 7 2^-13 of its largest product.  It is the only FP8 product the matrix cores
// have; everything added after it, block sums and scales, is float32.
//
// Measured: 8192 x 8192 x 8192 with E8M0 scales 381 us (2.88 PFLOP/s), with float32 ones 502 (the fused multiplies share the
// issue slots: registers alone give 4.1 PFLOP/s without and 3.3 with them); 4096 x 7168 x 7168 173 to 186 with E8M0 scales (the
// matrix cores 58 % busy), with float32 ones 205 to 237 by card (44 %), float32 results the same.  With 256 experts of 6144 x 2048, top 8,
// and 4096 tokens the weights' bytes bound it: 1500 to 1556 us for gate and up, 4.2 TB/s.
#include <algorithm>

#include "fp8.h"
#include "tile_sched.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWRows = 256, kMaxRows = 256;
// Blocks whose scales are in LDS at a time, one byte a row and block (row stride odd in dwords: 16 rows, 16 banks).
constexpr int window_of(int WK) { return WK == MOE_FP8_SCALE_E8M0_ROW ? 32 : 64; }
constexpr int scale_row(int WK) { return window_of(WK) + 4; }

constexpr int stages_of(int TT) { return TT >= 3 ? 2 : 3; }
constexpr int stage_bytes(int TT) { return (kWRows + 64 * TT) * 128; }
constexpr int panel_bytes(int WK, int TT) { return (64 * TT + (WK == MOE_FP8_SCALE_E8M0_ROW ? kWRows : 0)) * scale_row(WK); }
constexpr int lds_of(int WK, int TT) { return stages_of(TT) * stage_bytes(TT) + panel_bytes(WK, TT); }
constexpr int cmax(int a, int b) { return a > b ? a : b; }
constexpr int lds_bytes(int WK) { return cmax(cmax(lds_of(WK, 4), lds_of(WK, 3)), cmax(lds_of(WK, 2), lds_of(WK, 1))); }

__device__ __attribute__((aligned(16))) const uint32_t g_fp8_zero[4] = {0, 0, 0, 0};

// global -> LDS copies of 16 bytes a lane to dst + 16 lane (asm: the compiler would otherwise wait for all copies in
// flight before every LDS read; s_nop is the wait state between a write of M0 and its use).
MOE_DEV void copy16(const void *base, uint32_t voff, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
MOE_DEV void copy16_addr(const void *src, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(lds) : "memory");
}
MOE_DEV const uint8_t *uniform(const void *q) {
    const uint64_t v = (uint64_t)(uintptr_t)q;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t *)(uintptr_t)(((uint64_t)hi << 32) | lo);
}
constexpr int kNowhere = 0x7ffffff0;                      // an offset past every buffer

// The lane id, read so that the compiler neither hoists it nor keeps values derived from it alive across a loop.
MOE_DEV int lane_fresh() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}
MOE_DEV uint32_t bf16_pair(float a, float b) {            // round to nearest even
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
MOE_DEV void lds_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Rows [m0, m0 + live) of expert e (first sorted row row0) by weight rows n0 .. (pair: columns n0 .. of gate and up),
// blocks [s0, s1) of the sum, part `sp` of it.
struct Unit {
    int e, row0, m0, live, n0, s0, s1, sp;
};

// Four scale bytes from byte `at` of a row of `left` more bytes (bytes past the row's end are not read).
MOE_DEV uint32_t scale_word(const uint8_t *p, int left) {
    uint32_t v = 0;
    if (left >= 4) {
        __builtin_memcpy(&v, p, 4);
    } else {
        if (left > 0) v = p[0];
        if (left > 1) v |= (uint32_t)p[1] << 8;
        if (left > 2) v |= (uint32_t)p[2] << 16;
    }
    return v;
}

template <bool PAIR, int WK, int TT, bool S2>
MOE_DEV void fp8_unit(const Fp8Product &p, const Unit &u, unsigned char *smem, const int *s_row) {
    constexpr int ST = stages_of(TT), kStage = stage_bytes(TT), kXAt = kWRows * 128;
    constexpr int kWindow = window_of(WK), kScaleRow = scale_row(WK);
    constexpr int kPanel = ST * kStage, kWPanel = kPanel + 64 * TT * kScaleRow;
    constexpr int kPer = 4 + TT;                          // copies of a wave and step
    // (as the streamed form: of few rows h is to be exact to float32, or single values on the next 8-bit code show; 32 rows an
    // expert, 256 of 6144 x 2048, gate and up 1490 us for 1415, 16 of 2048 x 1024 all three 51 for 44)
    constexpr bool EXACT = PAIR && TT == 1;
    const int lane = lane_fresh(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int wn = wave >> 2, wt = wave & 3;
    const int lr = lane & 15, lg = lane >> 4;
    const int K = p.K, Kb = p.Kb;

    // ---- copy sources.  Wave w copies weight rows 32w .. 32w + 31 of the item, and activation rows 8 TT w ...
    // Pair: LDS weight row q holds, within wave row wn = q / 128, gate column 64 wn + q % 64 in the first half
    // and the up column in the second.
    const int wrow0 = 32 * wave;
    const int mat = PAIR ? (wrow0 >> 6) & 1 : 0;
    const int wcol0 = PAIR ? (wrow0 >> 7) * 64 + (wrow0 & 63) : wrow0;
    const uint8_t *wbase = uniform((mat ? p.w[1] : p.w[0]) + ((size_t)u.e * p.N + u.n0) * K + (size_t)u.s0 * 128);
    const uint8_t *xbase = uniform(p.x + (size_t)u.s0 * 128);
    const int cr = lane >> 3, cp = lane & 7;
    uint32_t woff[4], xoff[TT];
    auto chunk_of = [&](int q) __attribute__((always_inline)) { return cp ^ ((q >> 1) & 7); };
#pragma unroll
    for (int t = 0; t < 4; ++t)
        woff[t] = (uint32_t)min(wcol0 + 8 * t + cr, p.N - 1 - u.n0) * (uint32_t)K + 16u * chunk_of(wrow0 + 8 * t + cr);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int q = 8 * TT * wave + 8 * t + cr;
        xoff[t] = (uint32_t)s_row[q] * (uint32_t)K + 16u * chunk_of(q);
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
    const uint32_t wdst = lds0 + wrow0 * 128, xdst = lds0 + kXAt + 8 * TT * wave * 128;
    int live = K - 128 * u.s0;                            // bytes of a row left from the next step to copy
    // copy t of a step into buffer st; TAIL: the row's last, partial block, zeros past its end
    auto piece = [&](auto tt, int st, auto tail) __attribute__((always_inline)) {
        constexpr int t = decltype(tt)::value;
        constexpr bool W = t < 4;
        constexpr int v = W ? t : t - 4;
        const uint32_t at = (W ? wdst : xdst) + st * kStage + v * 1024;
        const uint32_t off = W ? woff[W ? v : 0] : xoff[W ? 0 : v];
        const uint8_t *base = W ? wbase : xbase;
        if constexpr (decltype(tail)::value) {
            // (read anew: 64-bit offsets kept across the steps would cost their registers)
            const int l = lane_fresh(), q = (W ? wrow0 : 8 * TT * wave) + 8 * v + (l >> 3);
            const int c = (l & 7) ^ ((q >> 1) & 7);
            uint32_t o = off;
            asm volatile("" : "+v"(o));
            copy16_addr(16 * c < live ? (const void *)(base + o) : (const void *)g_fp8_zero, at);
        } else {
            copy16(base, off, at);
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        live -= 128;
        wbase += 128;
        xbase += 128;
    };
    auto issue = [&](int st) __attribute__((always_inline)) {
        if (live >= 128) static_for<kPer>([&](auto t) __attribute__((always_inline)) { piece(t, st, std::false_type{}); });
        else static_for<kPer>([&](auto t) __attribute__((always_inline)) { piece(t, st, std::true_type{}); });
        advance();
    };

    // ---- scales of blocks b0 .. b0 + kWindow - 1.  Rows' bytes go to LDS; a block scale sits in lane b - b0's register.
    float wf[2] = {0.f, 0.f};
    uint32_t we[2] = {0, 0};
    const int nblk = (PAIR ? u.n0 : u.n0 + 128 * wn) >> 7, NB = (p.N + 127) >> 7;
    auto window = [&](int b0) __attribute__((always_inline)) {
        constexpr int kWords = kWindow / 4, kRowsPass = kThreads / kWords;
        const int tid = 64 * wave + lane_fresh(), d = 4 * (tid & (kWords - 1));
#pragma unroll
        for (int i = 0; i < 64 * TT / kRowsPass; ++i) {
            const int q = kRowsPass * i + tid / kWords;
            *(uint32_t *)(smem + kPanel + q * kScaleRow + d) = scale_word(p.xs + (size_t)s_row[q] * Kb + b0 + d, Kb - b0 - d);
        }
        if constexpr (WK == MOE_FP8_SCALE_E8M0_ROW) {
#pragma unroll
            for (int i = 0; i < kWRows / kRowsPass; ++i) {
                const int q = kRowsPass * i + tid / kWords;
                *(uint32_t *)(smem + kWPanel + q * kScaleRow + d) =
                    scale_word((const uint8_t *)p.ws[0] + (size_t)min(u.n0 + q, p.N - 1) * Kb + b0 + d, Kb - b0 - d);
            }
        } else {
            const size_t at = ((size_t)u.e * NB + min(nblk, NB - 1)) * Kb + min(b0 + (lane & (kWindow - 1)), Kb - 1);
#pragma unroll
            for (int m = 0; m < (PAIR ? 2 : 1); ++m) {
                if constexpr (WK == MOE_FP8_SCALE_F32) wf[m] = ((const float *)p.ws[m])[at];
                else we[m] = ((const uint8_t *)p.ws[m])[at];
            }
        }
    };

    f32x4 acc[8][TT];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int sw0 = (lg ^ (lr >> 1)) << 4, sw1 = ((4 + lg) ^ (lr >> 1)) << 4;
    const int arow = (128 * wn + lr) * 128, xrow = kXAt + (16 * TT * wt + lr) * 128;
    auto frag = [&](int at) __attribute__((always_inline)) {
        const u32x4 a = *(const u32x4 *)(smem + at + sw0), b = *(const u32x4 *)(smem + at + sw1);
        return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
    };
    // Operands of half a step: the activation tiles and weight tiles 0 - 3, then weight tiles 4 - 7.  b: the block within the window.
    struct Ops {
        i32x8 a[4], x[TT];
        int sx[TT], sw[4];
        float f;
        int e8;
    } o;
    auto read = [&](int st, int b, auto hh) __attribute__((always_inline)) {
        constexpr int H = decltype(hh)::value;
        if constexpr (H == 0) {
#pragma unroll
            for (int j = 0; j < TT; ++j) o.sx[j] = smem[kPanel + (16 * TT * wt + 16 * j + lr) * kScaleRow + b];
#pragma unroll
            for (int j = 0; j < TT; ++j) o.x[j] = frag(st * kStage + xrow + j * 2048);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (WK == MOE_FP8_SCALE_E8M0_ROW) o.sw[i] = smem[kWPanel + (128 * wn + 64 * H + 16 * i + lr) * kScaleRow + b];
            o.a[i] = frag(st * kStage + arow + (4 * H + i) * 2048);
        }
        constexpr int m = PAIR ? H : 0;
        if constexpr (WK == MOE_FP8_SCALE_F32) o.f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wf[m]), b));
        if constexpr (WK == MOE_FP8_SCALE_E8M0) o.e8 = __builtin_amdgcn_readlane((int)we[m], b);
    };
    // Their products, with copies P0 .. P1 - 1 of a later step into buffer cst between them.  Float32 weight scales: a
    // block's product is added three products later (a result may be read 11 instructions after its product); the half's last
    // three are left to settle(), which a wave calls when the other one multiplies.
    constexpr int kBehind = 3, kNM = 4 * TT;
    f32x4 q[kBehind + 1];
    auto add = [&](auto hh, auto mm, float f) __attribute__((always_inline)) {
        constexpr int H = decltype(hh)::value, m = decltype(mm)::value, i = m / TT, j = m % TT;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[4 * H + i][j][v] = fmaf(q[m % (kBehind + 1)][v], f, acc[4 * H + i][j][v]);
    };
    auto settle = [&](auto hh, float f) __attribute__((always_inline)) {
        if constexpr (WK == MOE_FP8_SCALE_F32 && !EXACT)
            static_for<kBehind>([&](auto mm) __attribute__((always_inline)) { add(hh, std::integral_constant<int, kNM - kBehind + decltype(mm)::value>{}, f); });
    };
    auto multiply = [&](auto hh, auto p0, auto p1, int cst) __attribute__((always_inline)) {
        constexpr int H = decltype(hh)::value, P0 = decltype(p0)::value, n = decltype(p1)::value - P0, NM = kNM;
        if constexpr (EXACT) {
            f32x4 r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bf16x8 xk = fp8_widen8(o.x[0], k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    r[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_widen8(o.a[i], k), xk, k ? r[i] : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            }
            const float f = o.f * e8m0_to_f32((uint8_t)o.sx[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[4 * H + i][0][v] = fmaf(r[i][v], f, acc[4 * H + i][0][v]);
            return;
        }
        static_for<NM>([&](auto mm) __attribute__((always_inline)) {
            constexpr int m = decltype(mm)::value, i = m / TT, j = m % TT;
            if constexpr (WK == MOE_FP8_SCALE_F32) {
                q[m % (kBehind + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(o.a[i], o.x[j], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, o.sx[j]);
            } else {
                const int se = WK == MOE_FP8_SCALE_E8M0_ROW ? o.sw[i] : o.e8;
                acc[4 * H + i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(o.a[i], o.x[j], acc[4 * H + i][j], 0, 0, 0, se, 0, o.sx[j]);
            }
            // (copy c goes out after product c NM / n)
            static_for<n>([&](auto cc) __attribute__((always_inline)) {
                if constexpr (decltype(cc)::value * NM / n == m) piece(std::integral_constant<int, P0 + decltype(cc)::value>{}, cst, std::false_type{});
            });
            if constexpr (WK == MOE_FP8_SCALE_F32 && m >= kBehind) add(hh, std::integral_constant<int, m - kBehind>{}, o.f);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    using C0 = std::integral_constant<int, 0>;
    using CN = std::integral_constant<int, kPer>;

    for (int w0 = u.s0 & ~(kWindow - 1); w0 < u.s1; w0 += kWindow) {
        const int s0 = max(w0, u.s0), s1 = min(w0 + kWindow, u.s1);
        if (w0 > u.s0) lds_meet();                        // every wave has read its last operands and scales
        if constexpr (TT >= 2) {
            // Two waves share a SIMD: w of the first half of the workgroup and w + 4 of the second.  While one multiplies
            // (4 TT matrix instructions), the other reads its next operands from LDS, then they change places at a barrier.
            // The second half runs one phase behind.  A step is four phases of a wave: read, multiply, read, multiply;
            // numbered from the first half's, step s reads its buffer in phases 4s .. 4s + 3 (the last one is the
            // second half's).  With ST buffers, the copies of step s + ST - 1 go out between matrix instructions into the buffer
            // of step s - 1, the second half's in phase 4s (its last of step s - 1), the first half's in 4s + 1; those of step
            // s + 1 have landed at the end of 4s + 3.
            auto phase_end = [&]() __attribute__((always_inline)) {
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("s_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            };
            auto read_end = [&]() __attribute__((always_inline)) {
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
            };
            // (also a read's or a multiplication's end; newer: the copies of ST - 2 newer steps are on their way)
            auto copies_end = [&](auto newer) __attribute__((always_inline)) {
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (decltype(newer)::value) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kPer * (ST - 2)) : "memory");
                else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            };
            constexpr int kAhead = S2 ? ST : ST - 1;      // the step whose copies a wave issues, past its own
            int st = 0;                                   // the step's buffer
            auto step = [&](int s, auto copy) __attribute__((always_inline)) {
                constexpr bool COPY = decltype(copy)::value;
                const int b = s - w0, into = S2 ? st : st == 0 ? ST - 1 : st - 1;
                if (!COPY && !S2 && s + kAhead < s1) issue(into);
                read(st, b, H0{});
                read_end();
                multiply(H0{}, C0{}, std::conditional_t<COPY && !S2, CN, C0>{}, into);
                phase_end();
                const float f0 = o.f;
                read(st, b, H1{});
                settle(H0{}, f0);
                if constexpr (S2) {
                    copies_end(copy);
                    __builtin_amdgcn_s_setprio(1);
                } else {
                    read_end();
                }
                if (!COPY && S2 && s + kAhead < s1) issue(into);
                multiply(H1{}, C0{}, std::conditional_t<COPY && S2, CN, C0>{}, into);
                if constexpr (S2) phase_end();
                else copies_end(copy);
                settle(H1{}, o.f);
                if constexpr (COPY) advance();
                st = st + 1 == ST ? 0 : st + 1;
            };
#pragma unroll
            for (int i = 0; i < ST - 1; ++i)
                if (s0 + i < s1) issue(i);
            window(w0);
            copies_end(std::false_type{});
            if (S2) {
                if (s0 + ST - 1 < s1) issue(ST - 1);
                phase_end();
            }
            // (steps whose copies are whole blocks run without a branch; a row's partial block is its last)
            const int sc = s0 + max(0, min(s1 - kAhead - s0, live >> 7));
            int s = s0;
            for (; s < sc; ++s) step(s, std::true_type{});
            for (; s < s1; ++s) step(s, std::false_type{});
            if (!S2) phase_end();
        } else {
            // At the top of step s its copies have landed (the newer steps' may be in flight) and every wave is done with
            // step s - 1, whose buffer takes the copies of step s + ST - 1.
            window(w0);
#pragma unroll
            for (int i = 0; i < ST - 1; ++i)
                if (s0 + i < s1) issue(i);
            int st = 0;
            for (int s = s0; s < s1; ++s) {
                if (s + ST - 1 <= s1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kPer * (ST - 2)) : "memory");
                else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
                if (s + ST - 1 < s1) issue(st == 0 ? ST - 1 : st - 1);
                read(st, s - w0, H0{});
                multiply(H0{}, C0{}, C0{}, 0);
                const float f0 = o.f;
                read(st, s - w0, H1{});
                settle(H0{}, f0);
                multiply(H1{}, C0{}, C0{}, 0);
                settle(H1{}, o.f);
                st = st + 1 == ST ? 0 : st + 1;
            }
        }
    }
    lds_meet();                                           // every wave has read its last operands

    // ---- epilogue.  Lane (lr, lg) of tile (i, j) holds weight rows 4 lg .. of activation row lr.
    const int el = lane_fresh(), elr = el & 15, elg = el >> 4;
    if constexpr (!PAIR) {
        // A wave's 16 rows x 128 columns at a time through LDS: 32 lanes a row, whole lines.  A row's residual is read before
        // it is written (it may be y), 16 rows at once.
        unsigned char *mine = smem + wave * 8192;
        const int ec = el & 31, er = el >> 5;
        const int c = u.n0 + 128 * wn + 4 * ec;
        const bool whole = (p.N & 3) == 0;                // 4 columns are one access, all or none of them there
        const bool f32 = p.split > 1 || p.y_f32;
        const int size = f32 ? 4 : 2;
        const unsigned char *res = p.split > 1 ? nullptr : (const unsigned char *)p.residual;
        unsigned char *y = p.split > 1 ? (unsigned char *)(p.part + (size_t)u.sp * p.R * p.N) : (unsigned char *)p.y;
        // Two rows as a buffer: accesses past the last live row are dropped (reads give 0), as are those at kNowhere.
        const int off = c < p.N ? (er * p.N + c) * size : kNowhere;
        auto rows = [&](const unsigned char *base, int r) __attribute__((always_inline)) {
            const int there = min(max(u.live - r, 0), 2);
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char *>(base) + (size_t)(u.row0 + u.m0 + r) * p.N * size, 0,
                                                     base ? there * p.N * size : 0, 0x00027000);
        };
#pragma unroll
        for (int j = 0; j < TT; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) *(f32x4 *)(mine + elr * 512 + (((4 * i + elg) ^ elr) << 4)) = acc[i][j];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            const int r0 = 16 * TT * wt + 16 * j;
            auto value = [&](int it) __attribute__((always_inline)) {
                const int rr = 2 * it + er;
                return *(const f32x4 *)(mine + rr * 512 + ((ec ^ rr) << 4));
            };
            if (whole && f32) {
                u32x4 rv[8];
#pragma unroll
                for (int it = 0; it < 8; ++it) rv[it] = u32x4{0, 0, 0, 0};
                if (res) {
#pragma unroll
                    for (int it = 0; it < 8; ++it) rv[it] = __builtin_amdgcn_raw_buffer_load_b128(rows(res, r0 + 2 * it), off, 0, 0);
                }
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    f32x4 v = value(it);
                    if (res) v += __builtin_bit_cast(f32x4, rv[it]);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rows(y, r0 + 2 * it), off, 0, 0);
                }
            } else if (whole) {
                u32x2 rv[8];
#pragma unroll
                for (int it = 0; it < 8; ++it) rv[it] = u32x2{0, 0};
                if (res) {
#pragma unroll
                    for (int it = 0; it < 8; ++it) rv[it] = __builtin_amdgcn_raw_buffer_load_b64(rows(res, r0 + 2 * it), off, 0, 0);
                }
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    f32x4 v = value(it);
                    const f32x2 ra = bf16x2_to_f32x2(rv[it][0]), rb = bf16x2_to_f32x2(rv[it][1]);
                    if (res) v += f32x4{ra.x, ra.y, rb.x, rb.y};
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, rows(y, r0 + 2 * it), off, 0, 0);
                }
            } else {
#pragma unroll 1
                for (int it = 0; it < 8; ++it) {
                    const __amdgpu_buffer_rsrc_t yb = rows(y, r0 + 2 * it), rb = rows(res, r0 + 2 * it);
                    const f32x4 v = value(it);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int o = c + q < p.N ? off + q * size : kNowhere;
                        if (f32) {
                            const float add = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rb, o, 0, 0));
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(res ? v[q] + add : v[q]), yb, o, 0, 0);
                        } else {
                            const float add = bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, o, 0, 0));
                            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_pair(res ? v[q] + add : v[q], 0.0f), yb, o, 0, 0);
                        }
                    }
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
    } else {
        // h = silu(g) u through LDS, then 16 lanes take a row's 128 columns: the block's largest value, its codes
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 h;
#pragma unroll
                for (int v = 0; v < 4; ++v) h[v] = fp8_silu(acc[i][j][v]) * acc[i + 4][j][v];
                const int r = 16 * TT * wt + 16 * j + elr;
                *(f32x4 *)(smem + r * 512 + (((16 * wn + 4 * i + elg) ^ elr) << 4)) = h;
            }
        __syncthreads();
        const int q = el & 15;
#pragma unroll
        for (int it = 0; it < 2 * TT; ++it) {
            const int r = 32 * it + 4 * wave + (el >> 4);
            const f32x4 a = *(const f32x4 *)(smem + r * 512 + (((2 * q) ^ (r & 15)) << 4));
            const f32x4 b = *(const f32x4 *)(smem + r * 512 + (((2 * q + 1) ^ (r & 15)) << 4));
            uint32_t m = 0;
#pragma unroll
            for (int v = 0; v < 4; ++v) m = max(m, max(fp8_magnitude(a[v]), fp8_magnitude(b[v])));
            m = fp8_max16(m);
            if (r >= u.live) continue;
            const int X = fp8_exponent(m);
            const float inv = fp8_inverse(X);
            const size_t orow = (size_t)(u.row0 + u.m0 + r);
            const size_t at = orow * p.N + u.n0 + 8 * q;
            if (p.h) {
                *(f32x4 *)(p.h + at) = a;
                *(f32x4 *)(p.h + at + 4) = b;
            }
            *(u32x2 *)(p.hq + at) = u32x2{fp8_codes4(a[0], a[1], a[2], a[3], inv), fp8_codes4(b[0], b[1], b[2], b[3], inv)};
            if (q == 0) p.hs[orow * (p.N >> 7) + (u.n0 >> 7)] = (uint8_t)(X + 127);
        }
    }
}

// One workgroup a CU, persistent: each walks its share of the units.  Units: row tiles (of bt rows) x column tiles x
// parts of the sum; the items of a last, partial round are split by rows into halves or quarters (routed form).
template <bool PAIR, bool ROUTED, int WK>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void fp8_gemm_kernel(const Fp8Product p) {
    __shared__ __align__(16) unsigned char smem[lds_bytes(WK)];
    __shared__ uint16_t s_tp[ROUTED ? MOE_MAX_EXPERTS : 1];
    __shared__ int s_wave[kThreads / 64];
    __shared__ int s_row[kMaxRows];

    constexpr int kCols = PAIR ? 128 : 256;
    const int NT = (p.N + kCols - 1) / kCols;
    const int mt = ROUTED ? build_tile_prefix<kThreads, kMaxRows>(p.offsets, p.E, p.R, s_tp, s_wave) : (p.R + p.bt - 1) / p.bt;
    const int split = ROUTED ? 1 : p.split;
    const int bt = ROUTED ? kMaxRows : p.bt;
    const int items = mt * NT * split;
    const int G = gridDim.x;
    const int full = items / G * G, tail = items - full;
    // (parts of at least 64 rows)
    const int fmax = bt / 64;
    const int f = tail > 0 && 4 * tail <= G ? min(4, fmax) : (tail > 0 && 2 * tail <= G ? min(2, fmax) : 1);
    const int units = full + f * tail;
    const int slot = xcd_slot(blockIdx.x, G);
    for (int un = slot; un < units; un += G) {
        int item = un, part = 0, parts = 1;
        if (un >= full) {
            item = full + (un - full) / f;
            part = (un - full) % f;
            parts = f;
        }
        Unit u;
        int tile, nt, M;
        u.sp = 0;
        u.e = 0;
        u.row0 = 0;
        M = p.R;
        if constexpr (ROUTED) {
            u.e = __builtin_amdgcn_readfirstlane(tile_expert(s_tp, p.E, item / NT));
            const int before = u.e > 0 ? s_tp[u.e - 1] : 0, te = s_tp[u.e] - before;
            const int r = item - NT * before;
            nt = r / te;
            tile = r - nt * te;
            u.row0 = p.offsets[u.e];
            M = p.offsets[u.e + 1] - u.row0;
        } else {
            // (four column tiles share each row tile, so the 32 units of an XCD form a block of 8 x 4 tiles and share both
            // operands in its L2)
            u.sp = item / (NT * mt);
            const int r = item - u.sp * (NT * mt), g = r / (4 * mt), i = r - 4 * mt * g, n = min(4, NT - 4 * g);
            tile = i / n;
            nt = 4 * g + i - n * tile;
        }
        const int plen = bt / parts;
        u.m0 = tile * bt + part * plen;
        u.n0 = nt * kCols;
        u.live = __builtin_amdgcn_readfirstlane(min(M - u.m0, plen));
        u.s0 = (int)((int64_t)p.Kb * u.sp / split);
        u.s1 = (int)((int64_t)p.Kb * (u.sp + 1) / split);
        if (u.live <= 0) continue;
        for (int r = threadIdx.x; r < kMaxRows; r += kThreads) {      // (rows past the end repeat the last one)
            int src = u.row0 + min(u.m0 + r, M - 1);
            if (p.sorted_pairs) src = p.sorted_pairs[src] / p.k;
            s_row[r] = min(max(src, 0), p.n_x - 1);
        }
        __syncthreads();
        if (u.live > 192) {                                  // (the same barriers on both sides)
            if (__builtin_amdgcn_readfirstlane(wave_id()) >= 4) fp8_unit<PAIR, WK, 4, true>(p, u, smem, s_row);
            else fp8_unit<PAIR, WK, 4, false>(p, u, smem, s_row);
        } else if (u.live > 128) {
            if (__builtin_amdgcn_readfirstlane(wave_id()) >= 4) fp8_unit<PAIR, WK, 3, true>(p, u, smem, s_row);
            else fp8_unit<PAIR, WK, 3, false>(p, u, smem, s_row);
        } else if (u.live > 64) {
            if (__builtin_amdgcn_readfirstlane(wave_id()) >= 4) fp8_unit<PAIR, WK, 2, true>(p, u, smem, s_row);
            else fp8_unit<PAIR, WK, 2, false>(p, u, smem, s_row);
        } else {
            fp8_unit<PAIR, WK, 1, false>(p, u, smem, s_row);
        }
        __syncthreads();
    }
}

// y = the parts' sum, in order, with the residual; V values a thread
template <int V>
__global__ __launch_bounds__(256) void fp8_join_kernel(const float *__restrict__ part, size_t n, int split, const void *residual, void *y,
                                                       int y_f32) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= n) return;
    typedef float fv __attribute__((ext_vector_type(V)));
    typedef uint16_t hv __attribute__((ext_vector_type(V)));
    fv v = *(const fv *)(part + i);
#pragma unroll 4
    for (int s = 1; s < split; ++s) v += *(const fv *)(part + (size_t)s * n + i);
    if (y_f32) {
        if (residual) v += *(const fv *)((const float *)residual + i);
        *(fv *)((float *)y + i) = v;
    } else {
        hv o = {};
        if (residual) o = *(const hv *)((const uint16_t *)residual + i);
#pragma unroll
        for (int q = 0; q < V; ++q) o[q] = (uint16_t)bf16_pair(residual ? v[q] + bf16_to_f32(o[q]) : v[q], 0.0f);
        *(hv *)((uint16_t *)y + i) = o;
    }
}

template <bool PAIR, bool ROUTED, int WK>
void launch(const Fp8Product &p, int64_t bound, hipStream_t s) {
    const int g = (int)std::min<int64_t>(bound, device_cu_count());
    hipLaunchKernelGGL((fp8_gemm_kernel<PAIR, ROUTED, WK>), dim3((unsigned)g), dim3(kThreads), 0, s, p);
}

}  // namespace

moe_status fp8_product_launch(const Fp8Product &p, bool pair, hipStream_t s, const char *what) {
    const int cols = pair ? 128 : 256, NT = (p.N + cols - 1) / cols;
    const bool routed = p.offsets != nullptr;
    // (row tiles of all experts: at most one partial tile each; parts of a tile: at most 4)
    const int64_t mt = routed ? std::min<int64_t>(p.R, p.R / kMaxRows + p.E) : (p.R + p.bt - 1) / p.bt;
    const int64_t bound = 4 * mt * NT * (routed ? 1 : p.split);
    if (bound <= 0) return MOE_OK;
    if (pair) {
        if (routed) launch<true, true, MOE_FP8_SCALE_F32>(p, bound, s);
        else launch<true, false, MOE_FP8_SCALE_F32>(p, bound, s);
    } else if (routed) {
        launch<false, true, MOE_FP8_SCALE_F32>(p, bound, s);
    } else if (p.w_scale == MOE_FP8_SCALE_F32) {
        launch<false, false, MOE_FP8_SCALE_F32>(p, bound, s);
    } else if (p.w_scale == MOE_FP8_SCALE_E8M0) {
        launch<false, false, MOE_FP8_SCALE_E8M0>(p, bound, s);
    } else {
        launch<false, false, MOE_FP8_SCALE_E8M0_ROW>(p, bound, s);
    }
    MOE_TRY(launch_check(what));
    if (!routed && !pair && p.split > 1) {
        const size_t n = (size_t)p.R * p.N;
        if (n % 4 == 0)
            hipLaunchKernelGGL(fp8_join_kernel<4>, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, s, p.part, n, p.split, p.residual, p.y, p.y_f32);
        else
            hipLaunchKernelGGL(fp8_join_kernel<1>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p.part, n, p.split, p.residual, p.y, p.y_f32);
        MOE_TRY(launch_check(what));
    }
    return MOE_OK;
}

}  // namespace moe
