// The product loop of the operators' 16-bit matrix products: one work-group computes a BM x BN tile of
// out[m][q] = sum over c of P[m][c] Q[q][c], P and Q each KC or KS (gemm_tiles.h).
//
// Waves: WM x WN, each owning (BM/WM) rows and (BN/WN) columns as 16 x 16 MFMA blocks.  The MFMA's A operand
// is Q and its B operand P, so a lane's four accumulators are four consecutive columns of one row.
//
// Pipeline: NST LDS stages of one 64-deep step each, filled by LDS DMA.  Half-way through step s (its first
// 32 contraction values are being multiplied, its second fragments are on their way to registers) the
// work-group waits until stage s+1 has landed and everybody has read stage s, refills stage s with step
// s + NST and reads the first fragments of step s+1, which arrive under the second half's MFMAs.  Steps past
// the end read no memory and write zeros, so the wait count is a constant.
#pragma once

#include "gemm_tiles.h"

namespace mm {

//
// G > 1: G groups of waves take every G-th step, each in LDS stages of its own, and group 0 adds up their
// accumulators at the end.  For products with few tiles: the same tile with G times the bytes in flight and a
// G-th of the steps one after the other.
template <class T, bool kPKs, bool kQKs, int BM, int BN, int WM, int WN, int NST, int G = 1>
struct TileLoop {
    static constexpr int kGroup = WM * WN, kWaves = kGroup * G, kThreads = kWaves * 64;
    static constexpr int kRows = BM, MI = BM / 16 / WM, QI = BN / 16 / WN;
    static constexpr int kPBytes = BM * 128, kStage = (BM + BN) * 128;
    static constexpr int kStages = NST * G * kStage, kSums = (G - 1) * BM * BN * 4, kLds = kStages > kSums ? kStages : kSums;
    static constexpr int kPInstr = BM / 8 / kGroup, kQInstr = BN / 8 / kGroup, kInstr = kPInstr + kQInstr;

    // Tile row of accumulator column j, tile column of accumulator row i (first of 16)
    static __device__ __forceinline__ int row(int wave, int j) { return (wave / WN % WM * MI + j) * 16; }
    static __device__ __forceinline__ int col(int wave, int i) { return (wave % WN * QI + i) * 16; }
    using Acc = f32x4;
    static constexpr int kRun = QI;       // accumulator rows i whose columns follow each other in the tile
    // Fragment r of half kk of a stage: 0 .. QI-1 are Q's, then P's.
    static __device__ __forceinline__ void read(int r, const uint8_t* st, int kk, int wm, int wn, int lane, i32x4 (&p)[MI],
                                                i32x4 (&q)[QI]) {
        if (r < QI)
            q[r] = kQKs ? ks_frag<BN>(st + kPBytes, wn * QI + r, kk, lane) : kc_frag(st + kPBytes, wn * QI + r, kk, lane);
        else
            p[r - QI] = kPKs ? ks_frag<BM>(st, wm * MI + r - QI, kk, lane) : kc_frag(st, wm * MI + r - QI, kk, lane);
    }
    // The MFMAs of one half, with `reads` fragment reads and `loads` DMA instructions spread between them in the
    // order they are written here (sched_barrier: left alone, the compiler gathers the reads right before
    // their use).  The reads end three quarters of the way through, so the last ones arrive under the rest.
    template <int reads, int loads, class R, class D>
    static __device__ __forceinline__ void multiply(const i32x4 (&p)[MI], const i32x4 (&q)[QI], f32x4 (&acc)[QI][MI], R read_one,
                                                    D load_one) {
        constexpr int n = QI * MI;
#pragma unroll
        for (int u = 0; u < n; ++u) {
            // walk the blocks back and forth: consecutive MFMAs share a fragment
            const int i = u / MI, j = i & 1 ? MI - 1 - u % MI : u % MI;
            acc[i][j] = T::mfma(q[i], p[j], acc[i][j]);
            bool any = false;
#pragma unroll
            for (int r = 0; r < reads; ++r)
                if (r * (n * 3 / 4) / (reads ? reads : 1) == u) {
                    read_one(r);
                    any = true;
                }
#pragma unroll
            for (int d = 0; d < loads; ++d)
                if (d * n / (loads ? loads : 1) == u) {
                    load_one(d);
                    any = true;
                }
            if (any) __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // Whether this wave holds the tile's sums after run()
    static __device__ __forceinline__ bool owns(int wave) { return wave < kGroup; }
    // All waves take part; acc is overwritten.
    static __device__ __forceinline__ void run(const Operand& po, const Operand& qo, uint8_t* smem, int wave, int lane,
                                               f32x4 (&acc)[QI][MI]) {
        const int group = wave / kGroup, member = wave % kGroup;
        const auto P = PartOf<kPKs, BM, kGroup>::make(po, 0, member, lane);
        const auto Q = PartOf<kQKs, BN, kGroup>::make(qo, 0, member, lane);
        const int steps = (po.len + G * kStepK - 1) / (G * kStepK), wm = member / WN, wn = member % WN;
        uint8_t* stages = smem + group * NST * kStage;
        const uint32_t lds = lds_byte(stages);
#pragma unroll
        for (int i = 0; i < QI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NST; ++s) {
            const auto ps = P.step(s * G + group);
            const auto qs = Q.step(s * G + group);
#pragma unroll
            for (int j = 0; j < kPInstr; ++j) P.load(ps, j, lds + s * kStage, member);
#pragma unroll
            for (int j = 0; j < kQInstr; ++j) Q.load(qs, j, lds + s * kStage + kPBytes, member);
        }
        i32x4 p0[MI], q0[QI], p1[MI], q1[QI];
        wait_vm_barrier<(NST - 1) * kInstr>();
#pragma unroll
        for (int r = 0; r < QI + MI; ++r) read(r, stages, 0, wm, wn, lane, p0, q0);
        int cur = 0;
        for (int s = 0; s < steps; ++s) {
            const int nxt = cur + 1 == NST ? 0 : cur + 1;
            const uint8_t *here = stages + cur * kStage, *next = stages + nxt * kStage;
            multiply<QI + MI, 0>(p0, q0, acc, [&](int r) { read(r, here, 1, wm, wn, lane, p1, q1); }, [](int) {});
            wait_vm_barrier<(NST - 2) * kInstr>();
            __builtin_amdgcn_sched_barrier(0);
            const auto ps = P.step((s + NST) * G + group);
            const auto qs = Q.step((s + NST) * G + group);
            const uint32_t to = lds + cur * kStage;
            multiply<QI + MI, kInstr>(p1, q1, acc, [&](int r) { read(r, next, 0, wm, wn, lane, p0, q0); },
                                      [&](int d) {
                                          if (d < kPInstr) P.load(ps, d, to, member);
                                          else Q.load(qs, d - kPInstr, to + kPBytes, member);
                                      });
            cur = nxt;
        }
        // the loads past the end still write zeros to LDS: nothing may outlive the work-group or meet a reuse
        wait_vm_barrier<0>();
        if constexpr (G > 1) {
            f32x4* sums = reinterpret_cast<f32x4*>(smem) + (size_t)member * QI * MI * 64 + lane;
            constexpr int kNext = kGroup * QI * MI * 64;
            if (group > 0) {
#pragma unroll
                for (int i = 0; i < QI * MI; ++i) sums[(group - 1) * kNext + i * 64] = acc[i / MI][i % MI];
            }
            wait_vm_barrier<0>();
            if (group == 0) {
#pragma unroll
                for (int g = 0; g < G - 1; ++g)
#pragma unroll
                    for (int i = 0; i < QI * MI; ++i) acc[i / MI][i % MI] += sums[g * kNext + i * 64];
            }
            wait_vm_barrier<0>();
        }
    }
};

// The product loop for large tiles.  P and Q are each cut into two halves of rows (columns), four LDS regions per
// step and two buffers of each, and a wave owns a part of both halves, so a step is four quadrants P h x Q g:
//   A: (P0 Q0), (P0 Q1), reading Q1 and then P1 of this step from LDS
//   B: (P1 Q0), (P1 Q1), reading P0 and then Q0 of the next step
// A region is free as soon as its fragments are in registers: what A reads is refilled from B on with the step
// after next, what B reads from the next A on.  Every DMA so has one and a half steps to arrive, where a loop
// that frees whole stages gives it one with the same LDS; half of the time of that loop was this wait.
template <class T, bool kPKs, bool kQKs, int BM, int BN, int WM, int WN>
struct QuadLoop {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int kRows = BM, MI = BM / 16 / WM, QI = BN / 16 / WN, MH = MI / 2, QH = QI / 2;
    static constexpr int kPHalf = BM / 2 * 128, kQHalf = BN / 2 * 128, kLds = 4 * (kPHalf + kQHalf);
    static constexpr int kPInstr = BM / 16 / kWaves, kQInstr = BN / 16 / kWaves, kInstr = kPInstr + kQInstr;
    static constexpr int kQuad = MH * QH * 2;                 // MFMAs of a quadrant
    // LDS: P half h of buffer b, then Q half g of buffer b
    static constexpr int p_at(int b, int h) { return (b * 2 + h) * kPHalf; }
    static constexpr int q_at(int b, int g) { return 4 * kPHalf + (b * 2 + g) * kQHalf; }
    static __device__ __forceinline__ int row(int wave, int j) { return j / MH * (BM / 2) + (wave / WN * MH + j % MH) * 16; }
    static __device__ __forceinline__ int col(int wave, int i) { return i / QH * (BN / 2) + (wave % WN * QH + i % QH) * 16; }

    using Acc = f32x4;
    static constexpr int kRun = QH;       // accumulator rows i whose columns follow each other in the tile

    // Fragment r of a half: r / (blocks per half) is the half of the step, kk
    static __device__ __forceinline__ void read_p(int r, const uint8_t* at, int wm, int lane, i32x4 (&p)[2][MH]) {
        const int kk = r / MH, j = r % MH;
        p[kk][j] = kPKs ? ks_frag<BM / 2>(at, wm * MH + j, kk, lane) : kc_frag(at, wm * MH + j, kk, lane);
    }
    static __device__ __forceinline__ void read_q(int r, const uint8_t* at, int wn, int lane, i32x4 (&q)[2][QH]) {
        const int kk = r / QH, i = r % QH;
        q[kk][i] = kQKs ? ks_frag<BN / 2>(at, wn * QH + i, kk, lane) : kc_frag(at, wn * QH + i, kk, lane);
    }
    // Two quadrants' MFMAs, P half h with Q halves 0 and 1; between them the reads first(r) after every second MFMA,
    // second(r) from MFMA `from` on after every `every`, and the DMA instructions, in the order written here.
    template <int h, int first_n, int second_n, int from, int every, class F, class S, class D>
    static __device__ __forceinline__ void multiply(const i32x4 (&p)[2][MH], const i32x4 (&q0)[2][QH], const i32x4 (&q1)[2][QH],
                                                    f32x4 (&acc)[QI][MI], F first, S second, D load_one) {
#pragma unroll
        for (int u = 0; u < 2 * kQuad; ++u) {
            const int g = u / kQuad, v = u % kQuad, kk = v / (MH * QH), i = v / MH % QH;
            const int j = i & 1 ? MH - 1 - v % MH : v % MH;
            acc[g * QH + i][h * MH + j] = T::mfma(g ? q1[kk][i] : q0[kk][i], p[kk][j], acc[g * QH + i][h * MH + j]);
            bool any = false;
#pragma unroll
            for (int r = 0; r < first_n; ++r)
                if (2 * r == u) {
                    first(r);
                    any = true;
                }
#pragma unroll
            for (int r = 0; r < second_n; ++r)
                if (from + every * r == u) {
                    second(r);
                    any = true;
                }
#pragma unroll
            for (int d = 0; d < kInstr; ++d)
                if (d * kQuad / kInstr == u) {
                    load_one(d);
                    any = true;
                }
            if (any) __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    static __device__ __forceinline__ bool owns(int) { return true; }
    // All waves take part; acc is overwritten.
    static __device__ __forceinline__ void run(const Operand& po, const Operand& qo, uint8_t* smem, int wave, int lane,
                                               f32x4 (&acc)[QI][MI]) {
        const auto P0 = PartOf<kPKs, BM / 2, kWaves>::make(po, 0, wave, lane), P1 = PartOf<kPKs, BM / 2, kWaves>::make(po, BM / 2, wave, lane);
        const auto Q0 = PartOf<kQKs, BN / 2, kWaves>::make(qo, 0, wave, lane), Q1 = PartOf<kQKs, BN / 2, kWaves>::make(qo, BN / 2, wave, lane);
        const int steps = (po.len + kStepK - 1) / kStepK, wm = wave / WN, wn = wave % WN;
        const uint32_t lds = lds_byte(smem);
#pragma unroll
        for (int i = 0; i < QI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto load = [&](const auto& P, const auto& Q, int s, int p_to, int q_to) {
            const auto ps = P.step(s);
            const auto qs = Q.step(s);
#pragma unroll
            for (int d = 0; d < kPInstr; ++d) P.load(ps, d, lds + p_to, wave);
#pragma unroll
            for (int d = 0; d < kQInstr; ++d) Q.load(qs, d, lds + q_to, wave);
        };
        // groups of DMA instructions in the order of their use: (P0 Q0) of step 0, (P1 Q1) of 0, (P0 Q0) of 1, ...
        load(P0, Q0, 0, p_at(0, 0), q_at(0, 0));
        load(P1, Q1, 0, p_at(0, 1), q_at(0, 1));
        load(P0, Q0, 1, p_at(1, 0), q_at(1, 0));
        load(P1, Q1, 1, p_at(1, 1), q_at(1, 1));
        i32x4 p0[2][MH], p1[2][MH], q0[2][QH], q1[2][QH];
        wait_vm_barrier<3 * kInstr>();
#pragma unroll
        for (int r = 0; r < 2 * MH; ++r) read_p(r, smem + p_at(0, 0), wm, lane, p0);
#pragma unroll
        for (int r = 0; r < 2 * QH; ++r) read_q(r, smem + q_at(0, 0), wn, lane, q0);
        for (int s = 0; s < steps; ++s) {
            const int b = s & 1;
            const int pb = b * 2 * kPHalf, qb = b * 2 * kQHalf, pn = 2 * kPHalf - pb, qn = 2 * kQHalf - qb;
            // A: (P1 Q1) of this step has landed; (P0 Q0) of this step is in everybody's registers: refill its buffer
            wait_vm_barrier<2 * kInstr>();
            __builtin_amdgcn_sched_barrier(0);
            {
                const auto ps = P0.step(s + 2);
                const auto qs = Q0.step(s + 2);
                multiply<0, 2 * QH, 2 * MH, 4 * QH, 2>(
                    p0, q0, q1, acc, [&](int r) { read_q(r, smem + q_at(0, 1) + qb, wn, lane, q1); },
                    [&](int r) { read_p(r, smem + p_at(0, 1) + pb, wm, lane, p1); },
                    [&](int d) {
                        if (d < kPInstr) P0.load(ps, d, lds + p_at(0, 0) + pb, wave);
                        else Q0.load(qs, d - kPInstr, lds + q_at(0, 0) + qb, wave);
                    });
            }
            // B: (P0 Q0) of the next step has landed; (P1 Q1) of this step is in registers
            wait_vm_barrier<2 * kInstr>();
            __builtin_amdgcn_sched_barrier(0);
            {
                const auto ps = P1.step(s + 2);
                const auto qs = Q1.step(s + 2);
                multiply<1, 2 * MH, 2 * QH, kQuad, 1>(
                    p1, q0, q1, acc, [&](int r) { read_p(r, smem + p_at(0, 0) + pn, wm, lane, p0); },
                    [&](int r) { read_q(r, smem + q_at(0, 0) + qn, wn, lane, q0); },
                    [&](int d) {
                        if (d < kPInstr) P1.load(ps, d, lds + p_at(0, 1) + pb, wave);
                        else Q1.load(qs, d - kPInstr, lds + q_at(0, 1) + qb, wave);
                    });
            }
        }
        wait_vm_barrier<0>();
    }
};

// The epilogue: the accumulators of a wave go through its share of LDS (the stages are free by now), 16 rows of one
// run of columns at a time, so that a store instruction covers whole rows of the run, 16 bytes a lane.  Straight
// from the accumulators it would touch 16 rows by 32 (fp32: 64) bytes; those 256 instructions of 16 partial lines
// each took 7 us of a 256 x 256 tile.  put(place in the row, row, column, lane's 16 bytes) is called for what exists.
// kBytes: of an output value.
template <class L, int kBytes, class W, class P>
__device__ __forceinline__ void store_tile(const typename L::Acc (&acc)[L::QI][L::MI], uint8_t* smem, int rows, int cols, int wave,
                                           int lane, W write_lane, P put) {
    constexpr int kRun = L::kRun, kRow = 16 * kRun * kBytes, kStride = kRow + 16, kBlock = 16 * kStride;
    constexpr int kShare = L::kLds / L::kWaves / 16 * 16, kSlots = kShare / kBlock;
    static_assert(kSlots >= 1, "a block of rows fits a wave's share of LDS");
    constexpr int kChunks = kRow / 16, kPer = 16 / kBytes;        // 16-byte chunks of a row, values of a chunk
    if (!L::owns(wave)) return;
    uint8_t* mine = smem + wave * kShare;
#pragma unroll
    for (int j = 0; j < L::MI; ++j)
#pragma unroll
        for (int run = 0; run < L::QI / kRun; ++run) {
            // a wave's LDS accesses are served in order: a slot is written again only after its reads
            uint8_t* slot = mine + (j * (L::QI / kRun) + run) % kSlots * kBlock;
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                write_lane(slot + (lane & 15) * kStride + (i * 16 + (lane >> 4) * 4) * kBytes, acc[run * kRun + i][j]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int t = 0; t < (16 * kChunks + 63) / 64; ++t) {
                const int at = t * 64 + lane, r = at / kChunks, c = at % kChunks;
                const int m = L::row(wave, j) + r, col = L::col(wave, run * kRun) + c * kPer;
                if (r < 16 && m < rows && col < cols) put(m, col, *reinterpret_cast<const i32x4*>(slot + r * kStride + c * 16));
            }
            __builtin_amdgcn_wave_barrier();
        }
}
// 16-bit rows: out points at the tile's first row and column, ld values apart.
template <class L, class T>
__device__ __forceinline__ void store_halves(const typename L::Acc (&acc)[L::QI][L::MI], uint16_t* out, int rows, int cols, int ld,
                                             uint8_t* smem, int wave, int lane) {
    store_tile<L, 2>(
        acc, smem, rows, cols, wave, lane,
        [](uint8_t* p, f32x4 v) { *reinterpret_cast<u32x2*>(p) = u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])}; },
        [&](int m, int c, i32x4 v) { *reinterpret_cast<i32x4*>(out + (size_t)m * ld + c) = v; });
}

// A stream of tiles with two KS operands, for products whose contraction is short beside their output: QuadLoop's
// steps one tile after the other, the next tile's first two steps loading under the last two of the current one, and
// the output's stores completing under the first steps of the next.  (A tile per work-group spent as long on its first
// loads and its stores as on eight steps' MFMAs.)
//
// The waits count instructions, and stores count like loads, in order: after a tile's kStores stores the three waits
// for groups that were issued before them allow that many more to be outstanding.  So the number of stores of a tile
// is a constant: the stores of rows or columns that do not exist go past their descriptor's end.  Operations retire in
// order, so the fourth wait, one and a half steps (2 us) into the next tile, is for all of the stores; a CU's share of
// the fill rate takes about 10 us for a tile's 256 KB of fp32.  Their issue has no MFMA beside it.
//
// Tiles: next() gives the stream's next tile, made by of(); one without steps is its end.
template <class T, int kBytes>
struct KsStream {
    static constexpr int BM = 256, BN = 256;
    using L = QuadLoop<T, true, true, BM, BN, 4, 2>;
    static constexpr int kThreads = L::kThreads, MI = L::MI, QI = L::QI, MH = L::MH, QH = L::QH, kInstr = L::kInstr;
    // 16 rows of 128 bytes, and their padding, per wave beside the stages
    static constexpr int kRun = 8 / kBytes, kStride = 128 + 16, kSlot = 16 * kStride;
    static constexpr int kLds = L::kLds + L::kWaves * kSlot;
    static constexpr int kStores = MI * (QI / kRun) * 2;
    static_assert(2 * kInstr + kStores < 64, "vmcnt");
    using Lanes = KsLanes<BM / 2, L::kWaves>;

    // All wave-uniform (readfirstlane in of()).
    struct Tile {
        const uint16_t *p, *q;     // contraction row 0, column 0 of the operands
        int p_col, q_col;          // the tile's first columns
        int len, steps;            // contraction; at least two steps, so that a step's loads belong to its tile or the next
        char* out;                 // first row and column of the tile
        int rows, cols;            // that exist from there on
    };
    template <class U>
    static __device__ __forceinline__ U* uniform(U* ptr) {
        const uint64_t v = (uint64_t)(uintptr_t)ptr;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
        return (U*)(uintptr_t)((uint64_t)hi << 32 | lo);
    }
    static __device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
    // exists: false for the end of the stream (no steps, and nothing is read)
    static __device__ __forceinline__ Tile of(bool exists, const uint16_t* p, int p_col, const uint16_t* q, int q_col, int len, char* out,
                                              int rows, int cols) {
        const int n = exists ? uniform(len) : 0;
        return Tile{uniform(p),   uniform(q),    uniform(p_col), uniform(q_col), n, exists ? max((n + kStepK - 1) / kStepK, 2) : 0,
                    uniform(out), uniform(rows), uniform(cols)};
    }
    static __device__ __forceinline__ Tile either(bool first, const Tile& a, const Tile& b) {
        return Tile{first ? a.p : b.p,         first ? a.q : b.q,       first ? a.p_col : b.p_col,
                    first ? a.q_col : b.q_col, first ? a.len : b.len,   first ? a.steps : b.steps,
                    first ? a.out : b.out,     first ? a.rows : b.rows, first ? a.cols : b.cols};
    }

    // Accumulators to `out` through the wave's slot, kStores store instructions; each lane's 16 bytes go through
    // change(address, bytes) where they exist.
    template <class C>
    static __device__ __forceinline__ void store(const Tile& t, int ld, const f32x4 (&acc)[QI][MI], uint8_t* slot, int wave,
                                                 C change) {
        const uint32_t ldb = (uint32_t)ld * kBytes;
        // addresses are computed here and not before the steps, whose registers are full
        int lane = __lane_id();
        asm volatile("" : "+v"(lane));
        const auto desc = __builtin_amdgcn_make_buffer_rsrc(t.out, 0, (int)((uint32_t)min(t.rows, BM) * ldb), 0x00020000);
#pragma unroll
        for (int j = 0; j < MI; ++j)
#pragma unroll
            for (int run = 0; run < QI / kRun; ++run) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    const f32x4 v = acc[run * kRun + i][j];
                    uint8_t* at = slot + (lane & 15) * kStride + (i * 16 + (lane >> 4) * 4) * kBytes;
                    if constexpr (kBytes == 4) *reinterpret_cast<f32x4*>(at) = v;
                    else *reinterpret_cast<u32x2*>(at) = u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = h * 8 + (lane >> 3), m = L::row(wave, j) + r;
                    const int c = L::col(wave, run * kRun) + (lane & 7) * (16 / kBytes);
                    i32x4 v = *reinterpret_cast<const i32x4*>(slot + r * kStride + (lane & 7) * 16);
                    const bool exists = m < t.rows && c < t.cols;
                    const uint32_t off = exists ? (uint32_t)m * ldb + (uint32_t)c * kBytes : kPastEnd;
                    v = change(t.out + off, exists, v);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), desc, (int)off, 0, 0);
                }
                __builtin_amdgcn_wave_barrier();
            }
    }

    template <class N, class C>
    static __device__ __forceinline__ void run(N next, int ld_p, int ld_q, int ld_out, uint8_t* smem, int wave, int lane,
                                               C change) {
        const int wm = wave / 2, wn = wave % 2;
        const uint32_t lds = lds_byte(smem);
        uint8_t* slot = smem + L::kLds + wave * kSlot;
        const Lanes lp(ld_p, wave, lane), lq(ld_q, wave, lane);
        Tile cur = next();
        if (cur.steps == 0) return;
        Tile ahead = next();
        f32x4 acc[QI][MI];
        i32x4 p0[2][MH], p1[2][MH], q0[2][QH], q1[2][QH];
        const auto p_step = [&](const Tile& t, int h, int s) { return KsWhere(t.p, t.p_col + h * (BM / 2), ld_p, t.len).step(s); };
        const auto q_step = [&](const Tile& t, int h, int s) { return KsWhere(t.q, t.q_col + h * (BN / 2), ld_q, t.len).step(s); };
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 ps = p_step(cur, h, s), qs = q_step(cur, h, s);
#pragma unroll
                for (int d = 0; d < L::kPInstr; ++d) lp.load(ps, d, lds + L::p_at(s, h), wave);
#pragma unroll
                for (int d = 0; d < L::kQInstr; ++d) lq.load(qs, d, lds + L::q_at(s, h), wave);
            }
        wait_vm_barrier<3 * kInstr>();
#pragma unroll
        for (int r = 0; r < 2 * MH; ++r) L::read_p(r, smem + L::p_at(0, 0), wm, lane, p0);
#pragma unroll
        for (int r = 0; r < 2 * QH; ++r) L::read_q(r, smem + L::q_at(0, 0), wn, lane, q0);
        int b = 0, waits = 0;            // waits: how many more may leave a tile's stores outstanding
        const auto wait = [&] {
            if (waits > 0) {
                wait_vm_barrier<2 * kInstr + kStores>();
                --waits;
            } else {
                wait_vm_barrier<2 * kInstr>();
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        while (true) {
#pragma unroll
            for (int i = 0; i < QI; ++i)
#pragma unroll
                for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < cur.steps; ++s) {
                const int pb = b * 2 * L::kPHalf, qb = b * 2 * L::kQHalf, pn = 2 * L::kPHalf - pb, qn = 2 * L::kQHalf - qb;
                const bool here = s + 2 < cur.steps;
                const int s2 = here ? s + 2 : s + 2 - cur.steps;
                const Tile t = either(here, cur, ahead);
                wait();
                {
                    const u32x4 ps = p_step(t, 0, s2), qs = q_step(t, 0, s2);
                    L::template multiply<0, 2 * QH, 2 * MH, 4 * QH, 2>(
                        p0, q0, q1, acc, [&](int r) { L::read_q(r, smem + L::q_at(0, 1) + qb, wn, lane, q1); },
                        [&](int r) { L::read_p(r, smem + L::p_at(0, 1) + pb, wm, lane, p1); },
                        [&](int d) {
                            if (d < L::kPInstr) lp.load(ps, d, lds + L::p_at(0, 0) + pb, wave);
                            else lq.load(qs, d - L::kPInstr, lds + L::q_at(0, 0) + qb, wave);
                        });
                }
                wait();
                {
                    int l = lane;                // read addresses again, for want of registers to keep them
                    asm volatile("" : "+v"(l));
                    const u32x4 ps = p_step(t, 1, s2), qs = q_step(t, 1, s2);
                    L::template multiply<1, 2 * MH, 2 * QH, L::kQuad, 1>(
                        p1, q0, q1, acc, [&](int r) { L::read_p(r, smem + L::p_at(0, 0) + pn, wm, l, p0); },
                        [&](int r) { L::read_q(r, smem + L::q_at(0, 0) + qn, wn, l, q0); },
                        [&](int d) {
                            if (d < L::kPInstr) lp.load(ps, d, lds + L::p_at(0, 1) + pb, wave);
                            else lq.load(qs, d - L::kPInstr, lds + L::q_at(0, 1) + qb, wave);
                        });
                }
                b ^= 1;
            }
            store(cur, ld_out, acc, slot, wave, change);
            waits = 3;
            if (ahead.steps == 0) break;
            cur = ahead;
            ahead = next();
        }
        wait_vm_barrier<0>();
    }
};

// Which tile shape a row product of these sizes runs with (forward and backward of the groups, the adapters'
// shared product).  The time is estimated as `fixed` + steps * (a tile's time per step) * (rounds of tiles over the
// CUs), with the microseconds that every shape measured: `alone` with one tile to a CU, `full` with `resident` tiles
// on every CU.  The shapes in this order, bf16: at 21474 x 4344 x 7912 over 13 groups 1.67 ms, 2.12, 2.81, 3.1, 4.9,
// 3.6, 5.8, 6.5; at 1500 x 2048 x 4096 over 4 groups 90, 49, 35, 47, 68, 44, 82, 85 us; at 1999 x 1000 x 2056 over 10
// groups 45, 33, 24, 32, 39, 35, 40, 47; at 512 x 2048 x 8192 over 2 groups 148, 82, 54, 56, 57, 37, 67, 60; at 1024 x
// 7168 x 2048 over 32 groups (weights streamed) 215, 212, 201, 188, 191, 204, 204, 240; at 6 x 696 x 2096, one group,
// 24, 17, 13, 17, 13, 12, 10, 9.
// Over 56 sizes drawn from 4 to 32768 rows, 1 to 64 groups and 128 to 8192 columns, both directions, the shape picked took
// 1.5 % longer than the best of these shapes on average and 16 % at most.  `fixed` counts once, though every round of
// tiles has first loads and an epilogue: of a contraction of one or two steps over many rounds the estimate is too
// low (32768 x 7168 over 8 groups, contraction 64: 32 us estimated, 118 measured, 96 its bytes at a copy's rate).
struct RowShape {
    int bm, bn, resident;
    double fixed, alone, full;
};
enum { kShape256, kShape128, kShapeSquare, kShape64, kShape32, kShapeHalved, kShapeLeast, kShapeDeep };
constexpr RowShape kRowShapes[] = {{256, 256, 1, 8.5, 1.08, 1.60},    // quadrants
                                   {128, 256, 1, 5.5, 0.58, 1.02},
                                   {128, 128, 1, 5.0, 0.34, 0.62},    // four stages: three steps for a load to arrive
                                   {64, 128, 2, 4.2, 0.40, 0.84},
                                   {32, 128, 2, 3.8, 0.29, 0.67},
                                   {64, 128, 1, 4.6, 0.31, 0.52},     // two groups of waves along the contraction
                                   {32, 64, 2, 3.6, 0.17, 0.37},      // the forward's only, and the next
                                   {32, 64, 1, 4.8, 0.125, 0.26}};    // four groups
// choices: how many of them the product has.  Groups end inside a tile, half a tile to a group on average, or have one
// tile each where they are short.
inline int pick_row_shape(int rows, int cols, int depth, int groups, int choices) {
    int best = 0;
    double least = 0;
    const int used = groups < rows ? groups : rows;
    const double steps = (depth + kStepK - 1) / kStepK;
    for (int i = 0; i < choices; ++i) {
        const RowShape& s = kRowShapes[i];
        const double row_tiles = groups == 1                       ? (rows + s.bm - 1) / s.bm
                                 : (double)rows < 0.6 * s.bm * used ? used
                                                                    : (double)rows / s.bm + 0.5 * used;
        const double tiles = row_tiles * ((cols + s.bn - 1) / s.bn), rounds = tiles / (256.0 * s.resident);
        // one group's tiles are counted exactly, and one more than a round holds starts another; the count of several is
        // an estimate, and their short last tiles soften the step
        const double whole = (double)(int64_t)(rounds + (groups == 1 ? 1.0 - 1e-9 : 0.95));
        const double per_step = tiles <= 256 ? s.alone : s.full * (rounds > 1 ? whole : 1.0);
        const double t = s.fixed + steps * per_step;
        if (i == 0 || t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

}  // namespace mm
