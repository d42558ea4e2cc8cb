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

template <class T, bool kPKs, bool kQKs, int BM, int BN, int WM, int WN, int NST>
struct TileLoop {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MI = BM / 16 / WM, QI = BN / 16 / WN;
    static constexpr int kPBytes = BM * 128, kStage = (BM + BN) * 128, kLds = NST * kStage;
    static constexpr int kPInstr = BM / 8 / kWaves, kQInstr = BN / 8 / kWaves, kInstr = kPInstr + kQInstr;

    static __device__ __forceinline__ void frags(const uint8_t* st, int kk, int wm, int wn, int lane, i32x4 (&p)[MI],
                                                 i32x4 (&q)[QI]) {
#pragma unroll
        for (int i = 0; i < QI; ++i)
            q[i] = kQKs ? ks_frag<BN>(st + kPBytes, wn * QI + i, kk, lane) : kc_frag(st + kPBytes, wn * QI + i, kk, lane);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            p[i] = kPKs ? ks_frag<BM>(st, wm * MI + i, kk, lane) : kc_frag(st, wm * MI + i, kk, lane);
    }
    static __device__ __forceinline__ void multiply(const i32x4 (&p)[MI], const i32x4 (&q)[QI], f32x4 (&acc)[QI][MI]) {
#pragma unroll
        for (int i = 0; i < QI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = T::mfma(q[i], p[j], acc[i][j]);
    }
    // PT, QT: KcTile or KsTile.  All waves take part; acc is overwritten.
    template <class PT, class QT>
    static __device__ __forceinline__ void run(const PT& P, const QT& Q, int steps, uint8_t* smem, int wave, int lane,
                                               f32x4 (&acc)[QI][MI]) {
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t lds = lds_byte(smem);
#pragma unroll
        for (int i = 0; i < QI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NST; ++s) {
            P.load(s, lds + s * kStage, wave);
            Q.load(s, lds + s * kStage + kPBytes, wave);
        }
        i32x4 p0[MI], q0[QI], p1[MI], q1[QI];
        wait_vm_barrier<(NST - 1) * kInstr>();
        frags(smem, 0, wm, wn, lane, p0, q0);
        int cur = 0;
        for (int s = 0; s < steps; ++s) {
            const int nxt = cur + 1 == NST ? 0 : cur + 1;
            frags(smem + cur * kStage, 1, wm, wn, lane, p1, q1);
            multiply(p0, q0, acc);
            wait_vm_barrier<(NST - 2) * kInstr>();
            P.load(s + NST, lds + cur * kStage, wave);
            Q.load(s + NST, lds + cur * kStage + kPBytes, wave);
            frags(smem + nxt * kStage, 0, wm, wn, lane, p0, q0);
            multiply(p1, q1, acc);
            cur = nxt;
        }
        // the loads past the end still write zeros to LDS: nothing may outlive the work-group or meet a reuse
        wait_vm_barrier<0>();
    }
};

}  // namespace mm
