// The product loop of the weight gradient from 8-bit rows, gfx950 only: one work-group of four waves computes a 256 x 128
// tile of out[p][q] = sum over c of P[c][p] X[c][q], where P is 16-bit and X = codes * scales with a scale per row c and 128
// columns q: one scale per row of a tile.  A scale differs from one contraction index to the next, so codes cannot enter an
// MFMA and be scaled behind it; they become 16-bit numbers in LDS, once per tile.
//
// Two work-groups share a CU (79 KB of LDS each), so that the stores of one tile, the first loads of the next and the waits
// at a step's barrier meet the other one's MFMAs.
//
// Steps of 32 contraction rows, everything loaded by LDS DMA.  P goes to three stages of KS tiles (gemm_tiles.h), the
// codes and their scales to three stages as they are.  During step s a wave
//   multiplies P and X of step s,
//   starts the loads of P for step s + 2 and of the codes for step s + 3,
//   reads its codes of step s + 1, which it loaded itself, and writes them as 16-bit numbers to the other one of X's two stages.
// So a load has two steps to arrive.  Rows behind the group's end are zeros in both operands and are not read.
//
// Measured, bf16: 2000 rows in 10 groups, 1000 x 2056, 24 us, and 28 for the product of the same rows in 16 bits; 8 groups of 1024,
// 2048 x 2048, 72 and 70; one group of 16384, 4096 x 4096, 470 (1170 TFLOP/s) and 430.  Many steps over many tiles are bound by the loads'
// latency beside the MFMAs: of 1995 us (32 groups of 1024, 4096 x 7168), 1390 remain without loads, 1725 with loads that meet L2,
// 1745 without the conversion.
#pragma once

#include "gemm_kernels.h"

namespace mm {

// 4 bytes per lane, as dma_rows.
__device__ __forceinline__ void dma_words(u32x4 desc, uint32_t off, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :: "v"(off), "s"(desc), "s"(__builtin_amdgcn_readfirstlane(dst)) : "memory", "m0");
}

template <class T>
struct CodesLoop {
    static constexpr int BM = 256, BN = 128, kDepth = 32, kWaves = 4, kThreads = 256, WM = 2, WN = 2;
    static constexpr int MI = BM / 16 / WM, QI = BN / 16 / WN, kRun = QI;
    static constexpr int kP = kDepth * BM * 2, kX = kDepth * BN * 2, kRaw = kDepth * BN, kScales = kWaves * 256;
    static constexpr int kXAt = 3 * kP, kRawAt = kXAt + 2 * kX, kScalesAt = kRawAt + 3 * kRaw, kLds = kScalesAt + 3 * kScales;
    static constexpr int kPInstr = kDepth * BM * 2 / 1024 / kWaves, kInstr = kPInstr + 2;     // DMA instructions of a wave and step
    static_assert(2 * kLds <= 160 * 1024, "two to a CU");
    using Acc = f32x4;
    static __device__ __forceinline__ int row(int wave, int j) { return (wave / WN * MI + j) * 16; }
    static __device__ __forceinline__ int col(int wave, int i) { return (wave % WN * QI + i) * 16; }
    static __device__ __forceinline__ bool owns(int) { return true; }

    // One operand's rows of the step that is loaded next; wave-uniform.
    struct Rows {
        const char* base;          // first row, first column of the tile
        uint32_t step;             // bytes of a step's rows
        uint32_t full, tail;       // bytes that may be read from `base`: of a whole step, and of the last one
        __device__ __forceinline__ Rows(const void* p, uint32_t ld, uint32_t skip, int rows) {
            base = static_cast<const char*>(p) + skip;
            step = kDepth * ld;
            full = step - skip;
            tail = (uint32_t)((rows - 1) % kDepth + 1) * ld - skip;
        }
        __device__ __forceinline__ u32x4 next(int left) {
            const u32x4 d = buffer_of(base, left >= kDepth ? full : left > 0 ? tail : 0u);
            base += step;
            return d;
        }
    };
    struct Operands {
        Rows p, x, s;
        int left_p, left_x;                // contraction rows from the next step of P and of X on
        uint32_t at_p[kPInstr], at_x, at_s;
        uint32_t lds;                      // of the work-group
        int wave;
        __device__ __forceinline__ void load_p(const u32x4& d, int j, int stage) const {
            dma_rows(d, at_p[j], lds + stage * kP + (wave + j * kWaves) * 1024);
        }
        // Each wave has its own copy of a step's 32 scales.
        __device__ __forceinline__ void load_x(int stage) {
            const u32x4 dx = x.next(left_x), ds = s.next(left_x);
            dma_rows(dx, at_x, lds + kRawAt + stage * kRaw + wave * 1024);
            dma_words(ds, at_s, lds + kScalesAt + stage * kScales + wave * 256);
            left_x -= kDepth;
        }
    };

    // Places of a thread: of its 16 codes as 16-bit numbers, and of fragment reads.  Codes become one 32-byte pair of X.  A
    // write of 16 bytes a lane takes 8 lanes at a time, here the 8 pairs of a row: the halves of pairs 4 .. 7 are swapped, so
    // that their first (second) halves fill 128 bytes of banks (unswapped, a write took 13 cycles and not 8).
    struct Places {
        const uint8_t *raw, *scale;
        uint8_t* put[2];
        const uint8_t *get_p[MI], *get_x[QI];
        __device__ __forceinline__ Places(uint8_t* smem, int wave, int lane) {
            const int r = threadIdx.x >> 3, c = threadIdx.x & 7, at = c ^ ks_swz(r);
            raw = smem + kRawAt + threadIdx.x * 16;
            scale = smem + kScalesAt + wave * 256 + r * 4;
            put[0] = smem + kXAt + r * (BN * 2) + (at << 5) + (at & 4 ? 16 : 0);
            put[1] = smem + kXAt + r * (BN * 2) + (at << 5) + (at & 4 ? 0 : 16);
            const int k = (lane >> 4) * 8 + ((lane & 15) >> 2), wm = wave / WN, wn = wave % WN;      // as in ks_frag
#pragma unroll
            for (int j = 0; j < MI; ++j) get_p[j] = smem + k * (BM * 2) + (((wm * MI + j) ^ ks_swz(k)) << 5) + (lane & 3) * 8;
#pragma unroll
            for (int i = 0; i < QI; ++i) {
                const int pair = (wn * QI + i) ^ ks_swz(k);
                get_x[i] = smem + kXAt + k * (BN * 2) + (pair << 5) + (((lane & 3) * 8) ^ (pair & 4 ? 16 : 0));
            }
        }
    };
    template <int W>
    static __device__ __forceinline__ i32x4 fragment(const uint8_t* at) {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(void*)const_cast<uint8_t*>(at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(void*)const_cast<uint8_t*>(at + 4 * W * 2));
        const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
        return i32x4{(int)a[0], (int)a[1], (int)b[0], (int)b[1]};
    }
    // Half h of the thread's 16 codes as 16-bit numbers: the product with the scale in fp32, then rounded, which changes nothing
    // where the scale is a power of two (the hardware's scaled conversion of two codes, which takes such scales only, saved 2 to 4 %
    // with many rows and would need a second loop for other scales).  upper: of the row's last 8 columns, which were loaded
    // together with the 8 before them.
    static __device__ __forceinline__ u32x4 numbers(const u32x4& codes, float s, int h, bool upper) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = (int)(h == 0 && upper ? codes[2 + i] : codes[2 * h + i]);
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            v[2 * i] = T::pack(restored<T>(a[0] * s), restored<T>(a[1] * s));
            v[2 * i + 1] = T::pack(restored<T>(b[0] * s), restored<T>(b[1] * s));
        }
        return v;
    }

    // P [rows][ldp] from column m0 on, X (codes [rows][ldx], ldx >= 16, scales [rows][lds]) from column q0 on.  All waves
    // take part; acc is overwritten.
    static __device__ __forceinline__ void run(const uint16_t* p, int ldp, int m0, const uint8_t* x, int ldx, int q0, const float* scales, int lds,
                                               int rows, uint8_t* smem, int wave, int lane, f32x4 (&acc)[QI][MI]) {
#pragma unroll
        for (int i = 0; i < QI; ++i)
#pragma unroll
            for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (rows == 0) return;
        const int from = max(q0 - 8, 0);             // 8 columns ahead of the tile, where there are any
        Operands o{Rows(p, (uint32_t)ldp * 2, (uint32_t)m0 * 2, rows), Rows(x, (uint32_t)ldx, (uint32_t)from, rows),
                   Rows(scales, (uint32_t)lds * 4, (uint32_t)(q0 / 128) * 4, rows), rows, rows, {}, 0, 0, lds_byte(smem), wave};
#pragma unroll
        for (int j = 0; j < kPInstr; ++j) {      // an instruction covers two rows of 512 bytes
            const int r = (wave + j * kWaves) * 2 + (lane >> 5), pos = lane & 31;
            o.at_p[j] = (uint32_t)(r * ldp * 2 + (((((pos >> 1) ^ ks_swz(r)) << 1) | (pos & 1)) << 4));
        }
        const int r = threadIdx.x >> 3, first = q0 + (int)(threadIdx.x & 7) * 16;
        // the row's last 8 columns come with the 8 before them, so that every load lies inside its row
        const bool upper = first < ldx && first + 16 > ldx;
        o.at_x = first < ldx ? (uint32_t)(r * ldx + first - from - (upper ? 8 : 0)) : kPastEnd;
        o.at_s = lane < kDepth ? (uint32_t)(lane * lds * 4) : kPastEnd;
        const Places d(smem, wave, lane);
        const int steps = (rows + kDepth - 1) / kDepth;
        // the codes of step 0, then P and the codes as the steps -2 and -1 would have started them
        o.load_x(0);
        for (int s = 0; s < 2; ++s) {
            const u32x4 dp = o.p.next(o.left_p);
            o.left_p -= kDepth;
#pragma unroll
            for (int j = 0; j < kPInstr; ++j) o.load_p(dp, j, s);
            o.load_x(s + 1);
        }
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kInstr) : "memory");
        {
            const u32x4 codes = *reinterpret_cast<const u32x4*>(d.raw);
            const float scale = *reinterpret_cast<const float*>(d.scale);
#pragma unroll
            for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4*>(d.put[h]) = numbers(codes, scale, h, upper);
        }
        int st = 0;                                  // s % 3
        for (int s = 0; s < steps; ++s) {
            const int next = st == 2 ? 0 : st + 1, then = st == 0 ? 2 : st - 1;
            // P of step s and the codes of step s + 1 have landed, X of step s is written, and everybody is done with step s - 1
            wait_vm_barrier<kInstr>();
            __builtin_amdgcn_sched_barrier(0);
            const int pa = st * kP, xa = (s & 1) * kX;
            i32x4 q[QI], f[3];
#pragma unroll
            for (int i = 0; i < QI; ++i) q[i] = fragment<BN>(d.get_x[i] + xa);
#pragma unroll
            for (int j = 0; j < 2; ++j) f[j] = fragment<BM>(d.get_p[j] + pa);
            const u32x4 codes = *reinterpret_cast<const u32x4*>(d.raw + next * kRaw);
            const float scale = *reinterpret_cast<const float*>(d.scale + next * kScales);
            const u32x4 dp = o.p.next(o.left_p);
            o.left_p -= kDepth;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < MI; ++j) {
                if (j + 2 < MI) f[(j + 2) % 3] = fragment<BM>(d.get_p[(j + 2) % MI] + pa);
                if (j < kPInstr) o.load_p(dp, j, then);
                if (j == 2 || j == 3) *reinterpret_cast<u32x4*>(d.put[j - 2] + (kX - xa)) = numbers(codes, scale, j - 2, upper);
                if (j == 4) o.load_x(st);            // where the codes of step s were, which step s - 1 took
#pragma unroll
                for (int i = 0; i < QI; ++i) acc[i][j] = T::mfma(q[i], f[j % 3], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            st = next;
        }
        wait_vm_barrier<0>();                        // the loads past the end write LDS as well
    }
};

}  // namespace mm
